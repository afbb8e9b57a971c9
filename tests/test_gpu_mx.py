"""The microscaled 4-bit operators on cuda:0 against their definition in 64
bits (mx_reference): quantisation byte for byte, products within the bound of
their F32 sums."""

import pytest
import torch

import mx_reference as ref

pytestmark = pytest.mark.gpu

FLOATS = [torch.float32, torch.float16, torch.bfloat16]
NAME = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    import quantized_weight_backward_amd as q

    return q


def gen(seed):
    return torch.Generator().manual_seed(seed)


def values(rows, cols, dtype, seed, sigma=1.0):
    """Normal values with wide columns, a zero row, and ties of the grid."""
    g = gen(seed)
    x = torch.randn((rows, cols), generator=g) * sigma
    x *= torch.where(torch.rand((1, cols), generator=g) < 0.05, 16.0, 1.0)
    if rows > 2:
        x[rows // 2] = 0
    ties = torch.randint(0, 25, (rows, cols), generator=g) * 0.25
    x = torch.where(torch.rand((rows, cols), generator=g) < 0.1, ties * sigma, x)
    return x.to(dtype)


def check_planes(m, codes, e, K, where):
    want_c, want_s = ref.planes(codes, e, K)
    blocks = codes.shape[1]
    got_s = m.scales.cpu().permute(1, 0, 2).flatten(1)
    assert torch.equal(got_s[:, :blocks], want_s.permute(1, 0, 2).flatten(1)[:, :blocks]), where
    assert not (got_s[:, blocks:] == 255).any(), where
    fine = (e != 255).repeat_interleave(16, dim=1)
    got_c = m.codes.cpu()
    assert torch.equal(got_c[:, :blocks * 16][fine], want_c[:, :blocks * 16][fine]), where
    assert not got_c[:, blocks * 16:].any(), where


SHAPES = [(1, 1), (1, 32), (3, 31), (5, 33), (2, 255), (9, 256), (7, 257), (33, 64), (64, 96), (130, 300), (255, 130),
          (257, 72), (1, 5000), (600, 8), (512, 512)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
def test_quantize_rows_cols_and_both(q, dtype, shape):
    x = values(*shape, dtype, seed=hash(shape) % 1000)
    d = x.cuda()
    rows, cols = ref.mx_encode(x), ref.mx_encode(x.T)
    check_planes(q.mx_quantize(d), *rows, shape[1], "rows")
    check_planes(q.mx_quantize(d, axis=0), *cols, shape[0], "cols")
    r, c = q.mx_quantize_both(d)
    check_planes(r, *rows, shape[1], "both: rows")
    check_planes(c, *cols, shape[0], "both: cols")
    assert torch.equal(q.mx_dequantize(r).cpu().double(), ref.mx_values(*rows, shape[1]))
    assert torch.equal(q.mx_dequantize(c, torch.bfloat16).cpu().double(), ref.mx_values(*cols, shape[0]))


@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (8, 8), (8, 3), (5, 1)])
@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
def test_quantize_takes_views_of_any_alignment(q, dtype, pad, offset):
    x = values(70, 200, dtype, seed=3)
    wide = torch.full((70, 200 + pad + offset), float("nan"), dtype=dtype, device="cuda")
    view = wide[:, offset:offset + 200]
    view.copy_(x)
    r, c = q.mx_quantize_both(view)
    check_planes(r, *ref.mx_encode(x), 200, "rows")
    check_planes(c, *ref.mx_encode(x.T), 70, "cols")
    check_planes(q.mx_quantize(view), *ref.mx_encode(x), 200, "rows alone")
    check_planes(q.mx_quantize(view, axis=0), *ref.mx_encode(x.T), 70, "cols alone")
    assert torch.equal(q.quantize(q.MXFP4, view[:, :192]).cpu(), ref.mxfp4_bytes(*ref.mx_encode(x[:, :192])))
    assert torch.equal(q.quantize(q.NVFP4, view[:, :192]).cpu(), ref.nvfp4_bytes(x[:, :192])[0])


@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
def test_quantize_extreme_blocks(q, dtype):
    """Zero, subnormal, smallest, largest and non-finite blocks."""
    info = torch.finfo(dtype)
    x = torch.zeros((8, 64), dtype=dtype)
    x[1, 3] = info.max
    x[1, 4] = -info.max
    x[1, 40] = info.tiny
    x[2, 0] = info.smallest_normal / 4  # subnormal
    x[2, 33] = -info.smallest_normal
    x[3, 5] = float("inf")
    x[3, 40] = 1.0
    x[4, 6] = float("nan")
    x[5, 7] = -float("inf")
    x[6] = 6.0
    x[7] = -0.0
    codes, e = ref.mx_encode(x)
    d = x.cuda()
    m = q.mx_quantize(d)
    check_planes(m, codes, e, 64, "rows")
    check_planes(q.mx_quantize(d, axis=0), *ref.mx_encode(x.T), 8, "cols")
    back = q.mx_dequantize(m).cpu().double()
    want = ref.mx_values(codes, e, 64)
    assert torch.equal(torch.isnan(back), torch.isnan(want))
    assert torch.equal(back.nan_to_num(), want.nan_to_num())
    W = q.quantize(q.MXFP4, d)
    back = q.dequantize(q.MXFP4, W, 64, 8).cpu().double()
    assert torch.equal(torch.isnan(back), torch.isnan(want))
    assert torch.equal(back.nan_to_num(), want.nan_to_num())
    W = q.quantize(q.NVFP4, d)
    want, bad = ref.nvfp4_bytes(x)
    assert torch.equal(W.cpu()[:, :4], want[:, :4])
    fine = ~bad.repeat_interleave(8, dim=1)
    assert torch.equal(W.cpu()[:, 4:][fine], want[:, 4:][fine])


@pytest.mark.parametrize("shape", [(1, 64), (3, 128), (50, 320), (17, 4096)], ids=str)
@pytest.mark.parametrize("sigma", [1e-3, 1.0, 300.0])
@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
def test_packed_blocks(q, dtype, sigma, shape):
    x = values(*shape, dtype, seed=11, sigma=sigma)
    d = x.cuda()
    codes, e = ref.mx_encode(x)
    W = q.quantize(q.MXFP4, d)
    assert torch.equal(W.cpu(), ref.mxfp4_bytes(codes, e))
    assert torch.equal(q.quantize(q.NVFP4, d).cpu(), ref.nvfp4_bytes(x)[0])
    m = q.mx_from_blocks(W, shape[1], shape[0])
    check_planes(m, codes, e, shape[1], "from blocks")
    assert torch.equal(q.mx_dequantize(m), q.dequantize(q.MXFP4, W, shape[1], shape[0]))


def test_nvfp4_scales_at_every_middle(q):
    """amax on, just below and just above six times each middle of two E4M3
    values, and elements on and beside the middles of the grid."""
    mid6 = ((ref.E4M3[1:] + ref.E4M3[:-1]) * 3).float()
    tops = torch.cat((mid6, torch.nextafter(mid6, torch.zeros(())), torch.nextafter(mid6, torch.full((), 1e9)),
                      (ref.E4M3 * 6).float()))
    tops = tops[:len(tops) // 4 * 4]
    x = torch.zeros((len(tops) // 4, 4, 16))
    x[:, :, 0] = tops.reshape(-1, 4)
    S = ref.E4M3[ref.nvfp4_bytes(x.flatten(1))[0].reshape(-1, 36)[:, :4].long()].float()
    for i, m in enumerate((ref.GRID[1:] + ref.GRID[:-1]).tolist()):
        v = S * (m / 2)
        x[:, :, 1 + 2 * i] = torch.minimum(v, x[:, :, 0])
        x[:, :, 2 + 2 * i] = -torch.minimum(torch.nextafter(v, torch.full((), [0.0, 1e9][i % 2])), x[:, :, 0])
    x = x.flatten(1)
    assert torch.equal(q.quantize(q.NVFP4, x.cuda()).cpu(), ref.nvfp4_bytes(x)[0])


def matrix(q, planes_):
    codes, scales, v = planes_
    return lambda K: q.MXMatrix(codes.cuda(), scales.cuda(), K), v


PRODUCTS = [(1, 1, 1), (1, 32, 32), (1, 300, 100), (2, 17, 33), (3, 64, 256), (4, 1000, 512), (5, 40, 8000), (15, 16, 257),
            (16, 256, 1024), (17, 100, 300), (31, 33, 64), (33, 31, 129), (64, 64, 2048), (65, 129, 513), (100, 260, 700),
            (128, 128, 256), (129, 255, 511), (200, 520, 1111), (256, 256, 512), (257, 300, 768), (300, 257, 1300),
            (513, 700, 320), (700, 1030, 96)]


@pytest.mark.parametrize("TNK", PRODUCTS, ids=str)
@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
def test_product(q, dtype, TNK):
    T, N, K = TNK
    a, b = ref.random_planes(gen(T), T, K), ref.random_planes(gen(N + 1), N, K)
    A, B = q.MXMatrix(a[0].cuda(), a[1].cuda(), K), q.MXMatrix(b[0].cuda(), b[1].cuda(), K)
    out = torch.full((T, N + 3), float("nan"), dtype=dtype, device="cuda")
    y = q.mx_mul_mat(A, B, dtype, out=out[:, :N])
    assert out[:, N:].isnan().all()  # only Y is written
    bound = ref.product_bound(a[2], b[2], K, ref.OUT_ULP[dtype])
    assert ((y.cpu().double() - a[2] @ b[2].T).abs() <= bound).all()
    again = q.mx_mul_mat(A, B, dtype)
    assert torch.equal(again, y)


@pytest.mark.parametrize("TNK", PRODUCTS, ids=str)
def test_every_kernel_of_the_product(q, TNK):
    T, N, K = TNK
    a, b = ref.random_planes(gen(T), T, K), ref.random_planes(gen(N + 1), N, K)
    A, B = q.MXMatrix(a[0].cuda(), a[1].cuda(), K), q.MXMatrix(b[0].cuda(), b[1].cuda(), K)
    want = a[2] @ b[2].T
    for dtype in (torch.float32, torch.bfloat16):
        bound = ref.product_bound(a[2], b[2], K, ref.OUT_ULP[dtype])
        for variant, name in q.MX_VARIANT_NAMES.items():
            print(name, dtype, flush=True)
            try:
                y = q.mx_mul_mat(A, B, dtype, variant=variant)
            except q.RetroError as e:
                assert e.code == q.E_VARIANT and variant != q.mx_mul_mat_choice(K, N, T, dtype)
                continue
            assert ((y.cpu().double() - want).abs() <= bound).all(), name


@pytest.mark.parametrize("TNK", PRODUCTS, ids=str)
def test_linear_is_the_product_of_the_quantized_rows(q, TNK):
    T, N, K = TNK
    for dtype in FLOATS:
        x = values(T, K, dtype, seed=T + K)
        b = ref.random_planes(gen(N + 1), N, K)
        B = q.MXMatrix(b[0].cuda(), b[1].cuda(), K)
        wide = torch.full((T, K + 5), float("nan"), dtype=dtype, device="cuda")
        wide[:, :K] = x.cuda()
        y = q.mx_linear(wide[:, :K], B)
        A = ref.quantized(x)
        bound = ref.product_bound(A, b[2], K, ref.OUT_ULP[dtype])
        assert y.dtype == dtype and ((y.cpu().double() - A @ b[2].T).abs() <= bound).all(), dtype


@pytest.mark.parametrize("T,N,K", [(1, 200, 300), (16, 96, 600), (70, 130, 300), (300, 270, 520)])
def test_a_block_that_is_not_a_number_spoils_its_row_alone(q, T, N, K):
    x = values(T, K, torch.float32, seed=5)
    x[T // 2, K // 2] = float("nan")
    b = ref.random_planes(gen(6), N, K)
    codes, scales = b[0].cuda(), b[1].cuda()
    bad_row = N // 3
    scales[0, bad_row, 1] = 255
    y = q.mx_linear(x.cuda(), q.MXMatrix(codes, scales, K)).cpu()
    bad = torch.zeros((T, N), dtype=torch.bool)
    bad[T // 2] = True
    bad[:, bad_row] = True
    assert torch.equal(y.isnan(), bad)
    x[T // 2, K // 2] = 0
    A = ref.quantized(x)
    keep = ~bad
    bound = ref.product_bound(A, b[2], K, 2.0 ** -24)
    assert ((y.double() - A @ b[2].T).abs() <= bound)[keep].all()


def test_scales_of_opposite_ends_cancel(q):
    """2^-120 against 2^120: the scales' sum counts, not either alone."""
    T, N, K = 40, 50, 400
    a, b = ref.random_planes(gen(1), T, K, 5, 9), ref.random_planes(gen(2), N, K, 245, 249)
    y = q.mx_mul_mat(q.MXMatrix(a[0].cuda(), a[1].cuda(), K), q.MXMatrix(b[0].cuda(), b[1].cuda(), K))
    assert ((y.cpu().double() - a[2] @ b[2].T).abs() <= ref.product_bound(a[2], b[2], K, 2.0 ** -24)).all()


def test_empty_sizes(q):
    x = torch.zeros((0, 64), device="cuda")
    w = q.mx_quantize(torch.ones((5, 64), device="cuda"))
    assert q.mx_linear(x, w).shape == (0, 5)
    assert q.mx_quantize(x).shape == (0, 64) and q.mx_quantize(x, axis=0).shape == (64, 0)
    none = q.mx_quantize(torch.zeros((5, 0), device="cuda"))
    y = q.mx_mul_mat(q.mx_quantize(torch.zeros((3, 0), device="cuda")), none)
    assert y.shape == (3, 5) and not y.any()  # the empty sum
    assert not q.mx_linear(torch.zeros((3, 0), device="cuda"), none).any()
    dx, dw = q.mx_linear_backward(torch.zeros((0, 5), device="cuda"), x, q.mx_quantize(torch.ones((5, 64), device="cuda"), axis=0))
    assert dx.shape == (0, 64) and dw.shape == (5, 64) and not dw.any()
    assert q.quantize(q.MXFP4, x).shape == (0, 34)


@pytest.mark.parametrize("T,N,K", [(1, 40, 70), (16, 128, 96), (77, 130, 300), (300, 257, 512)])
@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
def test_gradients_are_the_formulas(q, dtype, T, N, K):
    x, dy, w = values(T, K, dtype, 1), values(T, N, dtype, 2, 0.25), values(N, K, torch.float32, 3, 0.05)
    wt = q.mx_quantize(w.cuda(), axis=0)
    dx, dw = q.mx_linear_backward(dy.cuda(), x.cuda(), wt)
    a, b = ref.quantized(dy), ref.quantized(w.T)
    assert dx.dtype == dtype
    assert ((dx.cpu().double() - a @ b.T).abs() <= ref.product_bound(a, b, N, ref.OUT_ULP[dtype])).all()
    a, b = ref.quantized(dy.T), ref.quantized(x.T)
    assert dw.dtype == torch.float32
    assert ((dw.cpu().double() - a @ b.T).abs() <= ref.product_bound(a, b, T, 2.0 ** -24)).all()


def test_gradients_are_the_differences(q):
    """On tensors that 4 bits hold exactly (each block has a 4 or a 6, so its
    scale is 1) the layer is bilinear: central differences of
    sum(dy * (x w^T)) are the gradients, up to the F32 sums."""
    T, N, K = 64, 96, 128
    g = gen(9)

    def on_grid(rows, cols):
        v = ref.e2m1_values(torch.randint(0, 16, (rows, cols), generator=g)).float()
        v[::32, :] = 4.0  # a 4 in every block of a column ...
        v[:, ::32] = 4.0  # ... and of a row
        return v

    x, w, dy = on_grid(T, K), on_grid(N, K), on_grid(T, N)
    dx, dw = q.mx_linear_backward(dy.cuda(), x.cuda(), q.mx_quantize(w.cuda(), axis=0))

    def loss(x, w):
        y = q.mx_linear(x.cuda(), q.mx_quantize(w.cuda()))
        return (y.cpu().double() * dy.double()).sum()

    # steps between neighbours of the grid: the perturbed tensors are exact too
    for t, k in [(1, 1), (17, 40), (63, 127)]:
        up, down = x.clone(), x.clone()
        up[t, k], down[t, k] = 2.0, 1.0
        assert float(loss(up, w) - loss(down, w)) == pytest.approx(float(dx[t, k]), rel=1e-6, abs=1e-3)
    for n, k in [(1, 1), (50, 40), (95, 127)]:
        up, down = w.clone(), w.clone()
        up[n, k], down[n, k] = 2.0, 1.0
        assert float(loss(x, up) - loss(x, down)) == pytest.approx(float(dw[n, k]), rel=1e-6, abs=1e-3)


def test_a_stream_of_its_own(q):
    """Everything a call allocates belongs to the stream it runs on."""
    x, w = values(300, 520, torch.bfloat16, 1).cuda(), values(200, 520, torch.float32, 2).cuda()
    want = q.mx_linear(x, q.mx_quantize(w))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [q.mx_linear(x, q.mx_quantize(w, stream=side), stream=side) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_a_captured_step_replays_like_eager_calls(q):
    T, N, K = 130, 96, 300
    w = values(N, K, torch.float32, 4).cuda()
    wr, wt = q.mx_quantize(w), q.mx_quantize(w, axis=0)
    x, dy, one = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((T, K), (T, N), (1, K)))

    def step():
        return (q.mx_linear(x, wr), *q.mx_linear_backward(dy, x, wt), q.mx_linear(one, wr))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        x.copy_(values(T, K, torch.bfloat16, 20 + i))
        dy.copy_(values(T, N, torch.bfloat16, 30 + i))
        one.copy_(values(1, K, torch.bfloat16, 40 + i))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), i


def test_offsets_past_32_bits(q):
    """x of 5.4 GB, its planes of more than 2^31 bytes of offsets, and a Y past
    4 GB: the last rows are right."""
    rows, K = 82000, 32768
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    tail = values(40, K, torch.bfloat16, 8)
    x[-40:] = tail.cuda()
    r, c = q.mx_quantize_both(x)
    last = q.MXMatrix(r.codes[-40:].contiguous(), r.scales[:, -40:].contiguous(), K)
    check_planes(last, *ref.mx_encode(tail), K, "rows")
    cols = q.mx_dequantize(q.MXMatrix(c.codes[-300:].contiguous(), c.scales[:, -300:].contiguous(), rows))
    want = ref.quantized(x[-96 - rows % 32:, -300:].float().cpu().T)  # whole blocks up to the ragged end
    assert torch.equal(cols[:, -want.shape[1]:].cpu().double(), want)
    del x, c, cols
    full = q.mx_dequantize(r, torch.bfloat16)
    assert torch.equal(full[-40:].cpu().double(), ref.quantized(tail))
    del full, r
    T, N, K = 70000, 40000, 64
    a, b = ref.random_planes(gen(1), 64, K), ref.random_planes(gen(2), 64, K)
    A = q.MXMatrix(a[0].cuda().repeat(T // 64 + 1, 1)[:T].contiguous(),
                   a[1].cuda().repeat(1, T // 64 + 1, 1)[:, :T].contiguous(), K)
    B = q.MXMatrix(b[0].cuda().repeat(N // 64, 1), b[1].cuda().repeat(1, N // 64, 1), K)
    y = q.mx_mul_mat(A, B, torch.bfloat16)
    at = torch.arange(T - 64, T)
    want = a[2][at % 64] @ b[2].T
    bound = ref.product_bound(a[2], b[2], K, 2.0 ** -8)[at % 64]
    assert ((y[-64:, -64:].cpu().double() - want).abs() <= bound).all()
    assert torch.equal(y[:64, :64], y[64 * 1000:64 * 1001, 64 * 600:64 * 601])


def test_a_matrix_follows_its_arrays(q):
    """Planes that get other storage: the products are those of the new bytes,
    and planes that went to the host are refused."""
    T, N, K = 20, 50, 300
    x = values(T, K, torch.bfloat16, 1).cuda()
    old, new = (q.mx_quantize(values(N, K, torch.float32, s).cuda()) for s in (2, 3))
    codes, scales = old.codes.clone(), old.scales.clone()
    m = q.MXMatrix(codes, scales, K)
    assert torch.equal(q.mx_linear(x, m), q.mx_linear(x, old))
    codes.data, scales.data = new.codes.clone(), new.scales.clone()
    assert torch.equal(q.mx_linear(x, m), q.mx_linear(x, new))
    codes.data = codes.data.cpu()
    with pytest.raises(ValueError):
        q.mx_linear(x, m)


def room(gigabytes):
    """Skips where other tenants of the card leave less."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes * 1e9:
        pytest.skip(f"needs {gigabytes} GB of device memory")


def test_more_rows_of_b_than_one_launch_takes(q):
    """2^27 + 37 rows of B are 2^23 + 3 workgroups of 512 threads: the linear
    call's own kernel and the skinny product take them in several launches."""
    room(40)
    N, K = (1 << 27) + 37, 40
    b = ref.random_planes(gen(2), 96, K)
    codes = torch.zeros((N, 128), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((1, N, 8), dtype=torch.uint8, device="cuda")
    starts = [0, (1 << 26) - 48, N - 96]  # the ends of the launches among them
    for at in starts:
        codes[at:at + 96] = b[0].cuda()
        scales[:, at:at + 96] = b[1].cuda()
    B = q.MXMatrix(codes, scales, K)
    x = values(2, K, torch.bfloat16, 3)
    A = ref.quantized(x)
    want, bound = A @ b[2].T, ref.product_bound(A, b[2], K, ref.OUT_ULP[torch.bfloat16])
    for y in (q.mx_linear(x.cuda(), B), q.mx_mul_mat(q.mx_quantize(x.cuda()), B, torch.bfloat16,
                                                      variant=q.mx.MX_VARIANT_SKINNY)):
        for at in starts:
            assert ((y[:, at:at + 96].cpu().double() - want).abs() <= bound).all(), at
        assert not y[:, 200:1 << 20].any()  # the zero rows between


def test_more_tiles_than_one_launch_takes(q):
    """2^26 + 2^13 tiles of a wave each in the simple kernel, Y of 137 GB."""
    room(150)
    T, N, K = (1 << 18) + 32, 1 << 18, 40
    a, b = ref.random_planes(gen(1), 96, K), ref.random_planes(gen(2), 96, K)

    def matrix(planes, rows):
        codes = torch.zeros((rows, 128), dtype=torch.uint8, device="cuda")
        scales = torch.zeros((1, rows, 8), dtype=torch.uint8, device="cuda")
        codes[:96], codes[-96:] = planes[0].cuda(), planes[0].cuda()
        scales[:, :96], scales[:, -96:] = planes[1].cuda(), planes[1].cuda()
        return q.MXMatrix(codes, scales, K)

    y = q.mx_mul_mat(matrix(a, T), matrix(b, N), torch.bfloat16, variant=q.mx.MX_VARIANT_SIMPLE)
    want, bound = a[2] @ b[2].T, ref.product_bound(a[2], b[2], K, ref.OUT_ULP[torch.bfloat16])
    for t in (0, T - 96):
        for n in (0, N - 96):
            assert ((y[t:t + 96, n:n + 96].cpu().double() - want).abs() <= bound).all(), (t, n)
    assert not y[T // 2:T // 2 + 64].any()
    del y
    torch.cuda.empty_cache()


def test_more_columns_than_one_launch_takes(q):
    """The columns of a 2 x (2^30 + 300) tensor: 2^23 + 3 workgroups of 512
    threads, codes of 137 GB."""
    room(165)
    cols = (1 << 30) + 300
    x = torch.zeros((2, cols), dtype=torch.bfloat16, device="cuda")
    tail = values(2, 600, torch.bfloat16, 5)  # both sides of a launches' border
    x[:, -600:] = tail.cuda()
    x[:, :600] = tail.cuda()
    m = q.mx_quantize(x, axis=0)
    for at in (0, cols - 600):
        part = q.MXMatrix(m.codes[at:at + 600].contiguous(), m.scales[:, at:at + 600].contiguous(), 2)
        check_planes(part, *ref.mx_encode(tail.T), 2, at)
    assert not m.codes[1 << 20:1 << 21].any()
    del x, m
    torch.cuda.empty_cache()


@pytest.mark.parametrize("TNK", PRODUCTS, ids=str)
def test_which_kernels_take_a_product(q, TNK):
    """Every tile and the simple kernel take all of these, the skinny one up to 32 rows."""
    T, N, K = TNK
    a, b = ref.random_planes(gen(T), T, K), ref.random_planes(gen(N + 1), N, K)
    A, B = q.MXMatrix(a[0].cuda(), a[1].cuda(), K), q.MXMatrix(b[0].cuda(), b[1].cuda(), K)
    for variant, name in q.MX_VARIANT_NAMES.items():
        if name == "skinny" and T > 32:
            with pytest.raises(q.RetroError) as refused:
                q.mx_mul_mat(A, B, variant=variant)
            assert refused.value.code == q.E_VARIANT
        else:
            assert q.mx_mul_mat(A, B, variant=variant).shape == (T, N), name


# Several tile rows and columns of every size, with remainders; 12, 9 and 2 steps
# of K, whole and ragged; no row like another.
MANY_TILES = [(1100, 1300, 2900), (700, 2100, 2304), (1537, 450, 300)]
TILED = ["simple", "tile_256x256", "tile_256x192", "tile_128x128", "tile_64x128", "tile_64x64", "tile_64x64_k4",
         "tile_32x64_k4"]


@pytest.mark.parametrize("kernel", TILED)
@pytest.mark.parametrize("TNK", MANY_TILES, ids=str)
def test_products_of_many_tiles(q, TNK, kernel):
    T, N, K = TNK
    a, b = ref.random_planes(gen(T), T, K), ref.random_planes(gen(N + 1), N, K)
    A, B = q.MXMatrix(a[0].cuda(), a[1].cuda(), K), q.MXMatrix(b[0].cuda(), b[1].cuda(), K)
    want, size = a[2] @ b[2].T, a[2].abs() @ b[2].abs().T
    variant = next(v for v, name in q.MX_VARIANT_NAMES.items() if name == kernel)
    for dtype in FLOATS:
        out = torch.full((T, N + 5), float("nan"), dtype=dtype, device="cuda")
        y = q.mx_mul_mat(A, B, dtype, out=out[:, :N], variant=variant)
        assert out[:, N:].isnan().all()
        bound = -(-K // 64) * 2.0 ** -22 * size + ref.OUT_ULP[dtype] * want.abs() + 2.0 ** -149
        assert ((y.cpu().double() - want).abs() <= bound).all(), dtype


@pytest.mark.parametrize("T,N,K", [(1, 1500, 2900), (16, 700, 4100), (17, 1100, 2304), (32, 533, 5000)])
def test_skinny_products_of_many_steps(q, T, N, K):
    a, b = ref.random_planes(gen(T), T, K), ref.random_planes(gen(N + 1), N, K)
    A, B = q.MXMatrix(a[0].cuda(), a[1].cuda(), K), q.MXMatrix(b[0].cuda(), b[1].cuda(), K)
    for dtype in FLOATS:
        y = q.mx_mul_mat(A, B, dtype, variant=q.mx.MX_VARIANT_SKINNY)
        bound = ref.product_bound(a[2], b[2], K, ref.OUT_ULP[dtype])
        assert ((y.cpu().double() - a[2] @ b[2].T).abs() <= bound).all(), dtype


@pytest.mark.parametrize("kernel", TILED + ["skinny"])
def test_sums_keep_what_f32_holds(q, kernel):
    """1 + 2^-j from two blocks is exact up to F32's last place, whichever comes
    first and whether or not one instruction takes both; beyond it the result is
    one of the two neighbours."""
    K, last = 512, list(range(16, 28))
    variant = next(v for v, name in q.MX_VARIANT_NAMES.items() if name == kernel)

    def matrix(rows):  # each row's list of (block, scale byte): the value 1 times the scale at its first element
        codes, scales = torch.zeros((len(rows), 256), dtype=torch.uint8), torch.full((2, len(rows), 8), 127,
                                                                                   dtype=torch.uint8)
        for r, row in enumerate(rows):
            for block, e in row:
                codes[r, block * 16] = 2
                scales[block // 8, r, block % 8] = e
        return q.MXMatrix(codes.cuda(), scales.cuda(), K)

    for one, small in [(0, 1), (1, 0), (0, 4), (4, 0), (0, 2), (0, 8), (8, 0), (3, 15), (15, 3)]:
        A = matrix([[(one, 127), (small, 127 - j)] for j in last])
        y = q.mx_mul_mat(A, matrix([[(one, 127), (small, 127)]]), variant=variant)[:, 0].cpu().double()
        for j, v in zip(last, y.tolist()):
            assert v == 1 + 2.0 ** -j if j < 24 else v in (1.0, 1 + 2.0 ** -23), (one, small, j)


def test_results_require_no_gradient(q):
    """The calls are outside autograd, whatever their operands: gradients come from mx_linear_backward."""
    x = values(4, 64, torch.float32, 1).cuda().requires_grad_()
    w = values(8, 64, torch.float32, 2).cuda().requires_grad_()
    wr, wt = q.mx_quantize_both(w)
    dx, dw = q.mx_linear_backward(torch.ones((4, 8), device="cuda"), x, wt)
    results = [q.mx_linear(x, wr), dx, dw, q.mx_dequantize(wr),
               q.mx_moe(x, w, q.mx_quantize(torch.ones((8 * 2 * 32, 64), device="cuda")),
                        q.mx_quantize(torch.ones((8 * 64, 32), device="cuda")), 2)]
    assert not any(t.requires_grad for t in results)
    with pytest.raises(RuntimeError):
        results[0].sum().backward()
