"""The operators over a vocabulary on cuda:0 against their definition in 64 bits
(vocab_reference), within bounds that count their roundings."""

import numpy as np
import pytest
import torch

import oracle
import vocab_reference as ref
import workloads as wl

pytestmark = pytest.mark.gpu

FLOATS = [torch.float32, torch.float16, torch.bfloat16]
NAME = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
TYPE = {torch.float32: wl.F32, torch.float16: wl.F16, torch.bfloat16: wl.BF16}
PACKED = [t for t in wl.TYPE_NAMES if t not in (wl.F32, wl.F16, wl.BF16)]


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    import quantized_weight_backward_amd as q

    return q


def gen(seed):
    return torch.Generator().manual_seed(seed)


def packed(wtype, N, K, seed):
    """(bytes on the device, values in 64 bits)"""
    W = wl.make_weight(wtype, N, K, np.random.Generator(np.random.PCG64(seed)))
    return torch.from_numpy(W).cuda(), torch.from_numpy(oracle.dequantize(wtype, W, K)).reshape(N, K).double()


def tokens(T, N, seed, none=0.2, dtype=torch.int64):
    """Ids, some of them none: negative, N and beyond."""
    g = gen(seed)
    t = torch.randint(0, max(N, 1), (T,), generator=g)
    bad = torch.tensor([-1, N, -7, N + 5])[torch.randint(0, 4, (T,), generator=g)]
    return torch.where(torch.rand(T, generator=g) < none, bad, t).to(dtype)


def head(dtype, N, K, seed):
    return (torch.randn((N, K), generator=gen(seed)) * 0.3).to(dtype)


def close(got, want, bound, where=""):
    got = got.cpu().double()
    off = (got - want).abs()
    assert torch.isfinite(got).all(), where
    assert (off <= bound).all(), (where, float((off / bound.clamp(min=1e-300)).max()))


# ---------------------------------------------------------------- embedding

@pytest.mark.parametrize("out", FLOATS, ids=NAME.get)
@pytest.mark.parametrize("wtype", list(wl.TYPE_NAMES), ids=wl.TYPE_NAMES.get)
def test_embedding_of_every_type(q, wtype, out):
    N, K = 37, 512
    W, values = packed(wtype, N, K, seed=3)
    for T, scale, ids in ((1, 1.0, torch.int64), (130, 22.5, torch.int32)):
        t = tokens(T, N, seed=T, dtype=ids)
        known = (t >= 0) & (t < N)
        want = torch.where(known[:, None], values.float()[torch.where(known, t, 0).long()] * scale, 0.0).to(out)
        got = q.embedding(wtype, W, t.cuda(), K, scale=scale, dtype=out)
        assert got.dtype == out and torch.equal(got.cpu(), want)


@pytest.mark.parametrize("K", [1, 3, 7, 8, 9, 100, 1021, 2056])
@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
def test_embedding_of_odd_rows(q, dtype, K):
    N, T = 19, 67
    w, t = head(dtype, N, K, seed=K), tokens(T, N, seed=K)
    known = (t >= 0) & (t < N)
    want = torch.where(known[:, None], w.float()[torch.where(known, t, 0)] * 0.5, 0.0).to(dtype)
    assert torch.equal(q.embedding(TYPE[dtype], w.cuda(), t.cuda(), K, scale=0.5, dtype=dtype).cpu(), want)
    # rows of wider tensors
    wide = torch.full((N, K + 5), float("nan"), dtype=dtype)
    wide[:, :K] = w
    out = torch.full((T, K + 3), 7.0, dtype=dtype).cuda()
    q.embedding(TYPE[dtype], wide.cuda()[:, :K], t.cuda(), K, scale=0.5, dtype=dtype, out=out[:, :K])
    assert torch.equal(out[:, :K].cpu(), want) and (out[:, K:] == 7.0).all()


def test_embedding_of_strided_blocks(q):
    N, K = 21, 256
    for wtype in (wl.Q8_0, wl.Q6_K, wl.MXFP4, wl.NVFP4):
        W, values = packed(wtype, N, K, seed=8)
        wide = torch.full((N, W.shape[1] + 48), 255, dtype=torch.uint8, device="cuda")
        wide[:, :W.shape[1]] = W
        wide = wide[:, :W.shape[1]]
        t = tokens(40, N, seed=1)
        known = (t >= 0) & (t < N)
        want = torch.where(known[:, None], values.float()[torch.where(known, t, 0)], 0.0)
        assert torch.equal(q.embedding(wtype, wide, t.cuda(), K).cpu(), want)


def test_embedding_of_a_table_past_32_bits(q):
    """Rows whose offset passes 2^32 bytes."""
    N, K = 140000, 16384
    W = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 131071, 131072, 139999], device="cuda")
    W[rows] = (torch.arange(4, device="cuda", dtype=torch.float32) + 1).bfloat16()[:, None].expand(4, K)
    y = q.embedding(wl.BF16, W, rows, K)
    assert torch.equal(y[:, ::97].cpu(), torch.arange(1.0, 5.0)[:, None].expand(4, len(range(0, K, 97))))


# ---------------------------------------------------------------- its gradient

def dense_gradient(ids, dy, N, scale):
    """(dW, sum of magnitudes, tokens a row) in 64 bits."""
    known = (ids >= 0) & (ids < N)
    t = torch.nonzero(known)[:, 0]
    at = ids[t].long()
    dw = torch.zeros((N, dy.shape[1]), dtype=torch.float64)
    size, count = dw.clone(), torch.zeros(N, dtype=torch.float64)
    dw.index_put_((at,), dy[t].double() * scale, accumulate=True)
    size.index_put_((at,), dy[t].double().abs() * abs(scale), accumulate=True)
    count.index_put_((at,), torch.ones(len(t), dtype=torch.float64), accumulate=True)
    return dw, size, count


def gradient_bound(dw, size, count, dtype, old=None):
    # each addition of a row's F32 sum, and the scale's product, rounds what is at most the sum of magnitudes
    b = (count[:, None] + 2) * 2.0 ** -24 * size
    if old is not None:
        b += 2.0 ** -24 * (old.abs() + size)
    return b + ref.half_step(dtype) * (dw.abs() + b) + torch.finfo(dtype).smallest_normal * ref.half_step(dtype)


@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (2, 5, 3), (63, 7, 8), (64, 1, 40), (65, 1, 9), (129, 3, 100),
                                   (300, 1000, 17), (1000, 511, 64), (1025, 513, 12), (5000, 20, 8), (8192, 40000, 8),
                                   (8193, 70000, 8), (16384, 5000, 12), (16385, 90, 5), (20000, 300, 33), (30011, 2, 16), (40000, 300000, 4)], ids=str)
@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
def test_embedding_backward(q, dtype, T, N, K):
    ids = tokens(T, N, seed=T, dtype=torch.int32 if T % 2 else torch.int64)
    dy = torch.randn((T, K), generator=gen(T + 1)).to(dtype)
    dw, size, count = dense_gradient(ids, dy, N, 0.75)
    got = q.embedding_backward(ids.cuda(), dy.cuda(), N, scale=0.75)
    assert got.dtype == torch.float32
    close(got, dw, gradient_bound(dw, size, count, torch.float32))
    assert not got[count.cuda() == 0].any()
    again = q.embedding_backward(ids.cuda(), dy.cuda(), N, scale=0.75)
    assert torch.equal(got, again)
    # added to a table of the gradient's own type: rows of no token are not touched
    old = torch.randn((N, K), generator=gen(5)).to(dtype)
    out = old.cuda()
    q.embedding_backward(ids.cuda(), dy.cuda(), N, scale=0.75, out=out, accumulate=True)
    close(out, dw + old.double(), gradient_bound(dw + old.double(), size, count, dtype, old.double()))
    assert torch.equal(out[count.cuda() == 0].cpu(), old[count == 0])


def test_embedding_backward_of_one_frequent_id(q):
    """All tokens one id, and tokens of two ids in turn: every run's parts."""
    for T in (64, 128, 8192, 16500):
        for N, ids in ((9, torch.full((T,), 4)), (9, torch.arange(T) % 2 + 3), (2, torch.arange(T) * 2 // T)):
            dy = torch.randn((T, 24), generator=gen(T)).bfloat16()
            dw, size, count = dense_gradient(ids, dy, N, 1.0)
            got = q.embedding_backward(ids.cuda(), dy.cuda(), N)
            close(got, dw, gradient_bound(dw, size, count, torch.float32))


def test_embedding_backward_of_no_tokens_and_of_none(q):
    for ids in (torch.empty(0, dtype=torch.int64), torch.full((300,), -1), torch.full((9000,), 12)):
        dy = torch.full((len(ids), 20), float("nan"), device="cuda")
        out = torch.full((12, 23), 3.0, device="cuda")
        q.embedding_backward(ids.cuda(), dy, 12, scale=float("inf"), out=out[:, :20])
        assert not out[:, :20].any() and (out[:, 20:] == 3.0).all()


def test_embedding_backward_keeps_padding_out(q):
    """What stands in the gradient of a padding token is not read into any row."""
    ids = torch.tensor([3, -1, 3, 8, 1])
    dy = torch.ones((5, 16))
    dy[1] = float("nan")
    dy[3] = float("inf")
    got = q.embedding_backward(ids.cuda(), dy.cuda(), 8).cpu()
    want = torch.zeros((8, 16))
    want[3], want[1] = 2, 1
    assert torch.equal(got, want)


def test_embedding_backward_strides(q):
    T, N, K = 200, 50, 37
    ids = tokens(T, N, seed=2)
    wide = torch.randn((T, K + 11), generator=gen(9)).half().cuda()
    dy = wide[:, 2:2 + K]
    dw, size, count = dense_gradient(ids, dy.cpu(), N, 1.0)
    out = torch.full((N, K + 4), 5.0, dtype=torch.bfloat16, device="cuda")
    q.embedding_backward(ids.cuda(), dy, N, dtype=torch.bfloat16, out=out[:, 1:1 + K])
    close(out[:, 1:1 + K], dw, gradient_bound(dw, size, count, torch.bfloat16))
    assert (out[:, 0] == 5.0).all() and (out[:, 1 + K:] == 5.0).all()


# ---------------------------------------------------------------- cross entropy

def part_error(xtype, wtype, result):
    if result == torch.float32:
        return 2.0 ** -22
    return 2.0 ** -8 if xtype == torch.bfloat16 and wtype == wl.BF16 else 2.0 ** -11


def check_cross_entropy(q, wtype, W, values, x, targets, weight_grad=False, where=""):
    w, xd, t = values, x.double(), targets.long()
    N, T = w.shape[0], x.shape[0]
    d_x, d_t = x.cuda(), targets.cuda()
    loss, lse = q.cross_entropy(wtype, W, d_x, d_t)
    assert loss.dtype == lse.dtype == torch.float32
    want, want_lse, learnt, _ = ref.cross_entropy(w, xd, t)
    bound = ref.loss_error(w, xd, want_lse)
    close(lse, want_lse, bound, where + " lse")
    close(loss, want, bound, where + " loss")
    assert not loss.cpu()[~learnt].any()
    dloss = torch.rand(T, generator=gen(T)) / T - 0.2 / T
    dx, dw = q.cross_entropy_backward(wtype, W, d_x, d_t, lse, dloss.cuda(), weight_grad=weight_grad)
    wdtype = {v: k for k, v in TYPE.items()}.get(wtype, torch.float32)
    err = max(part_error(x.dtype, wtype, x.dtype), part_error(x.dtype, wtype, wdtype) if weight_grad else 0)
    # a BF16 x takes the head in 11 bits, unless its gradient is F32
    narrow = x.dtype == torch.bfloat16 and not (weight_grad and wtype == wl.F32)
    (wx, bx), (ww, bw) = ref.gradients(w, xd, t, dloss, err, x.dtype, wdtype, 2.0 ** -11 if narrow else 0.0)
    assert dx.dtype == x.dtype
    close(dx, wx, bx, where + " dx")
    assert not dx.cpu()[~learnt].any()
    if weight_grad:
        assert dw.dtype == wdtype
        close(dw, ww, bw, where + " dw")
    else:
        assert dw is None
    # the same bits again
    loss2, lse2 = q.cross_entropy(wtype, W, d_x, d_t)
    dx2, dw2 = q.cross_entropy_backward(wtype, W, d_x, d_t, lse, dloss.cuda(), weight_grad=weight_grad)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2) and torch.equal(dx, dx2)
    assert dw is None or torch.equal(dw, dw2)


SHAPES = [(1, 1, 1), (1, 2, 64), (2, 33, 3), (5, 255, 31), (31, 256, 64), (32, 257, 65), (33, 100, 128), (64, 1000, 192),
          (65, 129, 72), (128, 513, 256), (129, 1000, 100), (300, 2100, 320), (257, 4100, 64)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", FLOATS, ids=NAME.get)
def test_cross_entropy_of_one_float_type(q, dtype, shape):
    T, N, K = shape
    w = head(dtype, N, K, seed=T)
    x = torch.randn((T, K), generator=gen(N)).to(dtype)
    check_cross_entropy(q, TYPE[dtype], w.cuda(), w.double(), x, tokens(T, N, seed=K), weight_grad=True)


@pytest.mark.parametrize("shape", [(3, 70, 33), (70, 600, 128), (200, 300, 64)], ids=str)
@pytest.mark.parametrize("xtype,wdtype", [(a, b) for a in FLOATS for b in FLOATS if a != b], ids=NAME.get)
def test_cross_entropy_of_two_float_types(q, xtype, wdtype, shape):
    T, N, K = shape
    w = head(wdtype, N, K, seed=T)
    x = torch.randn((T, K), generator=gen(N)).to(xtype)
    check_cross_entropy(q, TYPE[wdtype], w.cuda(), w.double(), x, tokens(T, N, seed=K, dtype=torch.int32),
                        weight_grad=True)


@pytest.mark.parametrize("T", [1, 17, 64, 65, 140])
@pytest.mark.parametrize("wtype", PACKED, ids=wl.TYPE_NAMES.get)
def test_cross_entropy_of_packed_heads(q, wtype, T):
    N, K = 700, 256
    W, values = packed(wtype, N, K, seed=T)
    for xtype in (torch.bfloat16, torch.float32):
        # logits of a few units whatever the type's values are
        x = (torch.randn((T, K), generator=gen(7)) / (float(values.std()) * K ** 0.5)).to(xtype)
        check_cross_entropy(q, wtype, W, values, x, tokens(T, N, seed=T), where=NAME[xtype])


@pytest.mark.parametrize("wtype", [wl.Q4_0, wl.Q4_1, wl.Q5_0, wl.Q5_1, wl.Q8_0, wl.MXFP4], ids=wl.TYPE_NAMES.get)
def test_cross_entropy_of_few_tokens_and_odd_rows(q, wtype):
    """Rows that end inside a chunk of 256, heads that end inside a wave's 32 rows."""
    for N, K, T in ((1, 32, 1), (31, 224, 16), (33, 256, 17), (127, 288, 33), (129, 480, 64), (257, 544, 32), (300, 1056, 5)):
        W, values = packed(wtype, N, K, seed=K)
        for xtype in (torch.bfloat16, torch.float32):
            x = (torch.randn((T, K), generator=gen(7)) / (float(values.std()) * K ** 0.5)).to(xtype)
            check_cross_entropy(q, wtype, W, values, x, tokens(T, N, seed=T), where=f"{N} {K} {T} {NAME[xtype]}")


@pytest.mark.parametrize("wtype", [wl.Q4_K, wl.Q5_K, wl.Q6_K], ids=wl.TYPE_NAMES.get)
def test_cross_entropy_of_few_tokens_and_several_blocks(q, wtype):
    for N, K, T in ((1, 256, 1), (33, 512, 16), (127, 768, 33), (300, 1280, 64)):
        W, values = packed(wtype, N, K, seed=K)
        for xtype in (torch.bfloat16, torch.float32):
            x = (torch.randn((T, K), generator=gen(7)) / (float(values.std()) * K ** 0.5)).to(xtype)
            check_cross_entropy(q, wtype, W, values, x, tokens(T, N, seed=T), where=f"{N} {K} {T} {NAME[xtype]}")


def test_cross_entropy_of_strided_operands(q):
    T, N, K = 90, 500, 256
    for dtype, pad in ((torch.bfloat16, 8), (torch.bfloat16, 3), (torch.float32, 5)):
        w, x = head(dtype, N, K, seed=1), torch.randn((T, K), generator=gen(2)).to(dtype)
        ww, xx = torch.full((N, K + pad), float("nan"), dtype=dtype), torch.full((T, K + pad), float("nan"), dtype=dtype)
        ww[:, :K], xx[:, :K] = w, x
        t = tokens(T, N, seed=3).cuda()
        g = torch.full((T,), 1 / T).cuda()
        got = q.cross_entropy(TYPE[dtype], ww.cuda()[:, :K], xx.cuda()[:, :K], t)
        want = q.cross_entropy(TYPE[dtype], w.cuda(), x.cuda(), t)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        dx_out = torch.full((T, K + 3), 9.0, dtype=dtype, device="cuda")
        dw_out = torch.full((N, K + 1), 9.0, dtype=dtype, device="cuda")
        q.cross_entropy_backward(TYPE[dtype], ww.cuda()[:, :K], xx.cuda()[:, :K], t, want[1], g, weight_grad=True,
                                 dx_out=dx_out[:, :K], dw_out=dw_out[:, :K])
        dx, dw = q.cross_entropy_backward(TYPE[dtype], w.cuda(), x.cuda(), t, want[1], g, weight_grad=True)
        assert torch.equal(dx_out[:, :K], dx) and torch.equal(dw_out[:, :K], dw)
        assert (dx_out[:, K:] == 9.0).all() and (dw_out[:, K:] == 9.0).all()
    # packed rows apart
    W, values = packed(wl.Q8_0, N, K, seed=4)
    wide = torch.full((N, W.shape[1] + 6), 255, dtype=torch.uint8, device="cuda")
    wide[:, :W.shape[1]] = W
    wide = wide[:, :W.shape[1]]
    for T in (5, 90):
        x = torch.randn((T, K), generator=gen(T)).bfloat16()
        check_cross_entropy(q, wl.Q8_0, wide, values, x, tokens(T, N, seed=T))


def test_cross_entropy_in_several_pieces_of_the_head(q):
    """More rows than one piece, and a last piece of odd size."""
    for dtype, T, N, K in ((torch.float32, 70, 33000, 64), (torch.bfloat16, 70, 33001, 40), (torch.float16, 16500, 4200, 64)):
        w = head(dtype, N, K, seed=T)
        x = torch.randn((T, K), generator=gen(N)).to(dtype)
        t = tokens(T, N, seed=K)
        if T < 1000:
            check_cross_entropy(q, TYPE[dtype], w.cuda(), w.double(), x, t, weight_grad=True)
            continue
        loss, lse = q.cross_entropy(TYPE[dtype], w.cuda(), x.cuda(), t.cuda())
        some = torch.arange(0, T, 331)
        want, want_lse, _, _ = ref.cross_entropy(w.double(), x[some].double(), t[some])
        close(loss[some.cuda()], want, ref.loss_error(w.double(), x[some].double(), want_lse))
        dx, _ = q.cross_entropy_backward(TYPE[dtype], w.cuda(), x.cuda(), t.cuda(), lse, torch.ones(T, device="cuda"),
                                         weight_grad=True)
        (wx, bx), _ = ref.gradients(w.double(), x[some].double(), t[some], torch.ones(len(some)), 2.0 ** -11, dtype, dtype)
        close(dx[some.cuda()], wx, bx)


@pytest.mark.parametrize("wtype,K,T", [(wl.Q8_0, 32, 3), (wl.BF16, 64, 2), (wl.Q3_K, 256, 64), (wl.F32, 64, 1)], ids=str)
def test_losses_of_many_pieces(q, wtype, K, T):
    """512 rows again and again: as many pieces as a head has past 2^24 logits or rows."""
    base, N = 512, (1 << 24) // (64 if T == 64 else 1) + 512
    if wtype in TYPE.values():
        dtype = torch.bfloat16 if wtype == wl.BF16 else torch.float32
        rows = head(dtype, base, K, seed=1).cuda()
        values, W = rows.cpu().double(), rows.repeat(N // base, 1)
    else:
        rows, values = packed(wtype, base, K, seed=1)
        W = rows.view(base, -1).repeat(N // base, 1)
    x = torch.randn((T, K), generator=gen(2)) / (float(values.std()) * K ** 0.5)
    x = x.to(torch.bfloat16 if wtype == wl.BF16 else torch.float32)
    t = torch.tensor([N - 5, 1, (1 << 18) - 1, 1 << 18, N])[torch.arange(T) % 5]
    loss, lse = q.cross_entropy(wtype, W, x.cuda(), t.cuda())
    inside = torch.where(t < N, t % base, -1)
    want, want_lse, learnt, _ = ref.cross_entropy(values, x.double(), inside)
    # every run again has the same sum, so that F32's log2(runs) joins of them are off by a step each
    bound = ref.loss_error(values, x.double(), want_lse) + N / (64 * 256) * 2.0 ** -24
    more = torch.log(torch.tensor(N / base, dtype=torch.float64))
    close(lse, want_lse + more, bound + more * 2.0 ** -22)
    close(loss, torch.where(learnt, want + more, 0.0), bound + more * 2.0 ** -22)


@pytest.mark.parametrize("wtype,K", [(wl.Q8_0, 32), (wl.Q2_K, 256)], ids=str)
def test_gradients_of_few_tokens_in_several_pieces(q, wtype, K):
    N, T = (1 << 18) + 37, 64
    W, values = packed(wtype, 1001, K, seed=5)
    again = torch.arange(N) % 1001
    x = torch.randn((T, K), generator=gen(2)) / (float(values.std()) * K ** 0.5)
    t = tokens(T, N, seed=3)
    t[0], t[1], t[2] = (1 << 18) - 1, 1 << 18, N - 1
    check_cross_entropy(q, wtype, W.view(1001, -1)[again.cuda()], values[again], x, t)


@pytest.mark.parametrize("wtype", [wl.BF16, wl.Q4_K, wl.MXFP4, wl.Q2_K], ids=wl.TYPE_NAMES.get)
def test_cross_entropy_of_long_rows(q, wtype):
    N, K = 90, 20480
    if wtype == wl.BF16:
        w = head(torch.bfloat16, N, K, seed=1)
        W, values = w.cuda(), w.double()
    else:
        W, values = packed(wtype, N, K, seed=1)
    for T in (1, 40, 130):
        x = (torch.randn((T, K), generator=gen(7)) / (float(values.std()) * K ** 0.5)).bfloat16()
        check_cross_entropy(q, wtype, W, values, x, tokens(T, N, seed=T))


def test_cross_entropy_of_rows_of_nothing(q):
    """K = 0: every logit is 0."""
    N, T = 37, 5
    t = torch.tensor([0, 36, 37, -1, 3], device="cuda")
    for wtype in (wl.F32, wl.BF16, wl.Q8_0):
        for xtype in (wl.F32, wl.BF16):
            need = q.lib.retro_cross_entropy_workspace_size(wtype, 0, xtype, 0, N, T)
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            out = torch.full((2, T), 9.0, device="cuda")
            assert q.lib.retro_cross_entropy(wtype, None, 0, xtype, None, 0, 27, t.data_ptr(), out[0].data_ptr(),
                                             out[1].data_ptr(), 0, N, T, ws.data_ptr(), need, None) == 0
            torch.cuda.synchronize()
            want = torch.log(torch.tensor(float(N), dtype=torch.float64))
            close(out[1], want.expand(T), torch.full((T,), 2.0 ** -20))
            close(out[0], torch.tensor([1.0, 1, 0, 0, 1]).double() * want, torch.full((T,), 2.0 ** -20))


def test_cross_entropy_in_whole_rounds_and_a_rest(q):
    """Tiles of 256 x 256 for most of the head, smaller ones for what is left of it."""
    for dtype, T, N, K in ((torch.bfloat16, 300, 33100, 64), (torch.float16, 257, 32769, 33), (torch.float32, 300, 33000, 64)):
        w = head(dtype, N, K, seed=T)
        x = torch.randn((T, K), generator=gen(N)).to(dtype)
        t = tokens(T, N, seed=K)
        t[:9] = torch.tensor([0, 255, 256, 32511, 32512, 32767, 32768, N - 1, N])  # about the borders
        check_cross_entropy(q, TYPE[dtype], w.cuda(), w.double(), x, t, weight_grad=True)


def test_cross_entropy_keeps_tokens_that_are_not_learnt_from_out(q):
    """Their x, lse and dloss may hold anything."""
    T, N, K = 80, 300, 128
    for dtype in FLOATS:
        w, x = head(dtype, N, K, seed=1), torch.randn((T, K), generator=gen(2)).to(dtype)
        t = torch.randint(0, N, (T,), generator=gen(3))
        none = torch.arange(T) % 3 == 0
        t[none] = -100
        clean_x, dirty_x = x.clone(), x.clone()
        clean_x[none], dirty_x[none] = 0, float("nan")
        dirty_x[0] = float("inf")
        g = torch.rand(T, generator=gen(4))
        dirty_g = torch.where(none, float("nan"), g)
        loss, lse = q.cross_entropy(TYPE[dtype], w.cuda(), dirty_x.cuda(), t.cuda())
        assert not loss.cpu()[none].any() and torch.isnan(lse.cpu()[none]).all()
        got = q.cross_entropy_backward(TYPE[dtype], w.cuda(), dirty_x.cuda(), t.cuda(), lse, dirty_g.cuda(), weight_grad=True)
        loss, lse = q.cross_entropy(TYPE[dtype], w.cuda(), clean_x.cuda(), t.cuda())
        want = q.cross_entropy_backward(TYPE[dtype], w.cuda(), clean_x.cuda(), t.cuda(), lse, g.cuda(), weight_grad=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        # all of them: no gradient
        t[:] = N
        dx, dw = q.cross_entropy_backward(TYPE[dtype], w.cuda(), dirty_x.cuda(), t.cuda(), lse, g.cuda(), weight_grad=True)
        assert not dx.any() and not dw.any()


def test_cross_entropy_of_a_token_that_is_not_finite(q):
    """Its own loss and gradient are NaN, others' are not touched."""
    T, N, K = 70, 200, 64
    for dtype in FLOATS:
        w, x = head(dtype, N, K, seed=1).cuda(), torch.randn((T, K), generator=gen(2)).to(dtype).cuda()
        t = torch.randint(0, N, (T,), generator=gen(3)).cuda()
        g = torch.ones(T, device="cuda")
        loss, lse = q.cross_entropy(TYPE[dtype], w, x, t)
        dx, _ = q.cross_entropy_backward(TYPE[dtype], w, x, t, lse, g)
        bad = x.clone()
        bad[7, 3] = float("nan")
        loss2, lse2 = q.cross_entropy(TYPE[dtype], w, bad, t)
        dx2, _ = q.cross_entropy_backward(TYPE[dtype], w, bad, t, lse2, g)
        assert torch.isnan(loss2[7]) and torch.isnan(dx2[7]).all()
        rest = torch.arange(T, device="cuda") != 7
        assert torch.equal(loss[rest], loss2[rest]) and torch.equal(dx[rest], dx2[rest])
    for wtype in (wl.Q4_K, wl.MXFP4, wl.Q3_K):
        W, values = packed(wtype, N, 256, seed=1)
        for T in (9, 70):
            x = (torch.randn((T, 256), generator=gen(2)) / (float(values.std()) * 16)).bfloat16().cuda()
            t, g = torch.randint(0, N, (T,), generator=gen(3)).cuda(), torch.ones(T, device="cuda")
            loss, lse = q.cross_entropy(wtype, W, x, t)
            dx, _ = q.cross_entropy_backward(wtype, W, x, t, lse, g)
            bad = x.clone()
            bad[7, 3] = float("nan")
            loss2, lse2 = q.cross_entropy(wtype, W, bad, t)
            dx2, _ = q.cross_entropy_backward(wtype, W, bad, t, lse2, g)
            assert torch.isnan(loss2[7]) and torch.isnan(dx2[7]).all()
            rest = torch.arange(T, device="cuda") != 7
            assert torch.equal(loss[rest], loss2[rest]) and torch.equal(dx[rest], dx2[rest])


def test_cross_entropy_of_wide_ranges(q):
    """Logits of hundreds, tokens and tables of very different sizes."""
    T, N, K = 80, 300, 128
    for dtype, sx, sw in ((torch.bfloat16, 30.0, 1.0), (torch.float32, 1e-20, 1e18), (torch.float32, 1e15, 1e-14),
                          (torch.float32, 1e-30, 1e-30), (torch.float16, 20.0, 1.0), (torch.float32, 1e-37, 1e37),
                          (torch.float32, 1e37, 1e-37)):
        w = head(dtype, N, K, seed=1) * sw
        x = (torch.randn((T, K), generator=gen(2)) * sx).to(dtype)
        check = dtype, sx, sw
        t = tokens(T, N, seed=5)
        want, want_lse, learnt, _ = ref.cross_entropy(w.double(), x.double(), t)
        loss, lse = q.cross_entropy(TYPE[dtype], w.cuda(), x.cuda(), t.cuda())
        close(loss, want, ref.loss_error(w.double(), x.double(), want_lse), check)
    # rows of x that differ by 2^60 do not disturb one another
    w, x = head(torch.float32, N, K, seed=1), torch.randn((T, K), generator=gen(2))
    x[::2] *= 2.0 ** -60
    t = tokens(T, N, seed=5, none=0)
    check_cross_entropy(q, wl.F32, w.cuda(), w.double(), x, t, weight_grad=True)


def test_cross_entropy_of_a_head_of_the_largest_scales(q):
    """MXFP4 blocks up to scales whose largest code would be infinite."""
    N, K = 200, 256
    W = wl.make_weight(wl.MXFP4, N, K, np.random.Generator(np.random.PCG64(3)))
    W = W.reshape(N, K // 32, 17)
    W[..., 0] = 252
    W[..., 1:] &= 0xBB  # magnitudes up to 1.5
    W[:, ::2, 0] = 253
    W = np.ascontiguousarray(W.reshape(N, -1))
    values = torch.from_numpy(oracle.dequantize(wl.MXFP4, W, K)).reshape(N, K).double()
    assert torch.isfinite(values).all()
    for T in (5, 70):
        x = (torch.randn((T, K), generator=gen(7)) * 2.0 ** -130).float()
        t = tokens(T, N, seed=T)
        want, want_lse, _, _ = ref.cross_entropy(values, x.double(), t)
        loss, lse = q.cross_entropy(wl.MXFP4, torch.from_numpy(W).cuda(), x.cuda(), t.cuda())
        close(lse, want_lse, ref.loss_error(values, x.double(), want_lse) + values.abs().max() * x.double().abs().sum(1) * 2.0 ** -20)


def test_cross_entropy_of_an_empty_head_and_of_no_tokens(q):
    x = torch.randn((4, 64), device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    W = torch.empty((0, 64), device="cuda")
    loss, lse = q.cross_entropy(wl.F32, W, x, t)
    assert not loss.any() and (lse == -float("inf")).all()
    dx, dw = q.cross_entropy_backward(wl.F32, W, x, t, lse, torch.ones(4, device="cuda"), weight_grad=True)
    assert not dx.any() and dw.shape == (0, 64)
    W = torch.randn((10, 64), device="cuda")
    loss, lse = q.cross_entropy(wl.F32, W, x[:0], t[:0])
    assert loss.shape == lse.shape == (0,)
    dx, dw = q.cross_entropy_backward(wl.F32, W, x[:0], t[:0], lse, lse, weight_grad=True)
    assert dx.shape == (0, 64) and dw.shape == (10, 64) and not dw.any()


def test_gradients_against_differences(q):
    """The loss's change along a direction, by the operator itself in F32."""
    T, N, K = 40, 90, 64
    w, x = head(torch.float32, N, K, seed=1).cuda(), torch.randn((T, K), generator=gen(2)).cuda()
    t = tokens(T, N, seed=3).cuda()
    g = torch.rand(T, generator=gen(4)).cuda()
    _, lse = q.cross_entropy(wl.F32, w, x, t)
    dx, dw = q.cross_entropy_backward(wl.F32, w, x, t, lse, g, weight_grad=True)
    h = 2.0 ** -7
    for grad, at in ((dx, x), (dw, w)):
        step = torch.randn(at.shape, generator=gen(6)).cuda()
        step /= step.norm()
        ends = []
        for s in (h, -h):
            moved = at + s * step
            l, _ = q.cross_entropy(wl.F32, w if at is x else moved, moved if at is x else x, t)
            ends.append(float((l.double() * g).sum()))
        slope = (ends[0] - ends[1]) / (2 * h)
        # losses of about 5 are off by some 2^-21 each, T of them over 2 h; the third derivative is below 1
        assert abs(slope - float((grad.double() * step).sum())) <= T * 5 * 2.0 ** -21 / (2 * h) + h * h


# ---------------------------------------------------------------- streams, graphs, together

def test_streams(q):
    """Calls on another stream, one of them beside another with operands of its own."""
    N, K, T = 900, 256, 100
    w = head(torch.bfloat16, N, K, seed=1).cuda()
    x = torch.randn((T, K), generator=gen(2)).bfloat16().cuda()
    t = tokens(T, N, seed=3).cuda()
    g = torch.ones(T, device="cuda")
    want = q.cross_entropy(wl.BF16, w, x, t)
    want_g = q.cross_entropy_backward(wl.BF16, w, x, t, want[1], g, weight_grad=True)
    want_e = q.embedding(wl.BF16, w, t, K)
    want_b = q.embedding_backward(t, x, N)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s in streams:
            l = q.cross_entropy(wl.BF16, w, x, t, stream=s)
            got.append((l, q.cross_entropy_backward(wl.BF16, w, x, t, l[1], g, weight_grad=True, stream=s),
                        q.embedding(wl.BF16, w, t, K, stream=s), q.embedding_backward(t, x, N, stream=s)))
    torch.cuda.synchronize()
    for l, b, e, d in got:
        assert all(torch.equal(a, c) for a, c in zip(l, want)) and all(torch.equal(a, c) for a, c in zip(b, want_g))
        assert torch.equal(e, want_e) and torch.equal(d, want_b)


def step_of(q, wtype, w, ids, targets, g, K, N):
    """One training step over a tied table: ids in, gradients of the table out."""
    x = q.embedding(wtype, w, ids, K, scale=4.0, dtype=torch.bfloat16)
    loss, lse = q.cross_entropy(wtype, w, x, targets)
    dx, dw = q.cross_entropy_backward(wtype, w, x, targets, lse, g, weight_grad=True)
    q.embedding_backward(ids, dx, N, scale=4.0, out=dw, accumulate=True)
    return loss, dx, dw


def test_a_tied_table_in_one_step(q):
    """Embedding, loss and both gradients into one table, against 64 bits."""
    N, K, T = 600, 128, 200
    w = head(torch.bfloat16, N, K, seed=1)
    ids, targets = tokens(T, N, seed=2), tokens(T, N, seed=3)
    g = torch.full((T,), 1 / T)
    loss, dx, dw = step_of(q, wl.BF16, w.cuda(), ids.cuda(), targets.cuda(), g.cuda(), K, N)
    known = (ids >= 0) & (ids < N)
    x = torch.where(known[:, None], w.float()[torch.where(known, ids, 0)] * 4.0, 0.0).bfloat16().double()
    want, want_lse, _, _ = ref.cross_entropy(w.double(), x, targets)
    close(loss, want, ref.loss_error(w.double(), x, want_lse))
    (wx, bx), (ww, bw) = ref.gradients(w.double(), x, targets, g, 2.0 ** -8, torch.bfloat16, torch.bfloat16)
    close(dx, wx, bx)
    more, size, count = dense_gradient(ids, dx.cpu(), N, 4.0)
    close(dw, ww + more, bw + gradient_bound(ww + more, size, count, torch.bfloat16, ww.abs() + bw))


def test_a_captured_step(q):
    """The step recorded once and replayed on new ids, beside eager work."""
    for N, K, T in ((600, 128, 200), (40000, 64, 9000), (3000, 64, 17000)):
        w = head(torch.bfloat16, N, K, seed=1).cuda()
        g = torch.full((T,), 1 / T, device="cuda")
        ids, targets = tokens(T, N, seed=2).cuda(), tokens(T, N, seed=3).cuda()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step_of(q, wl.BF16, w, ids, targets, g, K, N)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step_of(q, wl.BF16, w, ids, targets, g, K, N)
        for seed in (5, 6, 7):
            ids.copy_(tokens(T, N, seed=seed))
            targets.copy_(tokens(T, N, seed=seed + 10))
            w.copy_(head(torch.bfloat16, N, K, seed=seed))
            graph.replay()
            torch.cuda.synchronize()
            want = step_of(q, wl.BF16, w, ids, targets, g, K, N)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


def test_a_captured_loss_through_packed_heads(q):
    N, K = 800, 256
    W, _ = packed(wl.Q4_K, N, K, seed=1)
    for T in (9, 100):
        x, t, g = torch.empty((T, K), device="cuda"), torch.empty(T, dtype=torch.int64, device="cuda"), torch.ones(T, device="cuda")

        def step():
            loss, lse = q.cross_entropy(wl.Q4_K, W, x, t)
            return loss, q.cross_entropy_backward(wl.Q4_K, W, x, t, lse, g)[0]

        def fill(seed):
            x.copy_(torch.randn((T, K), generator=gen(seed)))
            t.copy_(tokens(T, N, seed=seed))

        fill(0)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        for seed in (1, 2, 3):
            fill(seed)
            graph.replay()
            torch.cuda.synchronize()
            want = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


def test_refusals_of_the_binding(q):
    w, x = torch.randn((10, 64), device="cuda"), torch.randn((3, 64), device="cuda")
    t = torch.zeros(3, dtype=torch.int64, device="cuda")
    v = torch.zeros(3, device="cuda")
    for call in (lambda: q.embedding(wl.F32, w.cpu(), t, 64), lambda: q.embedding(wl.F32, w, t.float(), 64),
                 lambda: q.embedding(wl.F32, w, t[None], 64), lambda: q.embedding(wl.F32, w, t, 64, dtype=torch.int8),
                 lambda: q.embedding(wl.F32, w, t, 64, out=x[:2]), lambda: q.embedding(wl.F32, w, t, 0),
                 lambda: q.embedding_backward(t, x[:2], 10), lambda: q.embedding_backward(t, x, 10, accumulate=True),
                 lambda: q.embedding_backward(t, x.T, 10), lambda: q.embedding_backward(t, x, 10, dtype=torch.int32),
                 lambda: q.cross_entropy(wl.F32, w, x, t[:2]), lambda: q.cross_entropy(wl.F32, w, x.T, t),
                 lambda: q.cross_entropy(wl.F32, w, x.double(), t), lambda: q.cross_entropy(wl.F32, w.flatten()[:100], x, t),
                 lambda: q.cross_entropy_backward(wl.F32, w, x, t, v[:2], v),
                 lambda: q.cross_entropy_backward(wl.F32, w, x, t, v, v.half()),
                 lambda: q.cross_entropy_backward(wl.F32, w, x, t, v, v, dw_out=w)):
        with pytest.raises(ValueError):
            call()
    W, _ = packed(wl.Q8_0, 10, 64, seed=1)
    for call, code in ((lambda: q.cross_entropy_backward(wl.Q8_0, W, x, t, v, v, weight_grad=True), q.E_TYPE),
                       (lambda: q.embedding(wl.Q8_0, W, t, 33), q.E_SHAPE), (lambda: q.embedding(77, W, t, 64), q.E_TYPE)):
        with pytest.raises(q.RetroError) as e:
            call()
        assert e.value.code == code
