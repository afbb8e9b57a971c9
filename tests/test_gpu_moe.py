"""The expert layer on cuda:0 against its definition in 64 bits."""

import pytest
import torch

import mx_reference as ref

pytestmark = pytest.mark.gpu

NAME = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    import quantized_weight_backward_amd as q

    return q


def layer(T, D, F, E, dtype, seed, router_dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, D), generator=g).to(dtype)
    router = (torch.randn((E, D), generator=g) / D ** 0.5).to(router_dtype)
    return x, router, ref.random_planes(g, E * 2 * F, D, 119, 122), ref.random_planes(g, E * D, F, 119, 122)


def on_gpu(q, planes, K):
    return q.MXMatrix(planes[0].cuda(), planes[1].cuda(), K)


def check(y, want, bound, dtype):
    err = (y.cpu().double() - want).abs()
    limit = bound + ref.OUT_ULP[dtype] * want.abs() + torch.finfo(dtype).smallest_normal
    assert (err <= limit).all(), float((err / limit).max())


CASES = [(1, 64, 32, 4, 2), (1, 256, 256, 1, 1), (2, 100, 33, 3, 3), (3, 257, 300, 8, 2), (5, 512, 100, 64, 8),
         (16, 300, 128, 16, 4), (17, 128, 520, 2, 1), (33, 96, 64, 4, 4), (40, 160, 96, 256, 16), (64, 288, 160, 8, 2),
         (64, 64, 48, 1, 1), (64, 64, 48, 16, 16), (7, 1, 1, 5, 2), (1, 2048, 1000, 32, 4), (20, 40, 2000, 6, 3)]


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=NAME.get)
def test_layer(q, dtype, case, renormalize):
    T, D, F, E, k = case
    x, router, gu, dn = layer(T, D, F, E, dtype, seed=T + D)
    out = torch.full((T, D + 3), float("nan"), dtype=dtype, device="cuda")
    y = q.mx_moe(x.cuda(), router.cuda(), on_gpu(q, gu, D), on_gpu(q, dn, F), k, renormalize, out=out[:, :D])
    assert out[:, D:].isnan().all()
    check(y, *ref.moe(x, router, gu[2], dn[2], k, renormalize), dtype)


# Layers large enough for workgroups to share the down product's rows: outputs that
# end in the first and in the second half of a workgroup's, few pieces and many,
# experts with more than 16 tokens, all three types' stages.
LARGE = [(2, 520, 9000, 4, 2), (16, 300, 2000, 8, 4), (17, 390, 2000, 8, 4), (33, 1, 3000, 4, 2), (40, 96, 2000, 2, 2),
         (16, 96, 3000, 16, 4), (64, 257, 1100, 8, 8), (5, 1030, 5000, 3, 2), (32, 130, 4200, 2, 1),
         (32, 40, 300, 256, 16), (64, 40, 300, 256, 16)]


@pytest.mark.parametrize("case", LARGE, ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=NAME.get)
def test_large_layer(q, dtype, case):
    T, D, F, E, k = case
    x, router, *planes = layer(T, D, F, E, dtype, seed=T + D)
    gu, dn = on_gpu(q, planes[0], D), on_gpu(q, planes[1], F)
    out = torch.full((T, D + 3), float("nan"), dtype=dtype, device="cuda")
    y = q.mx_moe(x.cuda(), router.cuda(), gu, dn, k, out=out[:, :D])
    assert out[:, D:].isnan().all()
    again = [q.mx_moe(x.cuda(), router.cuda(), gu, dn, k) for _ in range(5)]
    assert all(torch.equal(a, y) for a in again)
    check(y, *ref.moe(x, router, planes[0][2], planes[1][2], k, True), dtype)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=NAME.get)
def test_a_token_that_is_not_finite_in_a_large_layer(q, dtype, bad):
    """The other columns of its tiles, which are multiplied beside it, are untouched."""
    T, D, F, E, k = 20, 390, 2000, 3, 2
    x, router, gu, dn = layer(T, D, F, E, dtype, 8)
    x[7, 100] = bad
    y = q.mx_moe(x.cuda(), router.cuda(), on_gpu(q, gu, D), on_gpu(q, dn, F), k)
    assert not torch.isfinite(y[7]).any()
    good = [t for t in range(T) if t != 7]
    check(y[good], *ref.moe(x[good], router, gu[2], dn[2], k, True), dtype)


@pytest.mark.parametrize("shape", [(3, 64, 32, 4, 2), (20, 130, 2000, 6, 3)], ids=str)
def test_the_largest_finite_x(q, shape):
    """x whose BF16 rounding is an infinity, with weights small enough for finite
    products."""
    T, D, F, E, k = shape
    x, router, gu, dn = layer(T, D, F, E, torch.float32, 6)
    x[:, ::7] = torch.finfo(torch.float32).max * torch.sign(x[:, ::7])
    router = router * 2.0 ** -120
    gu = (gu[0], (gu[1].int() - 112).clamp(min=0).to(torch.uint8), gu[2] * 2.0 ** -112)
    y = q.mx_moe(x.cuda(), router.cuda(), on_gpu(q, gu, D), on_gpu(q, dn, F), k)
    assert torch.isfinite(y).all()
    check(y, *ref.moe(x, router, gu[2], dn[2], k, True), torch.float32)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=NAME.get)
def test_router_of_x_type_and_strided_views(q, dtype):
    T, D, F, E, k = 6, 130, 70, 9, 3
    x, router, gu, dn = layer(T, D, F, E, dtype, 4, router_dtype=dtype)
    wide = torch.full((T, D + 7), float("nan"), dtype=dtype, device="cuda")
    wide[:, 5:5 + D] = x.cuda()
    rw = torch.full((E, D + 1), float("nan"), dtype=dtype, device="cuda")
    rw[:, :D] = router.cuda()
    y = q.mx_moe(wide[:, 5:5 + D], rw[:, :D], on_gpu(q, gu, D), on_gpu(q, dn, F), k)
    check(y, *ref.moe(x, router, gu[2], dn[2], k, True), dtype)


def test_equal_logits_go_to_the_lowest_index(q):
    T, D, F, E, k = 4, 64, 32, 12, 3
    x, router, gu, dn = layer(T, D, F, E, torch.float32, 5)
    router[:] = router[0]
    y = q.mx_moe(x.cuda(), router.cuda(), on_gpu(q, gu, D), on_gpu(q, dn, F), k)
    check(y, *ref.moe(x, router, gu[2], dn[2], k, True), torch.float32)
    router[:] = 0
    y = q.mx_moe(x.cuda(), router.cuda(), on_gpu(q, gu, D), on_gpu(q, dn, F), k, renormalize=False)
    check(y, *ref.moe(x, router, gu[2], dn[2], k, False), torch.float32)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_token_that_is_not_finite_spoils_its_row_alone(q, bad):
    T, D, F, E, k = 9, 96, 64, 8, 2
    x, router, gu, dn = layer(T, D, F, E, torch.bfloat16, 6)
    want, bound = ref.moe(x, router, gu[2], dn[2], k, True)
    x[4, 10] = bad
    y = q.mx_moe(x.cuda(), router.cuda(), on_gpu(q, gu, D), on_gpu(q, dn, F), k)
    assert y[4].isnan().all()
    keep = [t for t in range(T) if t != 4]
    check(y[keep], want[keep], bound[keep], torch.bfloat16)


def test_an_expert_that_no_token_chose_is_not_read(q):
    T, D, F, E, k = 3, 64, 32, 6, 2
    x, router, gu, dn = layer(T, D, F, E, torch.float32, 7)
    want, bound = ref.moe(x, router, gu[2], dn[2], k, True)
    ids = torch.topk(x.double() @ router.double().T, k, dim=1).indices
    unused = [e for e in range(E) if not (ids == e).any()]
    assert unused
    for e in unused:
        gu[1][:, e * 2 * F:(e + 1) * 2 * F] = 255
        dn[1][:, e * D:(e + 1) * D] = 255
    y = q.mx_moe(x.cuda(), router.cuda(), on_gpu(q, gu, D), on_gpu(q, dn, F), k)
    check(y, want, bound, torch.float32)


def test_no_tokens(q):
    x, router, gu, dn = layer(0, 64, 32, 4, torch.bfloat16, 8)
    assert q.mx_moe(x.cuda(), router.cuda(), on_gpu(q, gu, 64), on_gpu(q, dn, 32), 2).shape == (0, 64)


def test_same_result_every_time_and_on_another_stream(q):
    T, D, F, E, k = 24, 300, 200, 16, 4
    x, router, gu, dn = layer(T, D, F, E, torch.bfloat16, 9)
    args = (x.cuda(), router.cuda(), on_gpu(q, gu, D), on_gpu(q, dn, F), k)
    want = q.mx_moe(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [q.mx_moe(*args, stream=side) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_a_captured_layer_replays_like_eager_calls(q):
    T, D, F, E, k = 5, 200, 90, 8, 2
    _, router, gu, dn = layer(T, D, F, E, torch.bfloat16, 10)
    x = torch.zeros((T, D), dtype=torch.bfloat16, device="cuda")
    args = (router.cuda(), on_gpu(q, gu, D), on_gpu(q, dn, F), k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q.mx_moe(x, *args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = q.mx_moe(x, *args)
    for i in range(4):
        x.copy_(layer(T, D, F, E, torch.bfloat16, 30 + i)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, q.mx_moe(x, *args)), i


# Batches whose router takes four tokens a wave (more than 2048 logits): whole
# 512-element steps and a ragged end, all tokens and a last few.
ROUTED = [(33, 1032, 64, 128, 4), (64, 2048, 40, 64, 8), (62, 520, 33, 40, 3), (43, 1537, 48, 64, 2)]


@pytest.mark.parametrize("router_of_x", [False, True])
@pytest.mark.parametrize("case", ROUTED, ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=NAME.get)
def test_router_of_many_tokens(q, dtype, case, router_of_x):
    T, D, F, E, k = case
    x, router, gu, dn = layer(T, D, F, E, dtype, T + D, router_dtype=dtype if router_of_x else torch.float32)
    planes = on_gpu(q, gu, D), on_gpu(q, dn, F)
    want = ref.moe(x, router, gu[2], dn[2], k, True)
    check(q.mx_moe(x.cuda(), router.cuda(), *planes, k), *want, dtype)
    wide = torch.full((T, D + 3), float("nan"), dtype=dtype, device="cuda")  # rows off the 16-byte boundaries
    wide[:, 1:1 + D] = x.cuda()
    check(q.mx_moe(wide[:, 1:1 + D], router.cuda(), *planes, k), *want, dtype)
