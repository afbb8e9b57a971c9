"""The operators over a vocabulary where their numbers are easily lost: scales far above
a head's values, confident tokens, small losses; and the forms of the calls that wide
tables and a head trained alone take. On cuda:0, against 64 bits."""

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


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    import quantized_weight_backward_amd as q

    return q


def gen(seed):
    return torch.Generator().manual_seed(seed)


def close(got, want, bound, where=""):
    got = got.cpu().double()
    off = (got - want).abs()
    assert torch.isfinite(got).all(), where
    assert (off <= bound).all(), (where, float((off / bound.clamp(min=1e-300)).max()))


# ---------------------------------------------------------------- scales far above the head's values

# (scale's bytes, bytes of 32 codes that are all zero)
ZEROS = {
    wl.MXFP4: [(bytes([e]), b"\x80\x08" * 8) for e in (150, 160, 200, 254)],
    wl.Q8_0: [(np.float16(d).tobytes(), bytes(32)) for d in (65504.0, -65504.0)],
    wl.Q4_0: [(np.float16(65504.0).tobytes(), b"\x88" * 16)],
    wl.Q5_0: [(np.float16(65504.0).tobytes(), b"\xff" * 4 + bytes(16))],
}


@pytest.mark.parametrize("wtype,scale,zeros", [(t, *z) for t, zs in ZEROS.items() for z in zs],
                         ids=lambda v: wl.TYPE_NAMES[v] if isinstance(v, int) else v.hex()[:4])
def test_a_block_of_zeros_under_a_large_scale(q, wtype, scale, zeros):
    """It is zeros, and leaves the other weights as they are: decoded in pieces (more than 64
    tokens, rows apart) as well as read in place."""
    N, K = 300, 128
    W = wl.make_weight(wtype, N, K, np.random.Generator(np.random.PCG64(11)))
    size = W.shape[1] // (K // 32)
    W[17, size:2 * size] = np.frombuffer(scale + zeros, dtype=np.uint8)
    values = torch.from_numpy(oracle.dequantize(wtype, W, K)).reshape(N, K).double()
    assert torch.isfinite(values).all() and not values[17, 32:64].any()
    apart = torch.zeros((N, W.shape[1] + 6), dtype=torch.uint8, device="cuda")
    apart[:, :W.shape[1]] = torch.from_numpy(W)
    spread = float(values.std()) * K ** 0.5
    for T, w in ((70, torch.from_numpy(W).cuda()), (9, torch.from_numpy(W).cuda()), (9, apart[:, :W.shape[1]])):
        t = torch.randint(-1, N, (T,), generator=gen(T))
        t[0] = 17
        g = torch.rand(T, generator=gen(4)) / T
        # tokens of all columns, and of one each, whose logits show a weight's own error
        single = torch.zeros((T, K)).scatter_(1, torch.randint(0, K, (T, 1), generator=gen(8)), 8 / float(values.std()))
        for dtype, of in ((d, o) for d in (torch.bfloat16, torch.float32)
                          for o in (torch.randn((T, K), generator=gen(7)) / spread, single)):
            x = of.to(dtype)
            loss, lse = q.cross_entropy(wtype, w, x.cuda(), t.cuda())
            want, want_lse, _, _ = ref.cross_entropy(values, x.double(), t)
            bound = ref.loss_error(values, x.double(), want_lse)
            close(lse, want_lse, bound, "lse")
            close(loss, want, bound, "loss")
            dx, _ = q.cross_entropy_backward(wtype, w, x.cuda(), t.cuda(), lse, g.cuda())
            part = 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -22
            (wx, bx), _ = ref.gradients(values, x.double(), t, g, part, dtype, torch.float32,
                                        2.0 ** -11 if dtype == torch.bfloat16 else 0.0)
            close(dx, wx, bx, "dx")


@pytest.mark.parametrize("xtype,size", [(torch.bfloat16, 1e6), (torch.bfloat16, 1e-30), (torch.float16, 1e5),
                                        (torch.float16, 1e-4)], ids=lambda v: NAME.get(v, str(v)))
def test_a_row_of_the_head_that_holds_an_infinity(q, xtype, size):
    """A logit of -inf is a probability of 0; the other rows' logits are what they were."""
    T, N, K, row = 80, 200, 64, 5
    w = torch.randn((N, K), generator=gen(1)) * size
    w[row, 0] = -float("inf")
    x = torch.randn((T, K), generator=gen(2)) / (size * K ** 0.5)
    x[:, 0] = x[:, 0].abs() + x.abs().max() / 8
    x = x.to(xtype)
    assert (x[:, 0] > 0).all() and torch.isfinite(x).all()
    t = torch.randint(row + 1, N, (T,), generator=gen(3))
    want, want_lse, _, l = ref.cross_entropy(w.double(), x.double(), t)
    assert (l[:, row] == -float("inf")).all()
    finite = w.double()
    finite[row, 0] = 0
    bound = ref.loss_error(finite, x.double(), want_lse)
    loss, lse = q.cross_entropy(wl.F32, w.cuda(), x.cuda(), t.cuda())
    close(lse, want_lse, bound, "lse")
    close(loss, want, bound, "loss")
    g = torch.full((T,), 2.0 ** -10)
    dx, _ = q.cross_entropy_backward(wl.F32, w.cuda(), x.cuda(), t.cuda(), lse, g.cuda())
    # the row without its infinity has nothing of the probability either: take it out
    keep = torch.arange(N) != row
    (wx, bx), _ = ref.gradients(finite[keep], x.double(), t - 1, g, 2.0 ** -11, xtype, torch.float32, 2.0 ** -11)
    close(dx[:, 1:], wx[:, 1:], bx[:, 1:], "dx")
    assert torch.isnan(dx[:, 0]).all()  # 0 times an infinity


# ---------------------------------------------------------------- confident tokens, small losses

def confident(wtype, T):
    """(W, values, x, targets): a head of values d q, d of 11 bits and q of 8, and tokens of
    one 1 or -1 for each of up to 16 columns, the largest of their target's row: their
    probabilities are from 0.9 to 0.9999. Each logit is a whole number of steps of d, below
    2^11 * 127 * 16 < 2^22 of them, as is each partial sum of parts of it, so that F32's sums
    of it are exact in whatever order."""
    N, K = 257, 64
    rng = np.random.Generator(np.random.PCG64(21))
    d, code = np.float16(0.010765), rng.integers(-127, 128, size=(N, K), dtype=np.int8)
    assert int(d.view(np.uint16)) & 1  # all its 11 bits are used
    values = torch.from_numpy(code.astype(np.float64)) * float(d)
    if wtype == wl.Q8_0:
        blocks = np.zeros((N, K // 32, 34), dtype=np.uint8)
        blocks[..., :2] = np.frombuffer(d.tobytes(), dtype=np.uint8)
        blocks[..., 2:] = code.reshape(N, K // 32, 32).view(np.uint8)
        W = torch.from_numpy(blocks.reshape(N, -1))
    else:
        W = values.float()
        assert torch.equal(W.double(), values)
    targets = torch.randint(0, N, (T,), generator=gen(5))
    rows = values[targets]
    columns = torch.topk(rows.abs(), 16, 1).indices
    some = torch.arange(16)[None] < (9 + torch.arange(T) % 8)[:, None]
    x = torch.zeros((T, K), dtype=torch.float64).scatter_(1, columns, torch.gather(rows, 1, columns).sign() * some)
    return W, values, x, targets


@pytest.mark.parametrize("T", [33, 70, 300])
@pytest.mark.parametrize("wtype", [wl.Q8_0, wl.F32], ids=wl.TYPE_NAMES.get)
def test_gradient_of_confident_tokens(q, wtype, T):
    """d = p - 1 is a small difference: the logits of the gradients are those that lse is of."""
    W, values, x, t = confident(wtype, T)
    g = torch.rand(T, generator=gen(6)) + 0.5
    d_x, d_w, d_t = x.bfloat16().cuda(), W.cuda(), t.cuda()
    loss, lse = q.cross_entropy(wtype, d_w, d_x, d_t)
    l = x @ values.T
    exact_lse = torch.logsumexp(l, 1)
    p = torch.exp(l - exact_lse[:, None])
    rest = 1 - p[torch.arange(T), t]
    assert ((rest < 0.2) & (rest > 1e-6)).all() and (rest < 1e-3).any() and (rest > 1e-2).any()
    # logits are exact: what is left is the sum of exponentials (up to 128 a lane, 32 runs a
    # thread, 16 joins), exp and log below 2^-20, and lse's own steps
    off = (128 + 32 + 16) * 2.0 ** -24 + 2.0 ** -20 + exact_lse.abs() * 2.0 ** -23
    close(lse, exact_lse, off, "lse")
    dx, _ = q.cross_entropy_backward(wtype, d_w, d_x, d_t, lse, g.cuda())
    d = p.clone()
    d[torch.arange(T), t] = -rest
    w = values.abs()
    # exp's argument is off by lse's error and a rounding, exp itself by |argument| 2^-24 and a step
    ed = 2 * p * (off[:, None] + 2.0 ** -22 * (1 + (l - exact_lse[:, None]).abs()))
    ed = ed + 2.0 ** -11 * d.abs() + 2.0 ** -38
    N = len(values)
    # the products: d and the head's values in 11 bits each, F32 sums over the head
    bound = ed @ w + (2.0 ** -11 + (N / 16 + 64) * ref.STEP) * (d.abs() @ w) + 2.0 ** -38 * w.max() * d.abs().sum(1, keepdim=True)
    want = g.double()[:, None] * (d @ values)
    bound = g.double()[:, None] * bound
    bound = bound + ref.half_step(torch.bfloat16) * (want.abs() + bound)
    # it says something: below a tenth of the gradient of a token that p leaves a thousandth
    size = want.norm(dim=1)
    assert (bound.norm(dim=1) < size / 10)[rest > 1e-3].all()
    close(dx, want, bound, "dx")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "q8_0"])
@pytest.mark.parametrize("T", [5, 90, 600])
def test_small_losses_beside_large_logits(q, kind, T):
    """Logits of 4096, the target's 5 to 14 above: whole eighths, exact in F32."""
    N, K = 127, 128
    w = torch.zeros((N, K))
    w[:, 0] = 64
    w[torch.arange(N), torch.arange(N) + 1] = 8
    t = torch.randint(0, N, (T,), generator=gen(1))
    a = 5 + torch.arange(T) % 10
    x = torch.zeros((T, K))
    x[:, 0] = 64
    x[torch.arange(T), t + 1] = a / 8
    if kind == "q8_0":
        blocks = np.zeros((N, K // 32, 34), dtype=np.uint8)
        blocks[..., :2] = np.frombuffer(np.float16(1).tobytes(), dtype=np.uint8)
        blocks[..., 2:] = w.numpy().astype(np.int8).view(np.uint8).reshape(N, K // 32, 32)
        wtype, W, x = wl.Q8_0, torch.from_numpy(blocks.reshape(N, -1)), x.bfloat16()
    else:
        dtype = {v: k for k, v in NAME.items()}[kind]
        wtype, W, x = TYPE[dtype], w.to(dtype), x.to(dtype)
    loss, lse = q.cross_entropy(wtype, W.cuda(), x.cuda(), t.cuda())
    want = torch.log1p((N - 1) * torch.exp(-a.double()))
    # (sums of exponentials, exp and log) as for any loss, and no step of a logit of 4096 (2^-11)
    close(loss, want, torch.full_like(want, (128 + 32 + 16) * 2.0 ** -24 + 2.0 ** -20), "loss")
    close(lse, want + 4096 + a, torch.full_like(want, 2.0 ** -11), "lse")


# ---------------------------------------------------------------- the gradient of wide tables

def wide_gradient(ids, dy, N, scale):
    """(dW, sum of magnitudes, tokens a row) in 64 bits, on the device."""
    known = (ids >= 0) & (ids < N)
    at = torch.where(known, ids, N).long()
    y = dy.double() * scale
    dw = torch.zeros((N + 1, dy.shape[1]), dtype=torch.float64, device=dy.device)
    size = dw.clone()
    dw.index_add_(0, at, y)
    size.index_add_(0, at, y.abs_())
    return dw[:N], size[:N], torch.bincount(at, minlength=N + 1)[:N].double()


def wide_bound(dw, size, count, dtype, old=None):
    # each addition of a row's F32 sum, and the scale's product, rounds what is at most the sum of magnitudes
    b = (count[:, None] + 2) * 2.0 ** -24 * size
    if old is not None:
        b += 2.0 ** -24 * (old.abs() + size)
    return b + ref.half_step(dtype) * (dw.abs() + b) + torch.finfo(dtype).smallest_normal * ref.half_step(dtype)


def ids_of(T, N, seed, kind):
    g = gen(seed)
    if kind == "one":
        ids = torch.full((T,), N // 2)
    elif kind == "frequent":  # half of them one id, the others spread
        ids = torch.where(torch.rand(T, generator=g) < 0.5, 1, torch.randint(0, N, (T,), generator=g))
    else:
        ids = torch.randint(0, N, (T,), generator=g)
    return torch.where(torch.rand(T, generator=g) < 0.1, torch.tensor([-1, N])[torch.randint(0, 2, (T,), generator=g)], ids)


# several chunks of 512 columns, the last one ragged; runs of 16 tokens, and, where tokens times
# columns are 2048 waves and more, of 64, on both sides of that
WIDE = [(1, 9, 513, "spread"), (63, 5, 1000, "frequent"), (300, 40, 1029, "spread"), (777, 3200, 1000, "frequent"),
        (2000, 7, 520, "one"), (8128, 30, 8192, "frequent"), (8200, 30, 8191, "spread"), (16320, 100, 4096, "spread"),
        (16384, 100, 4096, "frequent"), (16385, 2, 4100, "spread"), (43700, 11, 1029, "one"), (65600, 900, 520, "frequent"),
        (131009, 500, 24, "spread"), (131072, 3, 8, "frequent"), (140001, 5000, 33, "one")]


@pytest.mark.parametrize("T,N,K,kind", WIDE, ids=str)
def test_embedding_backward_of_wide_tables(q, T, N, K, kind):
    dtype = FLOATS[(T + K) % 3]
    ids = ids_of(T, N, T, kind).to(torch.int32 if T % 2 else torch.int64).cuda()
    dy = torch.randn((T, K), generator=torch.Generator(device="cuda").manual_seed(T), device="cuda").to(dtype)
    dw, size, count = wide_gradient(ids, dy, N, 0.75)

    def near(got, want, bound):
        assert torch.isfinite(got).all()
        assert ((got.double() - want).abs() <= bound).all()

    got = q.embedding_backward(ids, dy, N, scale=0.75)
    near(got, dw, wide_bound(dw, size, count, torch.float32))
    assert not got[count == 0].any()
    assert torch.equal(got, q.embedding_backward(ids, dy, N, scale=0.75))
    # rows of a wider tensor, of the gradient's own type: written, and added to
    base = torch.randn((N, K + 5), generator=gen(5)).to(dtype).cuda()
    out = base.clone()
    q.embedding_backward(ids, dy, N, scale=0.75, out=out[:, 2:2 + K], dtype=dtype)
    near(out[:, 2:2 + K], dw, wide_bound(dw, size, count, dtype))
    assert torch.equal(out[:, :2], base[:, :2]) and torch.equal(out[:, 2 + K:], base[:, 2 + K:])
    out = base.clone()
    q.embedding_backward(ids, dy, N, scale=0.75, out=out[:, 2:2 + K], accumulate=True)
    old = base[:, 2:2 + K].double()
    near(out[:, 2:2 + K], dw + old, wide_bound(dw + old, size, count, dtype, old))
    assert torch.equal(out[count == 0], base[count == 0])
    assert torch.equal(out[:, :2], base[:, :2]) and torch.equal(out[:, 2 + K:], base[:, 2 + K:])


def test_embedding_backward_of_whole_tokens(q):
    """Whole numbers, whose sums are exact: equal, whatever the runs are."""
    for T, N, K in ((16384, 50, 4096), (3000, 9, 700), (131100, 77, 16)):
        ids = ids_of(T, N, 3, "frequent").cuda()
        dy = torch.randint(-8, 9, (T, K), generator=gen(2)).to(torch.bfloat16).cuda()
        dw, _, _ = wide_gradient(ids, dy, N, 0.5)
        assert torch.equal(q.embedding_backward(ids, dy, N, scale=0.5).double(), dw)


# ---------------------------------------------------------------- the head's gradient alone

@pytest.mark.parametrize("xtype,wdtype,T,N,K", [
    (torch.bfloat16, torch.bfloat16, 70, 500, 128), (torch.bfloat16, torch.bfloat16, 300, 33100, 40),
    (torch.float32, torch.float32, 70, 33000, 64), (torch.float16, torch.float32, 5, 300, 33),
    (torch.float32, torch.bfloat16, 129, 1000, 72), (torch.float16, torch.float16, 1, 7, 3)], ids=str)
def test_the_gradient_of_the_head_alone(q, xtype, wdtype, T, N, K):
    """dX not asked for: the same bits of dW, through a workspace that is not cleared."""
    w = (torch.randn((N, K), generator=gen(1)) * 0.3).to(wdtype).cuda()
    x = torch.randn((T, K), generator=gen(2)).to(xtype).cuda()
    t = torch.randint(-1, N, (T,), generator=gen(3)).cuda()
    g = torch.rand(T, generator=gen(4)).cuda()
    wt, xt = TYPE[wdtype], TYPE[xtype]
    _, lse = q.cross_entropy(wt, w, x, t)
    _, want = q.cross_entropy_backward(wt, w, x, t, lse, g, weight_grad=True)
    ldw = K * w.element_size()
    need = q.lib.retro_cross_entropy_backward_workspace_size(wt, ldw, xt, 1, K, N, T)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    got = torch.full((N, K + 3), 9.0, dtype=wdtype, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        assert q.lib.retro_cross_entropy_backward(
            wt, w.data_ptr(), ldw, xt, x.data_ptr(), K, 27, t.data_ptr(), lse.data_ptr(), g.data_ptr(), None, 0,
            got.data_ptr(), K + 3, K, N, T, ws.data_ptr(), need, stream) == 0
        assert torch.equal(got[:, :K], want) and (got[:, K:] == 9.0).all()
        assert (ws[need:] == 255).all()
