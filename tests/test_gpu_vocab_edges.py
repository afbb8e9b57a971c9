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
