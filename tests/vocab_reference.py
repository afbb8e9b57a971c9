"""The operators over a vocabulary by their definition, in 64 bits on the CPU, and
bounds of what a result in fewer bits may be off by.

Half a step of rounding is eps / 2 of the value: 2^-9 BF16, 2^-12 F16, 2^-24 F32 (their
finfo eps is 2^-7, 2^-10, 2^-23; eps / 2 bounds the relative error as 2^-8, 2^-11, 2^-24).
"""

import torch

# a sum on the matrix cores: 16 products an instruction, each adding at most a few
# roundings of the running sum, whose size the sum of magnitudes bounds
STEP = 2.0 ** -22


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def cross_entropy(w, x, targets):
    """(loss, lse, learnt, logits) of float64 w (N x K) and x (T x K)."""
    l = x @ w.T
    lse = torch.logsumexp(l, 1)
    learnt = (targets >= 0) & (targets < w.shape[0])
    at = l[torch.arange(len(x)), torch.where(learnt, targets, 0)]
    return torch.where(learnt, lse - at, 0.0), lse, learnt, l


def logit_error(w, x):
    """What a logit may be off by: K / 16 instructions' sums, and the parts that the
    operands are taken in (2^-22 of each, and 2^-38 of the largest of x's row and of W, or 2^-151)."""
    K = x.shape[1]
    size = x.abs() @ w.abs().T
    of_x = torch.clamp(2.0 ** -38 * x.abs().amax(1, keepdim=True), min=2.0 ** -151)
    of_w = torch.clamp(2.0 ** -38 * w.abs().max(), min=2.0 ** -151)
    small = of_x * w.abs().sum(1) + of_w * x.abs().sum(1, keepdim=True)
    return ((K / 16 + 4) * STEP + 3 * 2.0 ** -22) * size + small


def loss_error(w, x, lse):
    """Of loss and lse: two logits', and those of exp, of the sum (up to 128 terms a
    lane, 32 runs a thread) and of log, each below 2^-20."""
    return 2 * logit_error(w, x).amax(1) + (128 + 32 + 16) * 2.0 ** -24 + 2.0 ** -20 + lse.abs() * 2.0 ** -22


def gradients(w, x, targets, dloss, part_error, dtype_x, dtype_w, head_error=0.0):
    """((dx, its bound), (dw, its bound)). part_error is the relative rounding of d in
    the products, head_error that of the head's values in logits and products; d's own
    error is that of exp: two logits' and lse's."""
    loss, lse, learnt, l = cross_entropy(w, x, targets)
    p = torch.exp(l - lse[:, None])
    d = p.clone()
    t = torch.nonzero(learnt)[:, 0]
    d[t, targets[t]] -= 1
    g = torch.where(learnt, dloss.double(), 0.0)[:, None]
    d = torch.where(learnt[:, None], d, 0.0)
    off = logit_error(w, x) + loss_error(w, x, lse)[:, None] + 2.0 ** -20 + head_error * (x.abs() @ w.abs().T)
    # exp(off) - 1, at most twice off while that is below 1
    off = torch.where(off < 1, 2 * off, torch.exp(off))
    # 2^-39: the smallest steps of F16 under the scale of 2^14
    ed = p * off + 2.0 ** -23 * d.abs() + part_error * d.abs() + 2.0 ** -38
    ed = torch.where(learnt[:, None], ed, 0.0)
    x = torch.where(learnt[:, None], x, 0.0)
    N, T = w.shape[0], x.shape[0]
    dx, dw = g * (d @ w), (g * d).T @ x
    sums = 3 * 2.0 ** -22
    bx = g.abs() * (ed @ w.abs() + ((N / 16 + 64) * STEP + sums + head_error) * (d.abs() @ w.abs()) + 2.0 ** -38 * w.abs().max() * d.abs().sum(1, keepdim=True))
    top = g.abs().max() * x.abs().max()
    bw = (g.abs() * ed).T @ x.abs() + ((T / 16 + 64) * STEP + sums) * ((g * d).abs().T @ x.abs()) + 2.0 ** -38 * top * T
    tiny_x, tiny_w = torch.finfo(dtype_x).smallest_normal, torch.finfo(dtype_w).smallest_normal
    return ((dx, bx + half_step(dtype_x) * (dx.abs() + bx) + tiny_x * half_step(dtype_x)),
            (dw, bw + half_step(dtype_w) * (dw.abs() + bw) + tiny_w * half_step(dtype_w)))
