"""The microscaled 4-bit operators and the mixture-of-experts layer: cases, plain forms and the definition in 64 bits.

Three groups of operators are measured:

quantise   float tensors to 4-bit elements with a shared scale per block: microscaled matrices along rows, along columns
           or both in one pass, and packed MXFP4 / NVFP4 blocks. Returned as the values the 4-bit form stands for.
linear     y = x W^T with x quantised in the call and W resident in 4 bits (forward), and its two gradients.
moe        a whole mixture-of-experts layer for a few tokens: router, top-k, gated expert products, weighted sum.

A microscaled matrix of `rows` x `K` is two tensors, with Kp = K rounded up to 256:
    codes   uint8 [rows, Kp / 2]       element 2i in the low nibble of byte i, element 2i + 1 in the high one
    scales  uint8 [Kp / 256, rows, 8]  the scale byte e (value 2^(e - 127)) of block 8c + j of row r is scales[c, r, j]
A block is 32 elements along K; codes past K are zero.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MXFP4, NVFP4 = 39, 40  # type ids of the packed blocks


# ---------------------------------------------------------------- cases

def listed():
    return [
        # activations of a 16-token batch in front of a 14336-wide product: a few microseconds, latency counts
        dict(name="quant_rows_t16_k14336", op="quant", axis="rows", rows=16, cols=14336, dtype="bf16", sigma=1.0),
        # the output gradient of a linear layer, needed along both axes by the two gradient products
        dict(name="quant_both_t4096_n4096", op="quant", axis="both", rows=4096, cols=4096, dtype="bf16", sigma=1e-3),
        # a ragged gradient along its columns only, in 32 bits
        dict(name="quant_cols_t1237_n1000", op="quant", axis="cols", rows=1237, cols=1000, dtype="f32", sigma=1e-3),
        # a whole weight into resident packed blocks, as after an optimiser's step
        dict(name="quant_nvfp4_n17408_k5120", op="quant", axis="nvfp4", rows=17408, cols=5120, dtype="f32", sigma=0.02),
        # one generated token through an up projection
        dict(name="linear_t1_n14336_k4096", op="linear", T=1, N=14336, K=4096, dtype="bf16"),
        # a short batch through a down projection
        dict(name="linear_t16_n4096_k14336", op="linear", T=16, N=4096, K=14336, dtype="bf16"),
        # a prompt through an up projection: the largest product
        dict(name="linear_t4096_n14336_k4096", op="linear", T=4096, N=14336, K=4096, dtype="bf16"),
        # odd sizes, half precision
        dict(name="linear_t333_n1000_k1500", op="linear", T=333, N=1000, K=1500, dtype="f16"),
        # the gradients of a large layer's input and weight
        dict(name="grad_t2048_n17408_k5120", op="grad", T=2048, N=17408, K=5120, dtype="bf16"),
        # one token through 4 of 32 experts
        dict(name="moe_t1_e32_top4", op="moe", T=1, D=2048, F=1024, E=32, top_k=4, renormalize=True, dtype="bf16"),
        # a decode batch through 8 of 64 experts of an odd width
        dict(name="moe_t16_e64_top8", op="moe", T=16, D=2048, F=1000, E=64, top_k=8, renormalize=True, dtype="bf16"),
        # wide experts, two a token, shares over all experts
        dict(name="moe_t32_e8_top2", op="moe", T=32, D=4096, F=14336, E=8, top_k=2, renormalize=False, dtype="bf16"),
    ]


def _size(rng, lo, hi):
    """A size spread over its logarithm: one in three odd, the others of whole 32s where they are large enough."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 1 / 3 or n < 32:
        n |= 1
    else:
        n = n // 32 * 32
    return min(max(n, lo), hi)


def draw(rng):
    while True:
        op = rng.choice(("quant", "linear", "grad", "moe"))
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        if op == "quant":
            axis = rng.choice(("rows", "cols", "both", "mxfp4", "nvfp4"))
            cols = _size(rng, 64, 17408)
            if axis in ("mxfp4", "nvfp4"):
                cols = max(64, cols // 64 * 64)  # packed rows are whole blocks
            c = dict(op=op, axis=axis, rows=_size(rng, 1, 17408), cols=cols, dtype=dtype,
                     sigma=10.0 ** rng.uniform(-2.0 if dtype == "f16" or axis == "nvfp4" else -6.0, 1.0))
        elif op == "linear":
            c = dict(op=op, T=_size(rng, 1, 4096), N=_size(rng, 256, 17408), K=_size(rng, 256, 14336), dtype=dtype)
        elif op == "grad":
            c = dict(op=op, T=_size(rng, 16, 4096), N=_size(rng, 256, 17408), K=_size(rng, 256, 8192), dtype=dtype)
        else:
            E = rng.choice((4, 8, 16, 32, 64, 128))
            c = dict(op=op, T=_size(rng, 1, 64), D=_size(rng, 256, 4096), F=_size(rng, 128, 4096), E=E,
                     top_k=rng.randint(1, min(8, E)), renormalize=rng.random() < 0.5, dtype=dtype)
        w, most = work(c), {"quant": 17408 * 5120 * 8.0, "moe": 7.4e8}.get(op, math.inf)
        if w["bytes"] <= most and w["flops"] <= 4.0 * 2048 * 17408 * 5120 and 3072 not in c.values():
            return c


# ---------------------------------------------------------------- inputs

def _activations(g, rows, cols, dtype, sigma=1.0):
    """Activations or gradients: normal values, a few wide columns, one row in 16 all zero (a masked token)."""
    x = torch.randn((rows, cols), generator=g, device="cuda") * sigma
    x *= torch.where(torch.rand((1, cols), generator=g, device="cuda") < 0.01, 8.0, 1.0)
    if rows > 4:
        x *= torch.rand((rows, 1), generator=g, device="cuda") >= 1 / 16
    return x.to(dtype)


def _planes(g, rows, K, scale_log2):
    """A resident microscaled weight: uniform codes, scale bytes of a few neighbouring powers of two, zeros past K."""
    Kp = (K + 255) // 256 * 256
    codes = torch.randint(0, 256, (rows, Kp // 2), generator=g, device="cuda", dtype=torch.uint8)
    codes[:, (K + 1) // 2:] = 0
    if K % 2:
        codes[:, K // 2] &= 15
    scales = torch.randint(127 + scale_log2 - 1, 127 + scale_log2 + 2, (Kp // 256, rows, 8), generator=g, device="cuda",
                           dtype=torch.uint8)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 2654435761 % (1 << 62))
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = dict(case)
    if op == "quant":
        s["x"] = _activations(g, case["rows"], case["cols"], dtype, case["sigma"])
    elif op == "linear":
        s["x"] = _activations(g, case["T"], case["K"], dtype)
        s["w"] = _planes(g, case["N"], case["K"], -7)
    elif op == "grad":
        s["x"] = _activations(g, case["T"], case["K"], dtype)
        s["dy"] = _activations(g, case["T"], case["N"], dtype, 1e-2)
        s["wt"] = _planes(g, case["K"], case["N"], -7)  # W^T, blocks along n
    else:
        T, D, F, E, k = (case[n] for n in ("T", "D", "F", "E", "top_k"))
        s["router"] = torch.randn((E, D), generator=g, device="cuda") / D ** 0.5
        # tokens whose k-th and next expert are nearer than 32 bits can tell apart are left out
        x = torch.randn((T + 64, D), generator=g, device="cuda").to(dtype)
        if k < E:
            top = torch.topk(x.double() @ s["router"].double().T, k + 1, dim=1).values
            x = x[torch.topk(top[:, k - 1] - top[:, k], T).indices.sort().values].contiguous()
        else:
            x = x[:T].contiguous()
        s["x"] = x
        s["gate_up"] = _planes(g, E * 2 * F, D, -7)  # each expert: F gate rows, then F up rows
        s["down"] = _planes(g, E * D, F, -7)
    return s


# ---------------------------------------------------------------- plain forms (32 bits)

def _pow2(e):
    """2^e for whole e of -126 .. 127, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _to_grid(v):
    """|v| of any size to the nearest of GRID, ties to the even code, with v's sign."""
    a = v.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.copysign(torch.clamp(torch.round(a / step) * step, max=6.0), v)


def _mx_values(x):
    """Values of x after microscaled quantisation along its last axis (float32)."""
    K = x.shape[-1]
    b = torch.nn.functional.pad(x.float(), (0, -K % 32)).unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.clamp(torch.frexp(amax).exponent - 3, -127, 127)
    e = torch.where(amax > 0, e, -127)
    # both factors of 2^-e are normal numbers, so no step of the scaling rounds
    h = e.div(2, rounding_mode="floor")
    v = _to_grid(b * _pow2(-h) * _pow2(h - e))
    return (v * _pow2(h) * _pow2(e - h)).flatten(-2)[..., :K]


def _nv_values(x):
    """Values of x after NVFP4 quantisation: blocks of 16, an E4M3 scale each (float32)."""
    b = x.float().unflatten(-1, (-1, 16))
    amax = b.abs().amax(-1, keepdim=True)
    # nearest E4M3 to amax / 6: the step at 2^p is 2^(p - 3), at least 2^-9; amax / (6 step) is rounded to even
    p = torch.clamp(torch.frexp(amax / 6.0).exponent - 1, min=-6)
    step = _pow2(p - 3)
    scale = torch.clamp(torch.round(amax / (6.0 * step)) * step, max=448.0)
    # |x| against scale times the grid's midpoints, which is exact where x / scale would round; at a tie the even code
    grid = torch.tensor(GRID, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2 * scale.unsqueeze(-1)
    a = b.abs().unsqueeze(-1)
    up = torch.arange(7, device=x.device) % 2 == 1
    code = ((a > mid) | ((a == mid) & up)).sum(-1, dtype=torch.uint8)
    return torch.where(scale > 0, torch.copysign(grid[code.int()], b) * scale, 0.0).flatten(-2)


def _plane_values(codes, scales, K):
    """A microscaled matrix's values (float32)."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    v = torch.stack((grid[(codes & 15).int()], grid[(codes >> 4).int()]), -1).flatten(-2)
    s = _pow2(scales.permute(1, 0, 2).flatten(1).int() - 127)
    return (v.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)[:, :K]


def _plain_quant(s):
    x, axis = s["x"], s["axis"]
    if axis == "nvfp4":
        return _nv_values(x)
    if axis == "mxfp4":
        return _mx_values(x)
    rows = _mx_values(x).to(x.dtype) if axis != "cols" else None
    cols = _mx_values(x.T).to(x.dtype) if axis != "rows" else None
    return [v for v in (rows, cols) if v is not None]


def _plain_linear(s):
    return (_mx_values(s["x"]) @ _plane_values(*s["w"], s["K"]).T).to(s["x"].dtype)


def _plain_grad(s):
    dx = (_mx_values(s["dy"]) @ _plane_values(*s["wt"], s["N"]).T).to(s["x"].dtype)
    return dx, _mx_values(s["dy"].T) @ _mx_values(s["x"].T).T


def _plain_moe(s):
    T, D, F, E, k = (s[n] for n in ("T", "D", "F", "E", "top_k"))
    x = s["x"].float()
    logits = x @ s["router"].T
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = order.values[:, :k], order.indices[:, :k]
    over = top if s["renormalize"] else logits
    e = torch.exp(over - top[:, :1])
    p = (torch.exp(top - top[:, :1]) / e.sum(1, keepdim=True))
    share = torch.zeros((T, E), device=x.device).scatter_(1, ids, p)
    gu = torch.matmul(_plane_values(*s["gate_up"], D).view(E, 2 * F, D), x.T)  # E, 2F, T
    gate, up = gu[:, :F], gu[:, F:]
    h = gate / (1 + torch.exp(-gate)) * up * share.T.unsqueeze(1)
    y = torch.matmul(_plane_values(*s["down"], F).view(E, D, F), h)  # E, D, T
    return y.sum(0).T.to(s["x"].dtype)


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["op"]
    if not own:
        return {"quant": _plain_quant, "linear": _plain_linear, "grad": _plain_grad, "moe": _plain_moe}[op](state)
    import quantized_weight_backward_amd as q

    x = state["x"]
    if op == "quant":
        axis = state["axis"]
        if axis in ("mxfp4", "nvfp4"):
            wtype = q.MXFP4 if axis == "mxfp4" else q.NVFP4
            return q.dequantize(wtype, q.quantize(wtype, x), x.shape[1], x.shape[0])
        made = q.mx_quantize_both(x) if axis == "both" else (q.mx_quantize(x, axis=1 if axis == "rows" else 0),)
        return [q.mx_dequantize(m, x.dtype) for m in made]
    if op == "linear":
        return q.mx_linear(x, q.MXMatrix(*state["w"], state["K"]))
    if op == "grad":
        return q.mx_linear_backward(state["dy"], x, q.MXMatrix(*state["wt"], state["N"]))
    return q.mx_moe(x, state["router"], q.MXMatrix(*state["gate_up"], state["D"]),
                    q.MXMatrix(*state["down"], state["F"]), state["top_k"], renormalize=state["renormalize"])


def work(case):
    """Bytes: each input read and each output written once, 4-bit operands at 17 bytes per 32 elements."""
    size = {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
    mx = 17 / 32
    if case["op"] == "quant":
        n = case["rows"] * case["cols"]
        # the values go out in x's type, once an axis; packed blocks decode to 32 bits
        out = 4 if case["axis"] in ("mxfp4", "nvfp4") else size * (2 if case["axis"] == "both" else 1)
        return {"bytes": n * (size + out), "flops": n}
    if case["op"] == "moe":
        T, D, F, E, k = (case[n] for n in ("T", "D", "F", "E", "top_k"))
        experts = min(E, E * (1 - (1 - k / E) ** T))  # distinct ones that T tokens choose, on average
        return {"bytes": experts * 3 * F * D * mx + E * D * 4 + 2 * T * D * size,
                "flops": 6 * T * k * F * D + 2 * T * E * D}
    T, N, K = case["T"], case["N"], case["K"]
    if case["op"] == "linear":
        return {"bytes": T * K * size + N * K * mx + T * N * size, "flops": 2 * T * N * K}
    return {"bytes": T * (K + N) * size + N * K * mx + T * K * size + N * K * 4, "flops": 4 * T * N * K}


# ---------------------------------------------------------------- the definition, in 64 bits

def _nearest(v):
    """v to the nearest of the 4-bit grid by comparison with the midpoints; a tie goes to the even code."""
    grid = torch.tensor(GRID, dtype=torch.float64, device=v.device)
    mid = (grid[1:] + grid[:-1]) / 2
    a = v.abs().contiguous()
    lo, hi = torch.searchsorted(mid, a, right=False), torch.searchsorted(mid, a, right=True)
    code = torch.where(lo % 2 == 0, lo, hi)  # lo != hi only at a midpoint, and then they are neighbours
    return grid[code] * torch.where(torch.signbit(v), -1.0, 1.0).double()


def _exact_mx(x, axis):
    x = x.double() if axis == 1 else x.double().T
    rows, K = x.shape
    b = torch.zeros((rows, (K + 31) // 32 * 32), dtype=torch.float64, device=x.device)
    b[:, :K] = x
    b = b.reshape(rows, -1, 32)
    amax = b.abs().max(2, keepdim=True).values
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, 2.0 ** -200)))
    # log2 may round at the ends of a binade
    e = torch.where(torch.exp2(e) > amax, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e)
    scale = torch.exp2(torch.clamp(e - 2, -127, 127))
    return (_nearest(b / scale) * scale).reshape(rows, -1)[:, :K]


def _exact_nv(x):
    b = x.double().reshape(x.shape[0], -1, 16)
    amax = b.abs().max(2, keepdim=True).values
    # all finite E4M3 values in order; an even position is an even mantissa
    m = [k * 2.0 ** -9 for k in range(8)] + [(8 + k) * 2.0 ** (p - 3) for p in range(-6, 9) for k in range(8)][:-1]
    table = torch.tensor(m, dtype=torch.float64, device=x.device)
    mid6 = (table[1:] + table[:-1]) * 3.0  # six times the midpoints, exact
    lo, hi = torch.searchsorted(mid6, amax, right=False), torch.searchsorted(mid6, amax, right=True)
    scale = table[torch.where(lo % 2 == 0, lo, hi)]
    # v / scale is only compared with midpoints of few bits: a quotient in 64 bits never rounds onto one
    return (_nearest(b / torch.where(scale > 0, scale, 1.0)) * scale).reshape(x.shape)


def _exact_planes(codes, scales, K):
    out = torch.empty((codes.shape[0], codes.shape[1] * 2), dtype=torch.float64, device=codes.device)
    for at, nibble in ((0, codes & 15), (1, codes >> 4)):
        mag = (nibble & 7).double()
        m = torch.where(mag < 2, mag / 2, (2 + mag % 2) * torch.exp2(torch.floor(mag / 2) - 2))
        out[:, at::2] = torch.where(nibble >= 8, -m, m)
    for c in range(scales.shape[0]):
        s = torch.exp2(scales[c].double() - 127)
        out[:, 256 * c:256 * c + 256] *= s.repeat_interleave(32, dim=1)
    return out[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    op, x = case["op"], s["x"]
    if op == "quant":
        axis = case["axis"]
        if axis == "nvfp4":
            return _exact_nv(x)
        if axis == "mxfp4":
            return _exact_mx(x, 1)
        return [_exact_mx(x, a) for a, on in ((1, axis != "cols"), (0, axis != "rows")) if on]
    if op == "linear":
        return torch.mm(_exact_mx(x, 1), _exact_planes(*s["w"], case["K"]).T)
    if op == "grad":
        dx = torch.mm(_exact_mx(s["dy"], 1), _exact_planes(*s["wt"], case["N"]).T)
        return dx, torch.mm(_exact_mx(s["dy"], 0), _exact_mx(x, 0).T)
    T, D, F, E, k = (case[n] for n in ("T", "D", "F", "E", "top_k"))
    x = x.double()
    logits = x @ s["router"].double().T
    prob = torch.softmax(logits, dim=1)
    y = torch.zeros((T, D), dtype=torch.float64, device=x.device)
    chosen = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    kept = torch.gather(prob, 1, chosen)
    if case["renormalize"]:
        kept = kept / kept.sum(1, keepdim=True)
    (gc, gs), (dc, ds) = s["gate_up"], s["down"]
    for e in range(E):
        t, j = torch.nonzero(chosen == e, as_tuple=True)
        if len(t) == 0:
            continue
        gu = x[t] @ _exact_planes(gc[2 * F * e:2 * F * (e + 1)], gs[:, 2 * F * e:2 * F * (e + 1)], D).T
        h = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
        y[t] += kept[t, j, None] * (h @ _exact_planes(dc[D * e:D * (e + 1)], ds[:, D * e:D * (e + 1)], F).T)
    return y
