"""The microscaled 4-bit operators and the expert layer from their definitions
in 64 bits on the CPU (torch double), sharing no code with the library."""

import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def e2m1_codes(v):
    """Nearest E2M1 code of each value, ties to the even code, saturated."""
    mid = (GRID[1:] + GRID[:-1]) / 2
    a = v.abs().contiguous()
    lo, hi = torch.searchsorted(mid, a, right=False), torch.searchsorted(mid, a, right=True)
    return torch.where(lo % 2 == 0, lo, hi) + 8 * torch.signbit(v)


def e2m1_values(codes):
    m = GRID[codes & 7]
    return torch.where(codes >= 8, -m, m)


def mx_encode(x):
    """(codes [rows, B, 32], scale bytes [rows, B]) of x along its rows, zero
    padded to whole blocks; B = ceil(K / 32)."""
    x = x.double().cpu()
    rows, K = x.shape
    B = -(-K // 32)
    b = torch.zeros((rows, B * 32), dtype=torch.float64)
    b[:, :K] = x
    b = b.reshape(rows, B, 32)
    bad = ~torch.isfinite(b).all(2)
    fine = torch.where(bad.unsqueeze(2), 0.0, b)
    amax = fine.abs().amax(2)
    e = torch.frexp(amax).exponent.long() - 1 - 2 + 127
    e = torch.where(amax > 0, e.clamp(0, 254), 0)
    codes = e2m1_codes(fine * torch.exp2(127.0 - e.double()).unsqueeze(2))
    return codes, torch.where(bad, 255, e)


def mx_values(codes, e, K):
    """float64 values of codes [rows, B, 32] and scale bytes [rows, B]."""
    s = torch.where(e == 255, torch.nan, torch.exp2(e.double() - 127))
    return (e2m1_values(codes) * s.unsqueeze(2)).flatten(1)[:, :K]


def quantized(x):
    """Values of x after microscaled quantisation along its rows."""
    return mx_values(*mx_encode(x), x.shape[1])


def planes(codes, e, K):
    """The arrays of a microscaled matrix: codes [rows, C * 128], scales [C, rows, 8]."""
    rows, B, _ = codes.shape
    C = -(-K // 256)
    full = torch.zeros((rows, C * 8, 32), dtype=torch.int64)
    full[:, :B] = codes
    full = full.reshape(rows, -1)
    s = torch.zeros((rows, C * 8), dtype=torch.int64)
    s[:, :B] = e
    return ((full[:, 0::2] | full[:, 1::2] << 4).to(torch.uint8),
            s.reshape(rows, C, 8).permute(1, 0, 2).contiguous().to(torch.uint8))


def random_planes(g, rows, K, lo=118, hi=124):
    """A random matrix as (codes plane, scales plane, float64 values)."""
    B = -(-K // 32)
    codes = torch.randint(0, 16, (rows, B * 32), generator=g)
    codes[:, K:] = 0
    codes = codes.reshape(rows, B, 32)
    e = torch.randint(lo, hi, (rows, B), generator=g)
    return (*planes(codes, e, K), mx_values(codes, e, K))


def mxfp4_bytes(codes, e):
    """Packed MXFP4 blocks [rows, B * 17]: scale byte, then (j, j + 16) nibbles."""
    by = (codes[:, :, :16] | codes[:, :, 16:] << 4)
    return torch.cat((e.unsqueeze(2), by), 2).flatten(1).to(torch.uint8)


E4M3 = torch.tensor([k * 2.0 ** -9 for k in range(8)]
                    + [(8 + k) * 2.0 ** (p - 3) for p in range(-6, 9) for k in range(8)][:-1], dtype=torch.float64)


def nvfp4_bytes(x):
    """Packed NVFP4 blocks [rows, K / 64 * 36] of finite x (or NaN scales)."""
    b = x.double().cpu().reshape(x.shape[0], -1, 16)
    bad = ~torch.isfinite(b).all(2)
    fine = torch.where(bad.unsqueeze(2), 0.0, b)
    amax = fine.abs().amax(2)
    mid6 = (E4M3[1:] + E4M3[:-1]) * 3
    lo, hi = torch.searchsorted(mid6, amax, right=False), torch.searchsorted(mid6, amax, right=True)
    i = torch.where(lo % 2 == 0, lo, hi)
    S = E4M3[i].unsqueeze(2)
    codes = e2m1_codes(fine / torch.where(S > 0, S, 1.0))
    codes = torch.where(S > 0, codes, codes & 8)
    i = torch.where(bad, 0x7F, i)
    by = codes[:, :, :8] | codes[:, :, 8:] << 4
    rows = x.shape[0]
    return torch.cat((i.reshape(rows, -1, 4), by.reshape(rows, -1, 32)), 2).flatten(1).to(torch.uint8), bad


def product_bound(A, B, K, out_ulp):
    """Largest error of a product taken as ceil(K / 64) scaled matrix
    instructions, each of which may drop what lies 2^-22 below the largest of
    its terms and its sum, and a rounding to the output's type. The result may
    also lose what is below F32's smallest subnormal."""
    S = A.abs() @ B.abs().T
    Y = A @ B.T
    return -(-K // 64) * 2.0 ** -22 * S + out_ulp * Y.abs() + 2.0 ** -149


OUT_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def moe(x, router, gate_up, down, k, renormalize):
    """(y, bound) of the expert layer; gate_up and down are float64 values. The
    bound follows a rounding of 2^-23 per F32 addition through the layer, and
    2^-15 for h in bf16 parts (two of 8 bits, the least that any type uses)."""
    x, router = x.double().cpu(), router.double().cpu()
    T, D = x.shape
    E, F = router.shape[0], down.shape[1]
    logits = x @ router.T
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices
    ids = order[:, :k]
    top = torch.gather(logits, 1, ids)
    w = torch.exp(top - top[:, :1])
    total = w.sum(1, keepdim=True) if renormalize else torch.exp(logits - top[:, :1]).sum(1, keepdim=True)
    p = w / total
    dl = (D + 2) * 2.0 ** -23 * (x.abs() @ router.abs().T).amax(1, keepdim=True)  # a logit's error
    y, bound = torch.zeros((T, D), dtype=torch.float64), torch.zeros((T, D), dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            gu = gate_up[e * 2 * F:(e + 1) * 2 * F]
            v, dv = gu @ x[t], (D + 8) * 2.0 ** -23 * (gu.abs() @ x[t].abs())
            gate, up, dg, du = v[:F], v[F:], dv[:F], dv[F:]
            silu = gate * torch.sigmoid(gate)
            h = silu * up
            dh = 1.1 * dg * (up.abs() + du) + silu.abs() * du + 2.0 ** -15 * h.abs() + 2.0 ** -20 * h.abs()
            wd = down[e * D:(e + 1) * D]
            out = wd @ h
            dout = wd.abs() @ dh + (F + 8) * 2.0 ** -23 * (wd.abs() @ h.abs())
            y[t] += p[t, j] * out
            bound[t] += p[t, j] * (dout + out.abs() * (4 * dl[t] + (E + 8) * 2.0 ** -22))
    return y, bound
