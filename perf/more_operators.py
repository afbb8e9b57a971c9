"""The operators over a model's vocabulary: cases, plain forms and the definition in 64 bits.

One table of V rows x K, of floats or of packed blocks, is a model's embedding and its output head:

embed  y[t] = scale * W[ids[t]]; an id outside 0 .. V-1 (padding) gives a row of zeros
grad   dW[v] = scale * sum of dy[t] over the t with ids[t] = v: the gradient of embed with respect to a float table
loss   l = x W^T, loss[t] = log sum_v exp l[t][v] - l[t][target[t]], without keeping l; a target outside 0 .. V-1 is
       a token that is not learnt from: its loss is 0. Returned with lse[t] = log sum_v exp l[t][v] (of every token)
step   loss and its gradient for given d loss[t]: dx = dl W and, where the table is trained, dW = dl^T x, with
       dl[t][v] = dloss[t] * (exp(l[t][v] - lse[t]) - [v = target[t]]), rows of zeros for tokens not learnt from

Packed tables are rows of GGUF blocks:
    q8_0  34 bytes / 32:   fp16 d, 32 int8 q; value d * q
    q4_k  144 bytes / 256: fp16 d, fp16 dmin, 12 bytes of eight 6-bit sub-scales and sub-mins, 128 bytes of nibbles
          (chunk c of 64 elements: 32 bytes, low nibbles sub-block 2c, high nibbles 2c + 1); (d * sc) * q - dmin * m
    q6_k  210 bytes / 256: 128 bytes of low nibbles, 64 bytes of 2-bit high parts, 16 int8 sub-scales, fp16 d
    mxfp4 17 bytes / 32:   scale byte e, 16 bytes of E2M1 nibbles (element j low nibble of byte j, j + 16 its high one)
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCKS = {"q8_0": (32, 34), "q4_k": (256, 144), "q6_k": (256, 210), "mxfp4": (32, 17)}
TYPE_IDS = {"f32": 0, "f16": 1, "bf16": 30, "q8_0": 8, "q4_k": 12, "q6_k": 14, "mxfp4": 39}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the token of one decoding step, from a packed table: latency
        dict(name="embed_t1_q8_0", op="embed", T=1, V=32768, K=4096, wtype="q8_0", dtype="bf16", scale=1.0),
        # the tokens of a training batch, float table, with the square root of the width as scale
        dict(name="embed_t16384_bf16", op="embed", T=16384, V=131072, K=4096, wtype="bf16", dtype="bf16", scale=64.0),
        # a ragged batch of prompts from a packed table into 32 bits
        dict(name="embed_t2741_q6_k", op="embed", T=2741, V=100003, K=5120, wtype="q6_k", dtype="f32", scale=1.0),
        # the table's gradient after a batch of text: few tokens make up most of it
        dict(name="grad_t16384_v131072", op="grad", T=16384, V=131072, K=4096, dtype="bf16", scale=64.0),
        # a short ragged batch of a narrow model, 32-bit gradients
        dict(name="grad_t777_v32000_f32", op="grad", T=777, V=32000, K=1000, dtype="f32", scale=1.0),
        # scoring one token: the head is read once
        dict(name="loss_t1_v32768", op="loss", T=1, V=32768, K=2048, wtype="bf16", dtype="bf16"),
        # scoring the next tokens of a batch of 16 sequences through a packed head
        dict(name="loss_t16_q4_k", op="loss", T=16, V=131072, K=4096, wtype="q4_k", dtype="bf16"),
        # perplexity of a ragged prompt in half precision
        dict(name="loss_t1021_f16", op="loss", T=1021, V=50001, K=2048, wtype="f16", dtype="f16"),
        # fine-tuning with a frozen packed head
        dict(name="step_t2048_q8_0", op="step", T=2048, V=131072, K=4096, wtype="q8_0", dtype="bf16", train=False),
        # a few tokens of one short sequence, frozen head
        dict(name="step_t64_bf16", op="step", T=64, V=32768, K=4096, wtype="bf16", dtype="bf16", train=False),
        # a 32-bit model, ragged, table trained
        dict(name="step_t999_f32", op="step", T=999, V=32000, K=2000, wtype="f32", dtype="f32", train=True),
        # training in bfloat16, table trained: the largest
        dict(name="step_t4096_bf16", op="step", T=4096, V=131072, K=4096, wtype="bf16", dtype="bf16", train=True),
    ]


def _size(rng, lo, hi, whole=32):
    """A size spread over its logarithm: one in three odd, the others of whole `whole`s where they are large enough."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 1 / 3 or n < 2 * whole:
        n |= 1
    else:
        n = n // whole * whole
    return min(max(n, lo), hi)


def draw(rng):
    while True:
        op = rng.choice(("embed", "grad", "loss", "step"))
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        wtype = rng.choice((dtype, dtype, "q8_0", "q4_k", "q6_k", "mxfp4"))
        K, V = _size(rng, 256, 8192), _size(rng, 1000, 131072, 256)
        if wtype in BLOCKS:
            K = K // BLOCKS[wtype][0] * BLOCKS[wtype][0]
        c = dict(op=op, T=_size(rng, 1, 16384 if op in ("embed", "grad") else 4096), V=V, K=K)
        if op == "grad":
            c.update(dtype=dtype, scale=rng.choice((1.0, 0.5, math.sqrt(K))))
        else:
            c.update(wtype=wtype, dtype=dtype)
        if op == "embed":
            c["scale"] = rng.choice((1.0, 0.5, math.sqrt(K)))
        if op == "step":
            c["train"] = wtype == dtype and rng.random() < 0.5
        w = work(c)
        # 32-bit products cost what six of 16 bits do
        if w["bytes"] <= 1.1e9 * (2 if op in ("grad", "step") else 1) and w["flops"] * (6 if dtype == "f32" else 1) <= 1.3e13:
            return c


# ---------------------------------------------------------------- inputs

def _table(g, V, K, wtype):
    """A table whose values are about 0.02 wide: floats V x K, or the packed rows' bytes V x row bytes."""
    if wtype not in BLOCKS:
        return (torch.randn((V, K), generator=g, device="cuda") * 0.02).to(DTYPES[wtype])
    block, size = BLOCKS[wtype]
    b = torch.randint(0, 256, (V, K // block, size), generator=g, device="cuda", dtype=torch.uint8)
    d = torch.rand((V, K // block, 2), generator=g, device="cuda") + 0.5
    if wtype == "q8_0":
        b[..., :2] = (d[..., :1] * 2.7e-4).half().view(torch.uint8)
    elif wtype == "q4_k":  # the sub-mins at 31.5 * dmin meet the codes' middle, 7.5 * 31.5 * d
        b[..., :4] = (d * torch.tensor((1.0e-4, 7.5e-4), device="cuda")).half().view(torch.uint8)
    elif wtype == "q6_k":
        b[..., 208:] = (d[..., :1] * 1.5e-5).half().view(torch.uint8)
    else:
        b[..., 0] = 118 + (b[..., 0] & 1)
    return b.flatten(1)


def _tokens(g, T, V, none):
    """Token ids of text: the frequent ones are few. A share `none` of them is no token (-1)."""
    ids = (V ** torch.rand(T, generator=g, device="cuda", dtype=torch.float64)).long() - 1
    # frequent ids lie anywhere in the table
    ids = (ids.clamp(0, V - 1) * 40503 + 977) % V
    return torch.where(torch.rand(T, generator=g, device="cuda") < none, -1, ids)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 2654435761 % (1 << 62))
    s = dict(case)
    op, T, V, K, dtype = case["op"], case["T"], case["V"], case["K"], DTYPES[case["dtype"]]
    if op in ("embed", "grad"):
        s["ids"] = _tokens(g, T, V, 1 / 16 if T > 4 else 0)
        if op == "embed":
            s["w"] = _table(g, V, K, case["wtype"])
        else:
            s["dy"] = (torch.randn((T, K), generator=g, device="cuda") * 1e-2).to(dtype)
        return s
    s["w"] = _table(g, V, K, case["wtype"])
    s["targets"] = _tokens(g, T, V, 1 / 8 if T > 4 else 0)
    # hidden states behind a norm, turned towards their targets as a trained model's are
    rows = s["w"][s["targets"].clamp(min=0)]
    rows = rows.float() if case["wtype"] not in BLOCKS else _decode(rows, case["wtype"])
    s["x"] = (torch.randn((T, K), generator=g, device="cuda")
              + rows * (12000.0 / K * torch.rand((T, 1), generator=g, device="cuda"))).to(dtype)
    # the mean over the batch; half precision with the scale that its training gives the loss
    s["dloss"] = torch.full((T,), (1024.0 if case["dtype"] == "f16" else 1.0) / T, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms (32 bits)

def _decode(b, wtype):
    """Values of packed rows (float32, rows x K)."""
    block, size = BLOCKS[wtype]
    b = b.reshape(b.shape[0], -1, size)
    half = lambda at: b[..., at:at + 2].contiguous().view(torch.float16).float()  # noqa: E731
    if wtype == "q8_0":
        return (half(0) * b[..., 2:].contiguous().view(torch.int8).float()).flatten(1)
    if wtype == "mxfp4":
        grid = torch.tensor(E2M1, device=b.device)
        scale = (b[..., :1].int() << 23).view(torch.float32)
        return (torch.cat((grid[(b[..., 1:] & 15).int()], grid[(b[..., 1:] >> 4).int()]), -1) * scale).flatten(1)
    if wtype == "q4_k":
        f = b[..., 4:16].int()
        low, mid, high = f[..., :4], f[..., 4:8], f[..., 8:]
        sc = torch.cat((low & 63, (high & 15) | ((low >> 6) << 4)), -1).float() * half(0)
        m = torch.cat((mid & 63, (high >> 4) | ((mid >> 6) << 4)), -1).float() * half(2)
        q = b[..., 16:].unflatten(-1, (4, 32))
        q = torch.stack((q & 15, q >> 4), -2).flatten(-3, -2).float()
        return (q * sc.unsqueeze(-1) - m.unsqueeze(-1)).flatten(1)
    ql, qh = b[..., :128].unflatten(-1, (2, 2, 32)), b[..., 128:192].unflatten(-1, (2, 32))
    low = torch.stack((ql & 15, ql >> 4), -3).flatten(-3, -2)  # half, part, 32
    two = torch.stack([(qh >> (2 * p)) & 3 for p in range(4)], -2)
    q = (low | (two << 4)).flatten(-3).float() - 32.0
    sc = b[..., 192:208].contiguous().view(torch.int8).float() * half(208)
    return (q.unflatten(-1, (16, 16)) * sc.unsqueeze(-1)).flatten(1)


def _values(s, rows=slice(None)):
    return _decode(s["w"][rows], s["wtype"]) if s["wtype"] in BLOCKS else s["w"][rows].float()


def _plain_embed(s):
    ids = s["ids"]
    known = (ids >= 0) & (ids < s["V"])
    y = _values(s, torch.where(known, ids, 0)) * s["scale"]
    return torch.where(known.unsqueeze(1), y, 0.0).to(DTYPES[s["dtype"]])


def _plain_grad(s):
    ids = s["ids"]
    known = (ids >= 0) & (ids < s["V"])
    dw = torch.zeros((s["V"] + 1, s["K"]), device=ids.device)
    dw.index_add_(0, torch.where(known, ids, s["V"]), s["dy"].float())
    return dw[:-1] * s["scale"]


def _plain_loss(s):
    """(loss, lse, l - its row's largest, that, whether a token is learnt from)"""
    y = s["targets"]
    learnt = (y >= 0) & (y < s["V"])
    w = _values(s)
    l = s["x"].float() @ w.T
    top = l.amax(1, keepdim=True)
    l -= top
    lse = torch.log(torch.exp(l).sum(1)) + top[:, 0]
    at = torch.gather(l, 1, torch.where(learnt, y, 0).unsqueeze(1))[:, 0]
    return torch.where(learnt, lse - top[:, 0] - at, 0.0), lse, w, l, top, learnt


def _plain_step(s):
    loss, lse, w, l, top, learnt = _plain_loss(s)
    l += (top[:, 0] - lse).unsqueeze(1)
    p = torch.exp_(l)
    p[torch.arange(s["T"], device=p.device), torch.where(learnt, s["targets"], 0)] -= 1.0
    p *= torch.where(learnt, s["dloss"], 0.0).unsqueeze(1)
    dtype = DTYPES[s["dtype"]]
    dx = (p @ w).to(dtype)
    return (loss, dx, (p.T @ s["x"].float()).to(dtype)) if s["train"] else (loss, dx)


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["op"]
    if not own:
        if op == "loss":
            return _plain_loss(state)[:2]
        return {"embed": _plain_embed, "grad": _plain_grad, "step": _plain_step}[op](state)
    import quantized_weight_backward_amd as q

    if op == "grad":
        return q.embedding_backward(state["ids"], state["dy"], state["V"], scale=state["scale"])
    wtype = TYPE_IDS[state["wtype"]]
    if op == "embed":
        return q.embedding(wtype, state["w"], state["ids"], state["K"], scale=state["scale"], dtype=DTYPES[state["dtype"]])
    loss, lse = q.cross_entropy(wtype, state["w"], state["x"], state["targets"])
    if op == "loss":
        return loss, lse
    dx, dw = q.cross_entropy_backward(wtype, state["w"], state["x"], state["targets"], lse, state["dloss"],
                                      weight_grad=state["train"])
    return (loss, dx, dw) if state["train"] else (loss, dx)


def work(case):
    """Bytes: each input read and each output written once. The logits' product counts once, each gradient's once."""
    T, V, K = case["T"], case["V"], case["K"]
    size = {"f32": 4, "f16": 2, "bf16": 2}
    row = size[case["dtype"]] * K
    if case["op"] == "grad":
        return {"bytes": T * (row + 8) + 4 * V * K, "flops": T * K}
    wtype = case["wtype"]
    w_row = K // BLOCKS[wtype][0] * BLOCKS[wtype][1] if wtype in BLOCKS else size[wtype] * K
    if case["op"] == "embed":
        return {"bytes": T * (w_row + row + 8), "flops": T * K}
    if case["op"] == "loss":
        return {"bytes": V * w_row + T * (row + 16), "flops": 2 * T * V * K}
    train = case["train"]
    return {"bytes": V * w_row * (2 if train else 1) + T * (2 * row + 20), "flops": 2 * T * V * K * (3 if train else 2)}


# ---------------------------------------------------------------- the definition, in 64 bits

def _exact_rows(b, wtype):
    """Values of packed rows by the blocks' definition, element by element of a block (float64)."""
    if wtype not in BLOCKS:
        return b.double()
    block, size = BLOCKS[wtype]
    b = b.reshape(b.shape[0], -1, size)
    out = torch.empty((*b.shape[:2], block), dtype=torch.float64, device=b.device)
    f16 = lambda at: (b[..., at].int() | (b[..., at + 1].int() << 8)).short().view(torch.float16).double()  # noqa: E731
    i8 = lambda at: (b[..., at].int() ^ 128).double() - 128  # noqa: E731
    for i in range(block):
        if wtype == "q8_0":
            out[..., i] = f16(0) * i8(2 + i)
        elif wtype == "mxfp4":
            code = (b[..., 1 + i % 16] >> (4 * (i // 16))) & 15
            mag = (code & 7).double()
            mag = torch.where(mag < 2, mag / 2, (2 + mag % 2) * torch.exp2(torch.floor(mag / 2) - 2))
            out[..., i] = torch.where(code >= 8, -mag, mag) * torch.exp2(b[..., 0].double() - 127)
        elif wtype == "q4_k":
            j = i // 32
            if j < 4:
                sc, m = b[..., 4 + j] & 63, b[..., 8 + j] & 63
            else:
                sc = (b[..., 8 + j] & 15) + (b[..., j] >> 6) * 16
                m = (b[..., 8 + j] >> 4) + (b[..., 4 + j] >> 6) * 16
            code = (b[..., 16 + 32 * (i // 64) + i % 32] >> (4 * (j % 2))) & 15
            out[..., i] = f16(0) * sc.double() * code.double() - f16(2) * m.double()
        else:
            h, p, l = i // 128, i // 32 % 4, i % 32
            low = (b[..., 64 * h + 32 * (p % 2) + l] >> (4 * (p // 2))) & 15
            high = (b[..., 128 + 32 * h + l] >> (2 * p)) & 3
            out[..., i] = f16(208) * i8(192 + 8 * h + 2 * p + l // 16) * (low.double() + 16 * high.double() - 32)
    return out.reshape(b.shape[0], -1)


def exact(case, seed):
    s = prepare(case, seed)
    op, T, V = case["op"], case["T"], case["V"]
    if op == "embed":
        y = torch.zeros((T, case["K"]), dtype=torch.float64, device="cuda")
        t = torch.nonzero(s["ids"] >= 0)[:, 0]
        y[t] = _exact_rows(s["w"][s["ids"][t]], case["wtype"]) * case["scale"]
        return y
    if op == "grad":
        t = torch.nonzero(s["ids"] >= 0)[:, 0]
        dw = torch.zeros((V, case["K"]), dtype=torch.float64, device="cuda")
        return dw.index_put_((s["ids"][t],), s["dy"][t].double() * case["scale"], accumulate=True)
    # in pieces of the tokens: 64-bit logits of all of them need not fit
    w, pieces, dw = _exact_rows(s["w"], case["wtype"]), [], None
    for t in torch.arange(T, device="cuda").split(1024):
        x, y = s["x"][t].double(), s["targets"][t]
        l = torch.mm(x, w.T)
        lse = torch.logsumexp(l, 1)
        learnt = y >= 0
        at = l[torch.arange(len(t), device="cuda"), y.clamp(min=0)]
        loss = torch.where(learnt, lse - at, 0.0)
        if op == "loss":
            pieces.append((loss, lse))
            continue
        p = torch.softmax(l, 1).index_put_((torch.nonzero(learnt)[:, 0], y[learnt]),
                                           torch.tensor(-1.0, dtype=torch.float64, device="cuda"), accumulate=True)
        p = p * (s["dloss"][t].double() * learnt).unsqueeze(1)
        pieces.append((loss, torch.mm(p, w)))
        if case["train"]:
            dw = torch.mm(p.T, x) if dw is None else dw.addmm_(p.T, x)
    out = tuple(torch.cat(v) for v in zip(*pieces))
    return out if dw is None else (*out, dw)
