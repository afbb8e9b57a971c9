"""A linear layer trained through 4-bit products, then served with an expert layer.

    python examples/microscaled_layers.py

Training: the F32 master weight is quantised along both axes after each update;
the forward product, the input gradient and the weight gradient all contract
4-bit operands. Serving: the trained weight as packed MXFP4 blocks, laid out once
for the products, takes single tokens; a mixture-of-experts layer over 4-bit
experts takes a few. Needs an MI355X.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_weight_backward_amd as q  # noqa: E402


def train(T=512, K=256, N=384, steps=60, lr=0.5, seed=0):
    """Fits w to a target's outputs; returns the losses and the master weight."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    target = torch.randn((N, K), generator=g, device="cuda") / K ** 0.5
    w = torch.zeros((N, K), device="cuda")
    losses = []
    for _ in range(steps):
        x = torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16)
        w_rows, w_cols = q.mx_quantize_both(w)  # w along k for the product, w^T along n for the gradient
        y = q.mx_linear(x, w_rows)
        error = y.float() - x.float() @ target.T
        losses.append(float(error.square().mean()))
        dx, dw = q.mx_linear_backward((error / T).to(torch.bfloat16), x, w_cols)
        assert dx.shape == x.shape  # for the layer before this one
        w -= lr * dw
    return losses, w


def serve(w, seed=1):
    """One token through the packed weight, and a few through an expert layer."""
    N, K = w.shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    packed = q.quantize(q.MXFP4, w)              # resident blocks, as out_prod and mul_mat take them
    ready = q.mx_from_blocks(packed, K, N)       # laid out once for the 4-bit products
    token = torch.randn((1, K), generator=g, device="cuda").to(torch.bfloat16)
    y = q.mx_linear(token, ready)

    E, F, T, top_k = 8, 128, 4, 2
    router = torch.randn((E, K), generator=g, device="cuda") / K ** 0.5
    gate_up = q.mx_quantize(torch.randn((E * 2 * F, K), generator=g, device="cuda") / K ** 0.5)
    down = q.mx_quantize(torch.randn((E * K, F), generator=g, device="cuda") / F ** 0.5)
    tokens = torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16)
    return y, q.mx_moe(tokens, router, gate_up, down, top_k)


def main():
    losses, w = train()
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps of 4-bit products")
    y, z = serve(w)
    print(f"one token: {tuple(y.shape)}, expert layer: {tuple(z.shape)}, all finite: "
          f"{bool(y.isfinite().all() and z.isfinite().all())}")


if __name__ == "__main__":
    main()
