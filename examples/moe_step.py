"""Training steps of a transformer's feed-forward block with routed experts, its norm
and balance loss inside, and its matrices moved along orthogonalised momenta:

    norm     h = LayerNorm(x)                           (layer_norm_func)
    router   logits = h Wr^T; ids, weights, balance     (linear_func, router_func)
    experts  y = x + sum_j weights_j MLP_{ids_j}(h)     (moe_func, residual inside)
    update   M = beta M + dW;  W -= lr c NS(M)          (mlp_orthogonalize; a stack of
             c = sqrt(max(1, rows / cols))               experts in one call)

The norm's weight and bias, which are vectors, take plain momentum.

    python examples/moe_step.py [--tokens 512] [--steps 20]
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import activated_mlp_gemms_gb300 as m  # noqa: E402

BF = torch.bfloat16


def make_params(H=256, inner=352, E=8, device="cuda", seed=0):
    """bf16 matrices (nn.Linear's uniform initialisation) and the norm's fp32 vectors."""
    gen = torch.Generator(device=device).manual_seed(seed)

    def uni(fan_in, *shape):
        t = torch.rand(shape, generator=gen, device=device) * 2 - 1
        return (t / math.sqrt(fan_in)).to(BF).requires_grad_(True)

    return {"norm_w": torch.ones(H, device=device, requires_grad=True),
            "norm_b": torch.zeros(H, device=device, requires_grad=True),
            "Wr": uni(H, E, H), "Wg": uni(H, E, inner, H), "Wu": uni(H, E, inner, H),
            "Wd": uni(inner, E, H, inner)}


def block(x, p, top_k=2, mask=None):
    """(the block's output for x [tokens, H], the balance loss, the experts' slots); mask
    [tokens] is false for padding, which passes through."""
    h = m.layer_norm_func(x, p["norm_w"], p["norm_b"])
    logits = m.linear_func(h, p["Wr"])
    ids, weights, counts, balance = m.router_func(logits, top_k, mask)
    y = m.moe_func(h, ids, weights, p["Wg"], p["Wu"], p["Wd"], "swiglu", residual=x)
    return y, balance, counts


def update(w, momentum, grad, lr, beta=0.9):
    """One step of w (in place); momentum is fp32 of its shape."""
    momentum.mul_(beta).add_(grad)
    if w.dim() == 1:
        w.sub_(lr * momentum)
        return
    rows, cols = w.shape[-2:]
    p = m.ortho(rows, cols, w.numel() // (rows * cols), scale=math.sqrt(max(1, rows / cols)),
                dtype=torch.float32)
    step = torch.empty_like(w)
    shape = (p.batch, rows, cols)
    m.mlp_orthogonalize(p, momentum.view(shape), step.view(shape))
    w.copy_(w.float() - lr * step.float())


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.02)
    a = ap.parse_args()
    params = make_params()
    momenta = {k: torch.zeros_like(v, dtype=torch.float32) for k, v in params.items()}
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((a.tokens, 256), generator=gen, device="cuda").to(BF)
    target = x.float() + torch.tanh(x.float().roll(1, -1))
    losses = []
    for step in range(a.steps):
        y, balance, counts = block(x, params)
        loss = (y.float() - target).square().mean() + 0.01 * balance
        grads = torch.autograd.grad(loss, list(params.values()))
        with torch.no_grad():
            for (k, w), g in zip(params.items(), grads):
                update(w, momenta[k], g, a.lr)
        losses.append(loss.item())
        if step % 5 == 0 or step == a.steps - 1:
            print(f"step {step:3d}  loss {losses[-1]:.4f}  slots {counts.tolist()}")
    return losses


if __name__ == "__main__":
    main()
