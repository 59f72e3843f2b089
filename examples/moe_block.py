"""A transformer's feed-forward block with routed experts and a shared biased MLP,
trained for a few steps and then run token by token:

    router   logits = x Wr^T + br                      (linear_func)
             the top_k experts of a token, their softmax weights
    experts  r = x + sum_j w_j MLP_{id_j}(x)           (moe_func, residual inside)
    shared   out = r + W2 gelu(W1 r + b1) + b2         (linear_func twice)

    python examples/moe_block.py [--tokens 512] [--steps 20]
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
    """bf16 parameters of the block, nn.Linear's uniform initialisation."""
    gen = torch.Generator(device=device).manual_seed(seed)

    def uni(fan_in, *shape):
        t = torch.rand(shape, generator=gen, device=device) * 2 - 1
        return (t / math.sqrt(fan_in)).to(BF).requires_grad_(True)

    return {"Wr": uni(H, E, H), "br": uni(H, E), "Wg": uni(H, E, inner, H),
            "Wu": uni(H, E, inner, H), "Wd": uni(inner, E, H, inner), "W1": uni(H, inner, H),
            "b1": uni(H, inner), "W2": uni(inner, H, inner), "b2": uni(inner, H)}


def block(x, p, top_k=2):
    """The block's output for x [tokens, H]."""
    logits = m.linear_func(x, p["Wr"], p["br"]).float()
    top, ids = torch.topk(logits, top_k, dim=-1)
    weights = torch.softmax(top, -1)
    r = m.moe_func(x, ids.int(), weights, p["Wg"], p["Wu"], p["Wd"], "swiglu", residual=x)
    h = m.linear_func(r, p["W1"], p["b1"], activation="gelu_tanh_approx")
    return m.linear_func(h, p["W2"], p["b2"], residual=r)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.01)
    a = ap.parse_args()
    params = make_params()
    masters = {k: v.detach().float() for k, v in params.items()}
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((a.tokens, 256), generator=gen, device="cuda").to(BF)
    target = torch.tanh(x.float().roll(1, -1))
    losses = []
    for step in range(a.steps):
        loss = (block(x, params).float() - target).square().mean()
        grads = torch.autograd.grad(loss * a.tokens, list(params.values()))
        with torch.no_grad():
            for (k, p), g in zip(params.items(), grads):
                masters[k] -= a.lr * g.float()
                p.copy_(masters[k])
        losses.append(loss.item())
        if step % 5 == 0 or step == a.steps - 1:
            print(f"step {step:3d}  loss {losses[-1]:.4f}")
    with torch.no_grad():  # the same block one token at a time: the serving kernels
        whole = block(x[:4], params)
        single = torch.cat([block(x[i:i + 1], params) for i in range(4)])
        print(f"one token at a time: {(whole.float() - single.float()).abs().max().item():.3g} "
              f"off, of {whole.float().abs().max().item():.3g}")
    return losses


if __name__ == "__main__":
    main()
