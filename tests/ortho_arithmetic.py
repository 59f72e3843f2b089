"""The orthogonalised update's arithmetic (include/mlp_ortho.h) on the CPU, for the bounds of the
tests: fp16 terms at their powers of two, and sums as the tensor cores add them, truncated to 24
bits after every 16 products."""
import math

import torch

MUON = (3.4445, -4.7750, 2.0315)
X_SCALE, A_SCALE = 16384.0, 8192.0


def plain(G, steps=5):
    """The formula in 64 bits (one matrix)."""
    a, b, c = MUON
    X = G.double()
    X = X / (X.norm() + 1e-7)
    tall = X.shape[0] > X.shape[1]
    X = X.t() if tall else X
    for _ in range(steps):
        A = X @ X.t()
        X = a * X + (b * A + c * A @ A) @ X
    return X.t() if tall else X


def off(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def momentum(M, N, gen, device="cpu"):
    """A few strong directions over noise, as momenta are."""
    rn = lambda *s: torch.randn(s, generator=gen, device=device, dtype=torch.float64)  # noqa: E731
    r = max(1, min(M, N) // 8)
    scale = torch.logspace(0, -1.5, r, device=device, dtype=torch.float64)
    return (1e-3 * ((rn(M, r) * scale) @ rn(r, N) / math.sqrt(r) + 0.3 * rn(M, N))).float()


def _fp32(v):
    return v.float().double()


def _terms(v):
    hi = v.float().half().double()
    return hi, (v - hi).float().half().double()


def _truncate(v):
    m, e = torch.frexp(v)
    return torch.ldexp(torch.trunc(m * 2.0 ** 24), e - 24)


def _product(P, Q, both, chunk):
    """The leading terms' product in chunks of `chunk`, rounded to nearest where they are added
    up; with `both` the small products first."""
    acc = torch.zeros(P[0].shape[0], Q[0].shape[1], dtype=torch.float64)

    def add(acc, p, q):
        for k in range(0, p.shape[1], 16):
            acc = _truncate(acc + p[:, k:k + 16] @ q[k:k + 16])
        return acc

    if both:
        acc = add(add(acc, P[0], Q[1]), P[1], Q[0])
    total = None
    for k in range(0, P[0].shape[1], chunk):
        acc = add(acc, P[0][:, k:k + chunk], Q[0][k:k + chunk])
        total = acc if total is None else _fp32(total + acc)
        acc = torch.zeros_like(acc)
    return total


def emulate(G, fp32, px_both, both=True, steps=5):
    """The result for G [m, n], m <= n: fp32, or bf16 whose P X takes both terms or the leading
    ones; both=False: an fp32 result without its small products (a mistake)."""
    a, b, c = MUON
    X = _terms(_fp32(X_SCALE * G.double() / (G.double().norm() + 1e-7)))
    whole = 1 << 30
    both = both and fp32
    for s in range(steps):
        A = _terms(_fp32(_product(X, (X[0].t(), X[1].t()), both, 256 if fp32 else whole)
                         * (A_SCALE / X_SCALE / X_SCALE)))
        if not fp32:
            A = (A[0], torch.zeros_like(A[1]))
        P = _terms(_fp32(c / A_SCALE * _product(A, A, both, 256 if fp32 else whole)
                         + b * (A[0] + A[1])))
        v = _product(P, X, both if fp32 else px_both, 512 if fp32 else whole) / A_SCALE
        v = _fp32(v + a * (X[0] + X[1]))
        X = _terms(v)
    v = _fp32(v / X_SCALE)
    return v if fp32 else v.bfloat16().double()
