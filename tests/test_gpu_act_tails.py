"""The activations of the linear layer and the experts' GELU where their result is
small: relative to it, point by point.

z is exact (one bf16 value times one). Tolerance: one rounding to bf16 (2^-8 of the
value) and the relative error of sigmoid(x) = 1 / (1 + e^-x) in fp32, from the
hardware's exponential and reciprocal (2^-22 and 2^-23 of their results): the
exponent's four roundings move the exponential by 4 |x| 2^-24, the sum and the
products add two: at most (8 + 6 |x|) 2^-24."""
import math

import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
C = math.sqrt(2 / math.pi)


def formula(act, z):
    """(act(z), act'(z), the sum of magnitudes in act'(z), x) with x the sigmoid's
    argument; fp64."""
    x = 2 * C * (z + 0.044715 * z ** 3) if act.startswith("g") else z
    s = 1 / (1 + torch.exp(-x))
    slope = s * (1 - s)
    if act == "sigmoid":
        return s, slope, slope, x
    bend = z * slope * (2 * C * (1 + 3 * 0.044715 * z * z) if act.startswith("g") else 1)
    return z * s, s + bend, s + bend.abs(), x


def points(lo, n):
    z = -torch.logspace(-3, math.log10(-lo), n, dtype=torch.float64, device="cuda")
    return z.to(BF)


@pytest.mark.parametrize("act,lo", [("gelu_tanh_approx", -8.0), ("silu", -40.0),
                                    ("sigmoid", -40.0)])
@pytest.mark.parametrize("M,policy", [(8, 0), (200, 0), (200, 1), (3000, 2)])
def test_linear(act, lo, M, policy):
    z = points(lo, M)
    x, W = torch.zeros((M, 8), dtype=BF, device="cuda"), torch.zeros((8, 8), dtype=BF, device="cuda")
    x[:, 0], W[:, 0] = z, 1
    p = m.linear(M, 8, 8, act)
    out, pre, dx = (torch.empty((M, 8), dtype=BF, device="cuda") for _ in range(3))
    dout = torch.zeros_like(out)
    dout[:, 0] = 1
    m.mlp_set_tile_policy(policy)
    try:
        m.mlp_linear_fwd(p, x, W, None, None, out, pre)
        m.mlp_linear_bwd(p, dout, x, W, pre, dx=dx)
    finally:
        m.mlp_set_tile_policy(0)
    assert torch.equal(pre[:, 0], z)
    a, da, mag, arg = formula(act, z.double())
    rel = (8 + 6 * arg.abs()) * 2.0 ** -24
    off = (out.double() - a[:, None]).abs()
    assert (off <= ((2.0 ** -8 + rel) * a.abs() + 1e-37)[:, None]).all()
    off = (dx[:, 0].double() - da).abs()
    assert (off <= 2.0 ** -8 * da.abs() + rel * mag + 1e-37).all()


@pytest.mark.parametrize("act", ["geglu", "gelu_tanh_approx"])
@pytest.mark.parametrize("T", [6, 50, 700])
def test_experts(act, T):
    z = points(-8.0, T)
    x = torch.zeros((T, 8), dtype=BF, device="cuda")
    x[:, 0], x[:, 1] = z, 1
    W1, Wu = torch.zeros((2, 8, 8), dtype=BF, device="cuda"), None
    W1[:, :, 0] = 1
    if act == "geglu":
        Wu = torch.zeros_like(W1)
        Wu[:, :, 1] = 1
    Wd = torch.eye(8, device="cuda").to(BF).expand(2, 8, 8).contiguous()
    p = m.moe(T, 2, 1, 8, 8, act)
    ids = (torch.arange(T, device="cuda") % 2).int().view(T, 1)
    out, w = torch.empty_like(x), torch.ones((T, 1), device="cuda")
    m.mlp_moe_fwd_infer(p, x, ids, w, W1, Wu, Wd, None, out)
    a, da, mag, arg = formula(act, z.double())
    rel = (8 + 6 * arg.abs()) * 2.0 ** -24
    assert ((out.double() - a[:, None]).abs() <= ((2.0 ** -8 + rel) * a.abs() + 1e-37)[:, None]).all()
    # dg in place of the saved preact, for a gradient of one at the first feature
    rows = m.mlp_moe_rows(p)
    plan = m.alloc_moe_plan(p)
    m.mlp_moe_sort(p, ids, plan)
    new = lambda: torch.zeros((rows, 8), dtype=BF, device="cuda")  # noqa: E731
    xs, y, G, U, dy, dxs = new(), new(), new(), (new() if Wu is not None else None), new(), new()
    m.mlp_moe_dispatch(p, plan, x, xs)
    m.mlp_moe_experts_fwd(p, plan, xs, W1, Wu, Wd, y, G, U)
    dout = torch.zeros_like(x)
    dout[:, 0] = 1
    m.mlp_moe_combine_bwd(p, plan, dout, None, w, dy, None)
    m.mlp_moe_experts_bwd(p, plan, dy, xs, W1, Wu, Wd, G, U, dxs=dxs)
    dg = G[m.moe_plan_views(p, plan)["pos"].view(-1).long(), 0].double()
    assert ((dg - da).abs() <= 2.0 ** -8 * da.abs() + rel * mag + 1e-37).all()
