"""The routing weights' gradient of a training step of few slots, against the formula
in fp64.

dweights[t, j] = <dout[t], y> sums H products of random signs, and a handful of slots
does not average the rounding of what it is formed from.  Tolerance, element by
element: one rounding of the result (u: 2^-8 for bf16, 2^-24 for fp32) and what fp32
leaves in y.  With h held as two bf16 terms (2^-16 of itself), the activation's own
error OWN (act.cuh) of max(1, |z|), and sums of n products in fp32 (which err by
(4 sqrt(n) + n / 4) 2^-24 of the products' root sum of squares): 4 times the root sum
of squares of those errors, as in the experts' tests."""
import math

import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
OWN = 2e-5


def act_ref(name, z):
    if name == "relu_sq":
        return torch.relu(z) ** 2
    if name == "swiglu":
        return z * torch.sigmoid(z)
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def rss(a, b):
    return ((a * a) @ (b * b)).sqrt()


def sums(n):
    return (4 * math.sqrt(n) + n / 4) * 2.0 ** -24


def y_ref(x, Wg, Wu, Wd, act):
    """An expert's result and the bound of its error in fp32."""
    H, inner = x.shape[1], Wg.shape[0]
    g, eg = x @ Wg.t(), sums(H) * rss(x, Wg.t())
    z = g.detach().requires_grad_(True)
    (da,) = torch.autograd.grad(act_ref(act, z).sum(), z)
    a, ea = act_ref(act, g), (da.abs() + 2 * eg) * eg + OWN * g.abs().clamp(min=1)
    u, eu = torch.ones_like(g), torch.zeros_like(g)
    if Wu is not None:
        u, eu = x @ Wu.t(), sums(H) * rss(x, Wu.t())
    h = a * u
    eh = ea * u.abs() + a.abs() * eu + ea * eu + 2.0 ** -16 * h.abs()
    y = h @ Wd.t()
    return y, 4 * rss(eh, Wd.t()) + sums(2 * inner) * rss(h, Wd.t())


def step(T, k, E, H, inner, act, wdt, seed, drop=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    p = m.moe(T, E, k, H, inner, act, weights_dtype=wdt)
    x, dout = rn(T, H).to(BF), rn(T, H).to(BF)
    Wg = (rn(E, inner, H) / math.sqrt(H)).to(BF)
    Wu = (rn(E, inner, H) / math.sqrt(H)).to(BF) if act in m.GATED_ACTS else None
    Wd = (rn(E, H, inner) / math.sqrt(inner)).to(BF)
    ids = torch.rand((T, E), generator=gen, device="cuda").topk(k, -1)[1].int()
    ids[torch.rand((T, k), generator=gen, device="cuda") < drop] = -1
    w = torch.rand((T, k), generator=gen, device="cuda").to(wdt)
    new = lambda *s: torch.full(s, float("nan"), dtype=BF, device="cuda")  # noqa: E731
    rows = m.mlp_moe_rows(p)
    plan = m.alloc_moe_plan(p)
    m.mlp_moe_sort(p, ids, plan)
    xs, y, G = new(rows, H), new(rows, H), new(rows, inner)
    U = new(rows, inner) if Wu is not None else None
    m.mlp_moe_dispatch(p, plan, x, xs)
    ws = m.mlp_moe_experts_fwd(p, plan, xs, Wg, Wu, Wd, y, G, U)
    assert m.mlp_device_status(ws) == 0
    dw = torch.full((T, k), float("nan"), dtype=wdt, device="cuda")
    m.mlp_moe_combine_bwd(p, plan, dout, y, w, None, dw)
    ref = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(ref)
    f = lambda t, e: None if t is None else t[e].double()  # noqa: E731
    for e in ids.unique().tolist():
        if e < 0:
            continue
        t, j = torch.nonzero(ids == e, as_tuple=True)
        yr, ey = y_ref(x[t].double(), f(Wg, e), f(Wu, e), f(Wd, e), act)
        d = dout[t].double()
        ref[t, j] = (d * yr).sum(1)
        tol[t, j] = 4 * (d * ey).norm(dim=1) + sums(H) * (d * yr).norm(dim=1)
    unit = 2.0 ** -8 if wdt == BF else 2.0 ** -24
    tol += unit * ref.abs() + 1e-12
    return p, plan, (x, xs, Wg, Wu, Wd, y, w, dout), dw, ref, tol


@pytest.mark.parametrize("act", ["swiglu", "relu_sq", "geglu"])
@pytest.mark.parametrize("T,k,E,H,inner", [
    (1, 1, 8, 384, 264), (1, 3, 4, 1384, 1384), (4, 3, 4, 264, 512), (7, 1, 1, 520, 136),
    (19, 2, 60, 256, 392), (5, 8, 16, 768, 72), (64, 1, 3, 136, 264), (2, 2, 2, 72, 8),
    (3, 2, 4, 72, 520), (2, 8, 16, 8, 520)])
def test_dweights_of_few_slots(T, k, E, H, inner, act):
    for seed in range(12):
        wdt = torch.float32 if seed % 2 else BF
        _, _, _, dw, ref, tol = step(T, k, E, H, inner, act, wdt, seed, 0.2 if seed % 3 == 2 else 0)
        off = (dw.double() - ref).abs()
        assert (off <= tol).all(), (seed, float((off / tol).max()), float(off.norm() / ref.norm()))


def test_another_y_is_taken_as_given():
    # the plan's fp32 values stand for the y that rounds to them only
    p, plan, (x, xs, Wg, Wu, Wd, y, w, dout), dw, _, _ = step(6, 2, 4, 264, 136, "swiglu",
                                                              torch.float32, 3)
    ids = m.moe_plan_views(p, plan)["pos"].long()
    gen = torch.Generator(device="cuda").manual_seed(9)
    other = torch.randn(y.shape, generator=gen, device="cuda").to(BF)
    mixed = y.clone()
    mixed[:, ::2] = other[:, ::2]
    for given in (other, mixed):
        got = torch.empty_like(dw)
        m.mlp_moe_combine_bwd(p, plan, dout, given, w, None, got)
        picked = given[ids].double() * dout[:, None].double()
        # half a step of the values that the plan has more of, and the fp32 sum
        tol = 2.0 ** -8 * picked.norm(dim=-1) * 4 if given is mixed else 0
        tol = tol + sums(264) * picked.norm(dim=-1)
        assert ((got.double() - picked.sum(-1)).abs() <= tol).all()
    # and the same bits again
    again = torch.empty_like(dw)
    m.mlp_moe_combine_bwd(p, plan, dout, y, w, None, again)
    assert torch.equal(again, dw)


def test_plan_without_a_forward():
    # sorted again, the plan has no fp32 values to take
    p, plan, (x, xs, Wg, Wu, Wd, y, w, dout), _, _, _ = step(6, 2, 4, 264, 136, "swiglu",
                                                             torch.float32, 4)
    ids = torch.arange(12, device="cuda").int().view(6, 2) % 4
    m.mlp_moe_sort(p, ids, plan)
    pos = m.moe_plan_views(p, plan)["pos"].long()
    got = torch.empty((6, 2), device="cuda")
    rows = torch.randn((m.mlp_moe_rows(p), 264), device="cuda").to(BF)
    m.mlp_moe_combine_bwd(p, plan, dout, rows, w, None, got)
    picked = rows[pos].double() * dout[:, None].double()
    assert ((got.double() - picked.sum(-1)).abs() <= sums(264) * picked.norm(dim=-1)).all()


def test_bounded_waits():
    # no work is published: every wait runs out, the status says so, the next call is right
    T, E, H, inner = 12, 2, 264, 136
    ones = lambda *s: torch.ones(s, dtype=BF, device="cuda")  # noqa: E731
    p = m.moe(T, E, 1, H, inner, "relu")
    ids = (torch.arange(T, device="cuda") % E).int().view(T, 1)
    plan, rows = m.alloc_moe_plan(p), m.mlp_moe_rows(p)
    m.mlp_moe_sort(p, ids, plan)
    xs, y, W1, Wd = ones(rows, H), ones(rows, H) * 7, ones(E, inner, H), ones(E, H, inner)
    m.mlp_set_wait_timeout_ms(20)
    m.mlp_debug_set_flags(m.DEBUG_NO_WORK)
    try:
        ws = m.mlp_moe_experts_fwd(p, plan, xs, W1, None, Wd, y)
        assert m.mlp_device_status(ws) == -6
    finally:
        m.mlp_debug_set_flags(0)
        m.mlp_set_wait_timeout_ms(0)
    ws = m.mlp_moe_experts_fwd(p, plan, xs, W1, None, Wd, y)
    assert m.mlp_device_status(ws) == 0
    used = int(m.moe_plan_views(p, plan)["offsets"][-1])
    assert (y[:used] == float(torch.tensor(float(H * inner)).to(BF))).all()
