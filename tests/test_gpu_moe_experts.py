"""The experts' MLPs over the sorted rows, their gradients, and the whole layer,
against each expert's formula in fp64.

Tolerances, from the formats (u = 2^-8, bf16's unit roundoff), as in the
linear layer's tests: every value that is stored in bf16 on the way (h, G, U,
dG, dU, the postact, y) errs by u of itself and by what its own operands'
roundings move it; a dot product over values with such errors e moves by at
most 4 times their root sum of squares against the other operand (random
signs; the largest of the elements compared), and rounds once more."""
import math

import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U = 2.0 ** -8
OWN = 2e-5  # the activations' own error (act.cuh), of max(1, |z|)
CURVE = {"swiglu": 0.5, "reglu": 0.0, "geglu": 0.85, "glu": 0.1, "relu_sq": 2.0, "relu": 0.0,
         "gelu_tanh_approx": 0.85}


def act_ref(name, z):
    if name in ("reglu", "relu"):
        return torch.relu(z)
    if name == "relu_sq":
        return torch.relu(z) ** 2
    if name == "swiglu":
        return z * torch.sigmoid(z)
    if name == "glu":
        return torch.sigmoid(z)
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def act_and_grad(name, z):
    z = z.detach().requires_grad_(True)
    a = act_ref(name, z)
    (da,) = torch.autograd.grad(a.sum(), z)
    return a.detach(), da


def rss(a, b):
    return ((a * a) @ (b * b)).sqrt()


def close(got, ref, tol, what):
    off = (got.double() - ref).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((off / tol)[bad].max()))


def nan(*s, dtype=BF):
    return torch.full(s, float("nan"), dtype=dtype, device="cuda")


def weights(E, H, I, act, gen):
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    Wg = (rn(E, I, H) / math.sqrt(H)).to(BF)
    Wu = (rn(E, I, H) / math.sqrt(H)).to(BF) if act in m.GATED_ACTS else None
    return Wg, Wu, (rn(E, H, I) / math.sqrt(I)).to(BF)


class Expert:
    """One expert's rows in fp64, with the bounds of each stored value's error."""

    def __init__(self, act, s, x, Wg, Wu, Wd):
        self.s, self.x, self.act, self.Wd = s, x, act, Wd
        H = x.shape[1]
        sums = (4 * math.sqrt(H) + H / 4) * 2.0 ** -24
        self.Wg, self.Wu = Wg, Wu
        self.g = x @ Wg.t()
        self.eg = sums * rss(x, Wg.t())
        self.a, self.da = act_and_grad(act, self.g)
        self.u = x @ Wu.t() if Wu is not None else torch.ones_like(self.g)
        self.eu = sums * rss(x, Wu.t()) if Wu is not None else torch.zeros_like(self.g)
        self.h = s * self.a * self.u
        own = OWN * self.g.abs().clamp(min=1)
        slope = self.da.abs() + CURVE[act] * self.eg
        eh = s * (self.u.abs() * (slope * self.eg + own) + self.a.abs() * self.eu)
        self.eh = eh + U * self.h.abs()
        self.y = self.h @ Wd.t()
        self.ey = U * self.y.abs() + 4 * rss(self.eh, Wd.t()) + 1e-6
        # the saved preacts, rounded
        self.rg, self.ru = self.eg + U * self.g.abs(), self.eu + U * self.u.abs()

    def backward(self, dy):
        s, c = self.s, CURVE[self.act]
        dh = s * (dy @ self.Wd)
        I = dh.shape[1]
        H = dy.shape[1]
        edh = s * (4 * math.sqrt(H) + H / 4) * 2.0 ** -24 * rss(dy, self.Wd)
        gated = self.Wu is not None
        da = self.da.abs()
        eda = c * self.rg + OWN * self.g.abs().clamp(min=1)
        if self.act in ("reglu", "relu"):
            eda = eda + (self.g.abs() <= self.eg)
        ea = (da + c * self.rg) * self.rg + OWN * self.g.abs().clamp(min=1)
        ru = self.ru if gated else torch.zeros_like(self.u)
        self.dg = dh * self.da * self.u
        big = lambda t, e: t.abs() + e  # noqa: E731
        edg = (edh * da * self.u.abs() + big(dh, edh) * (eda * big(self.u, ru) + da * ru)
               + U * self.dg.abs())
        self.dWg = self.dg.t() @ self.x
        self.eWg = 4 * rss(edg.t(), self.x)
        dx, ex2 = self.dg @ self.Wg, rss(edg, self.Wg) ** 2
        if gated:
            self.du = dh * self.a
            edu = edh * self.a.abs() + big(dh, edh) * ea + U * self.du.abs()
            self.dWu = self.du.t() @ self.x
            self.eWu = 4 * rss(edu.t(), self.x)
            dx, ex2 = dx + self.du @ self.Wu, ex2 + rss(edu, self.Wu) ** 2
        self.dx, self.ex = dx, U * dx.abs() + 4 * ex2.sqrt() + 1e-6
        ep = s * (ea * big(self.u, ru) + self.a.abs() * ru) + U * self.h.abs()
        self.dWd = dy.t() @ self.h
        self.eWd = 4 * rss(dy.t(), ep)


def plan_for(p, ids):
    plan = m.alloc_moe_plan(p)
    m.mlp_moe_sort(p, ids, plan)
    return plan, {k: v for k, v in m.moe_plan_views(p, plan).items()}


@pytest.fixture
def policy(request):
    m.mlp_set_tile_policy(request.param)
    yield request.param
    m.mlp_set_tile_policy(0)


def run_experts(counts, H, I, act, gm=1.25, dm=0.5, seed=0):
    E, T = len(counts), sum(counts)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.cat([torch.full((c,), e) for e, c in enumerate(counts)]).int()
    ids = ids[torch.randperm(T, generator=torch.Generator().manual_seed(seed))].view(T, 1).cuda()
    p = m.moe(T, E, 1, H, I, act, gm, dm)
    plan, v = plan_for(p, ids)
    rows = m.mlp_moe_rows(p)
    Wg, Wu, Wd = weights(E, H, I, act, gen)
    gated = Wu is not None
    x = torch.randn((T, H), generator=gen, device="cuda").to(BF)
    dout = torch.randn((T, H), generator=gen, device="cuda").to(BF)
    one = torch.ones((T, 1), device="cuda")
    xs, dy, y, G = nan(rows, H), nan(rows, H), nan(rows, H), nan(rows, I)
    Up = nan(rows, I) if gated else None
    m.mlp_moe_dispatch(p, plan, x, xs)
    m.mlp_moe_combine_bwd(p, plan, dout, None, one, dy, None)
    ws = m.mlp_moe_experts_fwd(p, plan, xs, Wg, Wu, Wd, y, G, Up)
    assert m.mlp_device_status(ws) == 0
    y2 = nan(rows, H)  # without saving the preacts: the same bits
    m.mlp_moe_experts_fwd(p, plan, xs, Wg, Wu, Wd, y2)
    used = int(v["offsets"][-1])
    assert torch.equal(y[:used], y2[:used])
    assert torch.isnan(y[used:]).all() and torch.isnan(G[used:]).all()  # not written
    keep = (G.clone(), Up.clone() if gated else None)
    dxs, dWg, dWd = nan(rows, H), nan(E, I, H), nan(E, H, I)
    dWu = nan(E, I, H) if gated else None
    ws = m.mlp_moe_experts_bwd(p, plan, dy, xs, Wg, Wu, Wd, G, Up, dxs, dWg, dWu, dWd)
    assert m.mlp_device_status(ws) == 0
    assert torch.isnan(dxs[used:]).all()
    # fp32 accumulation, and single gradients
    acc = [torch.ones_like(t, dtype=torch.float32) if t is not None else None
           for t in (dWg, dWu, dWd)]
    again = lambda: (keep[0].clone(), keep[1].clone() if gated else None)  # noqa: E731
    m.mlp_moe_experts_bwd(p, plan, dy, xs, Wg, Wu, Wd, *again(), None, *acc, fuse_grad_accum=True)
    only_d, only_x = nan(E, H, I), nan(rows, H)
    m.mlp_moe_experts_bwd(p, plan, dy, xs, Wg, Wu, Wd, *again(), dWd=only_d)
    m.mlp_moe_experts_bwd(p, plan, dy, xs, Wg, Wu, Wd, *again(), dxs=only_x)
    assert torch.equal(only_x[:used], dxs[:used])
    for e, n in enumerate(counts):
        r0 = int(v["offsets"][e])
        at = slice(r0, r0 + n)
        f = lambda t: None if t is None else t[e].double()  # noqa: E731
        ref = Expert(act, gm * dm, xs[at].double(), f(Wg), f(Wu), f(Wd))
        close(y[at], ref.y, ref.ey, f"y of expert {e}")
        ref.backward(dy[at].double())
        close(dxs[at], ref.dx, ref.ex, f"dx of expert {e}")
        for name, got, sums, want, err in (
                ("dWg", dWg, acc[0], ref.dWg, ref.eWg),
                ("dWd", dWd, acc[2], ref.dWd, ref.eWd)) + (
                (("dWu", dWu, acc[1], ref.dWu, ref.eWu),) if gated else ()):
            if n == 0:
                assert (got[e] == 0).all() and (sums[e] == 1).all()
                continue
            close(got[e], want, U * want.abs() + err + 1e-6, f"{name} of expert {e}")
            close(sums[e] - 1, want, err + 2.0 ** -22 * (want.abs() + 1), f"fp32 {name} of {e}")
        close(only_d[e], ref.dWd, U * ref.dWd.abs() + ref.eWd + 1e-6, f"dWd alone of {e}")


# no rows, one row, both sides of the 16-, 32-, 128- and 256-row edges
EDGES = [0, 1, 16, 17, 31, 33, 0, 127, 128, 129, 255, 257, 300, 0]


@pytest.mark.parametrize("policy", [1, 2], indirect=True)
@pytest.mark.parametrize("act", list(m.ACTS))
def test_ragged_experts(act, policy):
    run_experts(EDGES, 264, 136, act, seed=policy)


@pytest.mark.parametrize("policy", [1, 2], indirect=True)
@pytest.mark.parametrize("counts,H,I", [([1], 8, 8), ([5, 0], 72, 520), ([600, 30], 520, 1032),
                                        ([0, 0, 0, 700], 1032, 264), ([64] * 9, 256, 512)])
def test_widths(counts, H, I, policy):
    run_experts(counts, H, I, "swiglu", seed=len(counts))
    run_experts(counts, H, I, "relu_sq", 1.0, 1.0, seed=len(counts))


def run_layer(T, E, k, H, I, act, wdt, drop, residual, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    Wg, Wu, Wd = weights(E, H, I, act, gen)
    x = torch.randn((T, H), generator=gen, device="cuda").to(BF)
    ids = torch.rand((T, E), generator=gen, device="cuda").topk(k, -1)[1].int()
    if drop:
        ids[torch.rand((T, k), generator=gen, device="cuda") < drop] = -1
        ids[0] = E  # a token without any expert
    w = torch.rand((T, k), generator=gen, device="cuda").to(wdt)
    r = torch.randn((T, H), generator=gen, device="cuda").to(BF) if residual else None
    p = m.moe(T, E, k, H, I, act, 1.5, 0.5, weights_dtype=wdt)
    out = nan(T, H)
    ws = m.mlp_moe_fwd_infer(p, x, ids, w, Wg, Wu, Wd, r, out)
    assert m.mlp_device_status(ws) == 0
    ref = r.double() if residual else torch.zeros((T, H), dtype=torch.float64, device="cuda")
    err = torch.zeros_like(ref)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not len(t):
            continue
        f = lambda z: None if z is None else z[e].double()  # noqa: E731
        ex = Expert(act, 0.75, x[t].double(), f(Wg), f(Wu), f(Wd))
        wt = w[t, j].double()[:, None]
        ref.index_add_(0, t, wt * ex.y)
        err.index_add_(0, t, wt * ex.ey)
    close(out, ref, U * ref.abs() + err + 1e-6, "out")
    if residual:  # over the residual
        m.mlp_moe_fwd_infer(p, x, ids, w, Wg, Wu, Wd, r, r)
        assert torch.equal(r, out)


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 256, 520), (1, 64, 8, 520, 264), (2, 4, 4, 72, 72),
                                       (5, 64, 3, 264, 136), (8, 3, 3, 1032, 264),
                                       (9, 16, 2, 264, 264), (48, 60, 4, 264, 520),
                                       (300, 8, 2, 136, 264), (1500, 5, 2, 264, 136)])
@pytest.mark.parametrize("act", ["swiglu", "gelu_tanh_approx"])
def test_whole_layer(T, E, k, H, I, act):
    run_layer(T, E, k, H, I, act, torch.float32, 0.0, True, seed=T)
    run_layer(T, E, k, H, I, act, BF, 0.3, False, seed=T + 1)


@pytest.mark.parametrize("T", [1, 4, 40])
def test_nothing_routed(T):
    """Every slot dropped: the residual comes back, or zeros."""
    E, k, H, I = 4, 2, 64, 72
    gen = torch.Generator(device="cuda").manual_seed(1)
    Wg, Wu, Wd = weights(E, H, I, "swiglu", gen)
    x = torch.randn((T, H), generator=gen, device="cuda").to(BF)
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    p = m.moe(T, E, k, H, I)
    for r in (None, x):
        out = nan(T, H)
        m.mlp_moe_fwd_infer(p, x, ids, torch.ones(T, k, device="cuda"), Wg, Wu, Wd, r, out)
        assert torch.equal(out, torch.zeros_like(x) if r is None else x)


@pytest.mark.parametrize("T", [4, 40])
def test_one_expert_does_not_reach_another(T):
    """Weights that are not finite in one expert leave the other experts' tokens alone."""
    E, k, H, I = 6, 1, 136, 72  # neither a multiple of the 64-wide k-blocks
    gen = torch.Generator(device="cuda").manual_seed(2)
    Wg, Wu, Wd = weights(E, H, I, "swiglu", gen)
    x = torch.randn((T, H), generator=gen, device="cuda").to(BF)
    ids = (torch.arange(T, device="cuda") % E).int().view(T, 1)
    one = torch.ones(T, 1, device="cuda")
    p = m.moe(T, E, k, H, I)
    clean, got = nan(T, H), nan(T, H)
    m.mlp_moe_fwd_infer(p, x, ids, one, Wg, Wu, Wd, None, clean)
    for W in (Wg, Wu, Wd):
        W[3] = float("nan")
    m.mlp_moe_fwd_infer(p, x, ids, one, Wg, Wu, Wd, None, got)
    other = ids[:, 0] != 3
    assert torch.equal(got[other], clean[other]) and torch.isnan(got[~other]).all()


def test_gradient_against_differences():
    """The layer's gradients against central differences of the formula in fp64."""
    T, E, k, H, I, h = 10, 3, 2, 16, 24, 1e-5
    gen = torch.Generator(device="cuda").manual_seed(8)
    Ws = weights(E, H, I, "swiglu", gen)
    x = torch.randn((T, H), generator=gen, device="cuda").to(BF)
    dout = torch.randn((T, H), generator=gen, device="cuda").to(BF)
    ids = torch.rand((T, E), generator=gen, device="cuda").topk(k, -1)[1].int()
    w = torch.rand((T, k), generator=gen, device="cuda")
    p = m.moe(T, E, k, H, I)
    plan, _ = plan_for(p, ids)
    rows = m.mlp_moe_rows(p)
    xs, y, G, Up, dy, dxs = (nan(rows, H), nan(rows, H), nan(rows, I), nan(rows, I), nan(rows, H),
                             nan(rows, H))
    dx, dw, dW = nan(T, H), nan(T, k, dtype=torch.float32), [nan(*t.shape) for t in Ws]
    m.mlp_moe_dispatch(p, plan, x, xs)
    m.mlp_moe_experts_fwd(p, plan, xs, *Ws, y, G, Up)
    m.mlp_moe_combine_bwd(p, plan, dout, y, w, dy, dw)
    m.mlp_moe_experts_bwd(p, plan, dy, xs, *Ws, G, Up, dxs, *dW)
    m.mlp_moe_dispatch_bwd(p, plan, dxs, dx)
    leaves = [t.double() for t in (x, w, *Ws)]

    def terms(v):
        xx, ww, g, u, d = v
        e = ids.long()
        z = torch.einsum("th,tkih->tki", xx, g[e])
        hh = z * torch.sigmoid(z) * torch.einsum("th,tkih->tki", xx, u[e])
        return ww[..., None] * torch.einsum("tki,tkhi->tkh", hh, d[e])

    loss = lambda v: (terms(v).sum(1) * dout.double()).sum()  # noqa: E731
    # each of the at most eight roundings on the way (G, U, h, y, dy, dG, dU, the
    # result) moves a gradient by at most u of the sum of its terms' magnitudes,
    # which the formula on absolute values bounds (silu, silu' <= 1.1 |z|, 1.1)
    ab = [t.abs().requires_grad_(True) for t in leaves]
    e = ids.long()
    zb = torch.einsum("th,tkih->tki", ab[0], ab[2][e])
    hb = 1.1 * zb * torch.einsum("th,tkih->tki", ab[0], ab[3][e])
    big = (ab[1][..., None] * torch.einsum("tki,tkhi->tkh", hb, ab[4][e])).sum(1)
    bounds = torch.autograd.grad((big * dout.double().abs()).sum(), ab)
    for i, got in enumerate([dx, dw, *dW]):
        for at in (0, got.numel() // 2, got.numel() - 1):
            v = [t.clone() for t in leaves]
            v[i].view(-1)[at] += h
            up = loss(v)
            v[i].view(-1)[at] -= 2 * h
            slope = ((up - loss(v)) / (2 * h)).item()
            tol = 8 * U * bounds[i].reshape(-1)[at].item() + 1e-6
            assert abs(got.reshape(-1)[at].item() - slope) <= tol, (i, at)
