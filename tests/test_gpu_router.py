"""The router against its formulas in 64 bits.

Tolerances.  u = 2^-24 is fp32's unit roundoff.  The choice and the counts are whole numbers
and exact.  exp(l - m) in fp32: the difference rounds by u |l - m|, expf by 2 ulp (4 u); a sum
of n such terms adds at most n u, a quotient u.  So a probability or weight is within R u of
its value, R = 2 range + n + 16 with range the row's largest |l - m| whose exp is not
negligible (87 at most) and n the terms of the longest chain of sums (values a lane, lanes,
tokens and blocks), plus its type's rounding.  A gradient is a sum of products of those; its
error is R u of the sum of their magnitudes."""
import math

import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


def plain(logits, k, renorm, mask=None, dweights=None, dloss=0.0):
    """Everything in fp64, the choice by a stable sort, and the magnitudes of the gradient's
    terms."""
    z = logits.double().cpu()
    T, E = z.shape
    top = z.max(1)[0] if E else None
    nan = z.isnan().any(1)
    routed = (top > -math.inf) | nan
    if mask is not None:
        routed &= mask.cpu().bool()
    p = torch.softmax(z, 1)
    p[~routed] = 0
    order = torch.sort(torch.where(z.isnan(), math.inf, z), dim=1, descending=True, stable=True)[1]
    if nan.any():  # a NaN above infinity
        key = torch.where(z.isnan(), 2.0, torch.where(z == math.inf, 1.0, 0.0))
        for t in nan.nonzero()[:, 0].tolist():
            order[t] = torch.tensor(sorted(range(E), key=lambda e: (-key[t, e], -z[t, e].nan_to_num(
                0.0, 1e300, -math.inf), e)))
    ids = order[:, :k].clone()
    ids[~routed] = -1
    ids[torch.gather(z, 1, order[:, :k]) == -math.inf] = -1
    at = ids.clamp(min=0)
    has = ids >= 0
    pick = torch.where(has, torch.gather(p, 1, at), 0.0)
    total = pick.sum(1, keepdim=True)
    w = torch.where(has, pick / total, 0.0) if renorm else pick
    counts = torch.bincount(ids[has], minlength=E)
    N = max(int(routed.sum()), 1)
    coef = E * counts.double() / (k * N * N)
    loss = (coef * p.sum(0)).sum()
    res = dict(ids=ids, w=w, counts=counts, coef=coef, loss=loss, p=p, routed=routed)
    if dweights is not None:
        dw = torch.where(has, dweights.double().cpu(), 0.0)
        g = (coef * dloss).expand(T, E).clone()
        if renorm:
            base = p * (g - (p * g).sum(1, keepdim=True))
            mag = p * (g.abs() + (p * g.abs()).sum(1, keepdim=True))
            add = w * (dw - (w * dw).sum(1, keepdim=True))
            mag_add = w * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True))
            res["dl"] = base.scatter_add(1, at, torch.where(has, add, 0.0))
            res["mag"] = mag.scatter_add(1, at, torch.where(has, mag_add, 0.0))
        else:
            g = g.scatter_add(1, at, dw)
            res["dl"] = p * (g - (p * g).sum(1, keepdim=True))
            res["mag"] = p * (g.abs() + (p * g.abs()).sum(1, keepdim=True))
    return res


def chain(T, E):
    """Terms of the longest chain of sums."""
    return 32 + 8 + 32 + 304 + T / 304 + 16


def near(got, ref, tol, what):
    got = got.double().cpu()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(((got - ref).abs() - tol)[bad].max()))


def run(logits, k, renorm=True, mask=None, wt=F32, dweights=None, dloss=None):
    T, E = logits.shape
    p = m.router(T, E, k, renorm, logits_dtype=logits.dtype, weights_dtype=wt)
    ids = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 7.0, dtype=wt, device="cuda")
    counts = torch.full((E,), -9, dtype=torch.int32, device="cuda")
    bal = torch.full((E + 1,), 7.0, device="cuda")
    m.mlp_moe_router_fwd(p, logits, mask, ids, w, counts, bal)
    # without the sums: the same choice and weights
    ids2, w2 = torch.full_like(ids, -9), torch.full_like(w, 7.0)
    assert m.mlp_moe_router_fwd(p, logits, mask, ids2, w2) is None
    assert torch.equal(ids, ids2) and torch.equal(w.nan_to_num(-1), w2.nan_to_num(-1))
    dl = None
    if dweights is not None:
        dl = torch.full((T, E), 7.0, dtype=logits.dtype, device="cuda")
        m.mlp_moe_router_bwd(p, logits, mask, ids, bal, dweights, dloss, dl)
    return ids, w, counts, bal, dl


def check(logits, k, renorm=True, mask=None, wt=F32, grad=True):
    T, E = logits.shape
    gen = torch.Generator(device="cuda").manual_seed(T * 7 + E)
    dweights = torch.randn((T, k), generator=gen, device="cuda").to(wt) if grad else None
    dloss = torch.tensor([0.7], device="cuda")
    ids, w, counts, bal, dl = run(logits, k, renorm, mask, wt, dweights, dloss)
    ref = plain(logits, k, renorm, mask, dweights, float(dloss))
    assert torch.equal(ids.cpu().long(), ref["ids"])
    assert torch.equal(counts.cpu().long(), ref["counts"])
    # E / k, c / N, N and c themselves, their product and a division by N: six roundings
    near(bal[1:], ref["coef"], 6 * U * ref["coef"] + 1e-45, "coef")
    R = (2 * 87 + chain(T, E)) * U
    near(w, ref["w"], (R + half_step(wt)) * ref["w"] + 1e-37, "weights")
    near(bal[0], ref["loss"], R * ref["loss"] + 1e-37, "loss")
    if grad:
        near(dl, ref["dl"], R * ref["mag"] + half_step(logits.dtype) * ref["dl"].abs() + 1e-37,
             "dlogits")


def make(T, E, dtype, seed=0, scale=1.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn((T, E), generator=gen, device="cuda")).to(dtype)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype,wt", [(F32, F32), (BF, F32), (F32, BF), (BF, BF)])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (3, 5, 5), (31, 8, 2), (33, 60, 4),
                                   (257, 100, 7), (700, 128, 1), (65, 200, 8), (2049, 256, 8),
                                   (300, 500, 3), (40, 1024, 64), (5000, 64, 64), (20011, 16, 2),
                                   (40003, 64, 64), (20001, 128, 33), (9001, 250, 64)])
def test_sizes(T, E, k, dtype, wt, renorm):
    check(make(T, E, dtype, T + E), k, renorm, wt=wt)


@pytest.mark.parametrize("E,k", [(8, 3), (60, 8), (96, 9), (256, 6), (1000, 10)])
def test_ties_go_to_the_lowest(E, k):
    # values on a coarse grid, zeros of both signs among them
    x = (make(333, E, F32, 5) * 2).round() / 2
    assert (x == 0).any()
    x = torch.where((x == 0) & (make(333, E, F32, 6) > 0), -0.0, x)
    check(x, k)
    check(torch.zeros(4, E, device="cuda"), k, False)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_masked_tokens_and_experts(dtype, renorm):
    T, E, k = 1037, 60, 6
    x = make(T, E, dtype, 3)
    u = torch.rand((T, E), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    x[u < 0.9] = -math.inf  # often fewer than k experts left
    x[5] = -math.inf
    x[6, 1:] = -math.inf
    x[7] = torch.finfo(dtype).min  # a row at the type's lowest value is a row
    x[8, :58] = torch.finfo(dtype).min
    keep = u[:, 0] < 0.7
    keep[:9] = True
    check(x, k, renorm, keep)
    check(x, k, renorm, keep.to(torch.uint8), wt=BF)
    check(x, k, renorm, torch.zeros_like(keep))  # no token at all
    check(torch.full_like(x, -math.inf), k, renorm)
    # what masked tokens hold does not matter
    y = x.clone()
    y[~keep] = math.nan
    a, b = run(x, k, renorm, keep), run(y, k, renorm, keep)
    for s, t in zip(a[:4], b[:4]):
        assert torch.equal(s, t)


def test_nan_and_infinity():
    x = make(40, 64, F32, 9)
    x[3, 10] = math.nan
    x[4, 7] = math.inf
    x[5] = math.nan
    ids, w, counts, bal, _ = run(x, 4)
    ref = plain(x, 4, True)
    assert torch.equal(ids.cpu().long(), ref["ids"])
    assert ids[3, 0] == 10 and ids[4, 0] == 7 and ids[5].tolist() == [0, 1, 2, 3]
    assert w[3].isnan().all() and w[4].isnan().any() and w[5].isnan().all()
    rest = [i for i in range(40) if i not in (3, 4, 5)]
    assert w[rest].isfinite().all() and bal[0].isnan()
    assert int(counts.sum()) == 160


@pytest.mark.parametrize("dtype", [F32, BF])
def test_pitched_rows_and_odd_addresses(dtype):
    T, E, k = 77, 60, 4
    wide = make(T + 1, 72, dtype, 11)
    for view in (wide[1:, :60], wide[1:, 3:63], wide[1:, 8:68]):
        check(view, k)
    flat = make(1, T * 61 + 1, dtype, 12)[0]
    check(flat[1:1 + T * 61].view(T, 61), k)  # rows at odd addresses
    # a gradient into a pitched view leaves what lies between its rows
    p = m.router(T, E, k, logits_dtype=dtype)
    x = wide[1:, :60]
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    counts, bal = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E + 1, device="cuda")
    m.mlp_moe_router_fwd(p, x, None, ids, w, counts, bal)
    dw, dl = torch.randn(T, k, device="cuda"), torch.full((T, 72), 5.0, dtype=dtype, device="cuda")
    m.mlp_moe_router_bwd(p, x, None, ids, bal, dw, torch.ones(1, device="cuda"), dl[:, :60])
    assert (dl[:, 60:] == 5).all() and (dl[:, :60] != 5).all()
    # over the logits themselves
    want = dl[:, :60].clone()
    m.mlp_moe_router_bwd(p, x, None, ids, bal, dw, torch.ones(1, device="cuda"), x)
    assert torch.equal(x, want)


def test_parts_of_the_gradient_add_up():
    T, E, k = 129, 64, 8
    x = make(T, E, F32, 21)
    p = m.router(T, E, k)
    ids, w, counts, bal, _ = run(x, k)
    dw, one = torch.randn(T, k, device="cuda"), torch.ones(1, device="cuda")
    both, a, b, none = (torch.empty_like(x) for _ in range(4))
    m.mlp_moe_router_bwd(p, x, None, ids, bal, dw, one, both)
    m.mlp_moe_router_bwd(p, x, None, ids, None, dw, None, a)
    m.mlp_moe_router_bwd(p, x, None, ids, bal, None, one, b)
    m.mlp_moe_router_bwd(p, x, None, ids, None, None, None, none)
    ref = plain(x, k, True, None, dw, 1.0)
    near(a + b, both.double().cpu(), 300 * U * ref["mag"] + 1e-37, "sum")
    assert not none.any()


def test_ids_that_name_an_expert_twice_or_none():
    # not what the forward gives: the slots' gradients add up, foreign ids take no part
    x = make(3, 8, F32, 23)
    p = m.router(3, 8, 3, False)
    ids = torch.tensor([[2, 2, 5], [-1, 8, 1000000], [0, -7, 0]], dtype=torch.int32, device="cuda")
    dw = torch.randn(3, 3, device="cuda")
    dl = torch.empty_like(x)
    m.mlp_moe_router_bwd(p, x, None, ids, None, dw, None, dl)
    z = x.double().requires_grad_(True)
    pr = torch.softmax(z, 1)
    d = dw.double()
    (pr[0, 2] * (d[0, 0] + d[0, 1]) + pr[0, 5] * d[0, 2] + pr[2, 0] * (d[2, 0] + d[2, 2])).backward()
    assert (dl.double() - z.grad).abs().max() < 1e-6


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(renorm):
    # f = <dweights, weights> + loss along a direction that changes no choice: the values lie
    # 1/4 apart and move by at most 1/32 either way.  A central difference is off by
    # h^2/6 times the third derivative (below 8 |dweights| here) and by the rounding of f over
    # 2 h: with h = 2^-6 and f about 40, 1e-3 and 2e-4 a token.
    T, E, k, h = 16, 24, 4, 2.0 ** -6
    gen = torch.Generator(device="cuda").manual_seed(31)
    x = torch.stack([torch.randperm(E, generator=gen, device="cuda") for _ in range(T)]) / 4.0
    v = torch.rand((T, E), generator=gen, device="cuda") * 2 - 1
    dw = torch.rand((T, k), generator=gen, device="cuda")
    one = torch.ones(1, device="cuda")

    def f(z):
        _, w, _, bal, _ = run(z, k, renorm)
        return float((w.double() * dw.double()).sum() + bal[0].double())

    dl = run(x, k, renorm, None, F32, dw, one)[-1]
    slope = float((dl.double() * v.double()).sum())
    assert abs((f(x + h * v) - f(x - h * v)) / (2 * h) - slope) < T * 1.2e-3


def test_autograd_and_moe_func():
    """router_func into moe_func: the gradient of a whole layer through logits, with padding
    tokens, against autograd in 64 bits."""
    T, E, k, H, inner = 90, 8, 2, 64, 96
    gen = torch.Generator(device="cuda").manual_seed(41)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = rn(T, H).to(BF)
    Wr = (rn(E, H) / 8).to(BF)
    W = [(rn(E, inner, H) / 8).to(BF), (rn(E, inner, H) / 8).to(BF), (rn(E, H, inner) / 10).to(BF)]
    mask = torch.arange(T, device="cuda") < 81
    logits = (x.float() @ Wr.float().t()).requires_grad_(True)
    ids, w, counts, loss = m.router_func(logits, k, mask)
    out = m.moe_func(x, ids, w, *W, residual=x)
    dout = rn(T, H).to(BF)
    g, = torch.autograd.grad([out, loss], [logits], [dout, torch.tensor(3.0, device="cuda")])
    assert torch.equal(out[81:], x[81:]) and not g[81:].any() and int(counts.sum()) == 81 * k

    z = logits.detach().double().requires_grad_(True)
    p = torch.softmax(z[:81], 1)
    idl = ids[:81].long()
    pick = torch.gather(p, 1, idl)
    wd = pick / pick.sum(1, keepdim=True)
    xd = x[:81].double()
    y = torch.zeros(81, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(idl == e, as_tuple=True)
        a, b = xd[t] @ W[0][e].double().t(), xd[t] @ W[1][e].double().t()
        y = y.index_add(0, t, wd[t, j][:, None] * ((a * torch.sigmoid(a) * b) @ W[2][e].double().t()))
    f = counts.double() / (k * 81)
    ref_loss = E * (f * p.mean(0)).sum()
    ref, = torch.autograd.grad([y, ref_loss], [z], [dout[:81].double(), torch.tensor(
        3.0, dtype=torch.float64, device="cuda")])
    assert abs(float(loss.detach()) - float(ref_loss.detach())) < 1e-6 * float(ref_loss.detach())
    # dweights comes from y and dout in bf16: two roundings a term
    assert float((g - ref).norm() / ref.norm()) < 2e-2


def test_autograd_forms():
    x = make(30, 16, BF, 51).view(2, 15, 16).requires_grad_(True)
    ids, w, counts, loss = m.router_func(x, 3, weights_dtype=BF)
    assert ids.shape == w.shape == (2, 15, 3) and w.dtype == BF and loss.dim() == 0
    g, = torch.autograd.grad(loss, [x], retain_graph=True)
    h, = torch.autograd.grad(w.float().square().sum(), [x], retain_graph=True)
    both, = torch.autograd.grad(w.float().square().sum() + loss, [x])
    assert g.shape == x.shape and g.any() and h.any() and both.dtype == BF
    ids, w, counts, loss = m.router_func(x.detach(), 3, balance=False)
    assert counts is None and loss is None and not w.requires_grad
    e = torch.zeros(0, 16, device="cuda", requires_grad=True)
    ids, w, counts, loss = m.router_func(e, 3)
    assert ids.shape == (0, 3) and float(loss.detach()) == 0 and not counts.any()
    assert torch.autograd.grad(loss + w.sum(), [e])[0].shape == (0, 16)
    with pytest.raises(ValueError):
        m.router_func(x.half(), 2)
    with pytest.raises(m.MlpError):
        m.router_func(x, 17)
    with pytest.raises(ValueError):
        m.router_func(x, 2, torch.ones(30, dtype=torch.bool, device="cuda"))


def test_replayed_graph_and_streams():
    T, E, k = 4099, 60, 4
    p = m.router(T, E, k)
    x = make(T, E, F32, 61)
    ws = m.alloc_router_workspace(p)
    mk = lambda: (torch.empty(T, k, dtype=torch.int32, device="cuda"),  # noqa: E731
                  torch.empty(T, k, device="cuda"), torch.empty(E, dtype=torch.int32, device="cuda"),
                  torch.empty(E + 1, device="cuda"))
    out = mk()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.mlp_moe_router_fwd(p, x, None, *out, ws=ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.mlp_moe_router_fwd(p, x, None, *out, ws=ws)
    for seed in (62, 63):
        x.copy_(make(T, E, F32, seed))
        for o in out:
            o.zero_()
        graph.replay()
        want = mk()
        m.mlp_moe_router_fwd(p, x, None, *want)
        for a, b in zip(out, want):
            assert torch.equal(a, b)
    # an explicit stream
    got = mk()
    torch.cuda.synchronize()
    m.mlp_moe_router_fwd(p, x, None, *got, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_nan_of_either_sign():
    for bits in (0x7fc00000, 0xffc00000 - (1 << 32), 0x7f800001):
        x = make(5, 256, F32, 71)
        x[2, 77] = torch.tensor(bits, dtype=torch.int32, device="cuda").view(F32)
        ids, w, *_ = run(x, 4)
        assert ids[2, 0] == 77 and w[2].isnan().all()
        assert w[[0, 1, 3, 4]].isfinite().all()


@pytest.mark.parametrize("E,k", [(8, 2), (256, 2), (64, 20)])
def test_ids_of_experts_that_vanish(E, k):
    """A caller's own choice of experts 200 below the largest: no gradient, and no NaN."""
    x = make(9, E, F32, 81)
    x[:, -1] = 250
    ids = torch.arange(k, dtype=torch.int32, device="cuda").expand(9, k).contiguous()
    dl = torch.full((9, E), 7.0, device="cuda")
    m.mlp_moe_router_bwd(m.router(9, E, k), x, None, ids, None,
                         torch.ones(9, k, device="cuda"), None, dl)
    assert not dl.any()
