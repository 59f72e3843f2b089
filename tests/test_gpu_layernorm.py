"""The layer norm and its gradients against their formulas in 64 bits.

Tolerances.  u = 2^-24 is fp32's unit roundoff.  A row's sum of H terms passes through chains
of at most 32 values a thread, 5 steps of a warp and 16 warps: n = 64 roundings with what
follows, so the mean is within n u of the mean magnitude, and xhat = (h - mean) rstd within
d = n u (max|h| rstd + 2 |xhat|).  y adds the products with weight and bias; dx is a sum of
terms whose magnitudes are added up below; dweight and dbias sum over rows, in chains of at
most M / blocks + 80.  Each output also rounds once to its type."""
import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U, N = 2.0 ** -24, 64


def half_step(t):
    return torch.finfo(t).eps / 2


def near(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol * 1.001 + 1e-37)
    assert not bad.any(), (what, int(bad.sum()),
                           float(((got.double() - ref).abs() - tol)[bad].max()))


def make(M, H, t, wt, residual=True, bias=True, seed=0, shift=0.3, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed + M * 31 + H)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    return dict(x=(scale * rn(M, H) + shift * rn(M, 1)).to(t),
                r=(scale * rn(M, H)).to(t) if residual else None,
                w=(1 + 0.3 * rn(H)).to(wt), b=(0.3 * rn(H)).to(wt) if bias else None,
                dy=rn(M, H).to(t), dh=rn(M, H).to(t) if residual else None)


def reference(a, eps, dh=True):
    """(h as stored, results and tolerances by name)"""
    t, wt = a["x"].dtype, (a["w"] if a["w"] is not None else a["x"]).dtype
    h = a["x"] if a["r"] is None else (a["x"].float() + a["r"].float()).to(t)
    z = h.double()
    M, H = z.shape
    w = torch.ones(H, dtype=torch.float64, device="cuda") if a["w"] is None else a["w"].double()
    b = torch.zeros_like(w) if a["b"] is None else a["b"].double()
    mean = z.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((z - mean) ** 2).mean(1, keepdim=True) + eps)
    xh = (z - mean) * rstd
    top = z.abs().amax(1, keepdim=True) * rstd
    d = N * U * (top + 2 * xh.abs())
    y = xh * w + b
    dy = a["dy"].double()
    g = dy * w
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = rstd * (g - m1 - xh * m2)
    mg = g.abs().mean(1, keepdim=True)
    # g, m1 and the products round; xhat is off by d wherever it stands
    t_dx = rstd * (N * U * (g.abs() + 2 * mg + 3 * xh.abs() * (g * xh).abs().mean(1, keepdim=True)) +
                   d * m2.abs() + xh.abs() * (g.abs() * d).mean(1, keepdim=True))
    if a["dh"] is not None:
        dx = dx + a["dh"].double()
        t_dx = t_dx + 2 * U * a["dh"].double().abs()
    rows = M * U + 80 * U
    dw, db = (dy * xh).sum(0), dy.sum(0)
    return h, dict(
        y=(y, w.abs() * d + 3 * U * (y.abs() + b.abs()) + half_step(t) * y.abs()),
        mean=(mean[:, 0], N * U * z.abs().mean(1)),
        rstd=(rstd[:, 0], 2 * N * U * (1 + top[:, 0] ** 2 * N * U) * rstd[:, 0]),
        dx=(dx, t_dx + half_step(t) * dx.abs()),
        dw=(dw, rows * (dy * xh).abs().sum(0) + (dy.abs() * d).sum(0) + half_step(wt) * dw.abs()),
        db=(db, rows * dy.abs().sum(0) + half_step(wt) * db.abs()))


def run(a, eps=1e-5, fuse=None):
    M, H = a["x"].shape
    t, wt = a["x"].dtype, a["w"].dtype if a["w"] is not None else a["x"].dtype
    p = m.layernorm(M, H, eps, t, wt)
    y, h = torch.empty(M, H, dtype=t, device="cuda"), None
    if a["r"] is not None:
        h = torch.empty_like(y)
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    m.mlp_layernorm_fwd(p, a["x"], a["r"], a["w"], a["b"], y, h, mean, rstd)
    dx = torch.empty_like(y)
    dw = torch.empty(H, dtype=wt, device="cuda") if fuse is None else fuse[0].clone()
    db = torch.empty_like(dw) if fuse is None else fuse[1].clone()
    hh = a["x"].contiguous() if h is None else h
    m.mlp_layernorm_bwd(p, a["dy"], hh, a["w"], mean, rstd, a["dh"], dx, dw, db,
                        fuse_grad_accum=fuse is not None)
    return dict(y=y, h=h, mean=mean, rstd=rstd, dx=dx, dw=dw, db=db)


def check(a, eps=1e-5):
    got = run(a, eps)
    h, ref = reference(a, eps)
    if a["r"] is not None:
        assert torch.equal(got["h"], h)
    for name, (r, tol) in ref.items():
        near(got[name], r, tol, name)
    return got


@pytest.mark.parametrize("t,wt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("M,H", [(1, 8), (1, 4096), (7, 64), (9, 256), (130, 264), (33, 512),
                                 (65, 1024), (5, 1032), (700, 2048), (31, 2056), (400, 4096),
                                 (37, 4872), (20, 8192), (11, 8200), (6, 14336), (3, 16384),
                                 (9, 520), (300, 3064), (5, 6152)])
@pytest.mark.parametrize("residual", [True, False])
def test_sizes(M, H, t, wt, residual):
    check(make(M, H, t, wt, residual, bias=M % 2 == 1))


@pytest.mark.parametrize("M,H", [(5001, 256), (3000, 1024), (2500, 2048), (1111, 4096),
                                 (333, 16384)])
def test_many_rows(M, H):
    check(make(M, H, BF, F32))


def test_without_weight_and_bias():
    a = make(50, 768, F32, F32)
    a["w"] = a["b"] = None
    check(a)


def test_rows_far_from_zero():
    # a mean of 1000 over a deviation of 1: the squares are of what is left of the mean
    check(make(40, 1024, F32, F32, False, shift=1000.0))
    check(make(40, 4096, BF, BF, False, shift=100.0))


def test_constant_rows():
    a = make(4, 512, F32, F32, False)
    a["x"][1] = 3.25
    a["x"][2] = 0
    got = check(a)
    assert torch.equal(got["y"][1], a["b"]) and torch.equal(got["y"][2], a["b"])


def test_a_nan_stays_in_its_row():
    a = make(9, 1024, BF, F32)
    clean = run(a)
    a["x"][4, 17] = float("nan")
    a["x"][6, 3] = float("inf")
    got = run(a)
    rows = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(got["y"][rows], clean["y"][rows])
    assert torch.equal(got["dx"][rows], clean["dx"][rows])
    assert got["y"][4].isnan().all() and got["y"][6].isnan().any()


def test_pitched_rows():
    for t in (BF, F32):
        a = make(50, 1024, t, F32)
        want = run(a)
        wide = torch.zeros(50, 3 * 1024, dtype=t, device="cuda")
        wide[:, 1024:2048], wide[:, 2048:] = a["x"], a["r"]
        b = dict(a, x=wide[:, 1024:2048], r=wide[:, 2048:])
        got = run(b)
        for k in want:
            assert torch.equal(got[k], want[k]), k


def test_outputs_over_inputs():
    a = make(70, 1024, BF, F32)
    want = run(a)
    p = m.layernorm(70, 1024, 1e-5, BF, F32)
    x, r = a["x"].clone(), a["r"].clone()
    m.mlp_layernorm_fwd(p, x, r, a["w"], a["b"], x, r)  # y over x, h over the residual
    assert torch.equal(x, want["y"]) and torch.equal(r, want["h"])
    for name in ("dy", "dh"):
        dy, dh = a["dy"].clone(), a["dh"].clone()
        to = dy if name == "dy" else dh
        m.mlp_layernorm_bwd(p, dy, want["h"], a["w"], want["mean"], want["rstd"], dh, to)
        assert torch.equal(to, want["dx"])


def test_single_outputs():
    a = make(300, 2048, BF, F32)
    want = run(a)
    p = m.layernorm(300, 2048, 1e-5, BF, F32)
    args = (a["dy"], want["h"], a["w"], want["mean"], want["rstd"], a["dh"])
    dx, dw, db = torch.empty_like(a["dy"]), torch.empty_like(a["w"]), torch.empty_like(a["w"])
    assert m.mlp_layernorm_bwd(p, *args, dx) is None
    m.mlp_layernorm_bwd(p, *args, None, dw)
    m.mlp_layernorm_bwd(p, *args, None, None, db)
    for got, name in ((dx, "dx"), (dw, "dw"), (db, "db")):
        assert torch.equal(got, want[name]), name


@pytest.mark.parametrize("H", [512, 4096])
def test_fused_accumulation(H):
    a = make(600, H, BF, BF)
    plain = run(dict(a, w=a["w"].float(), b=a["b"].float()))
    old = torch.randn(2, H, device="cuda")
    got = run(a, fuse=old)
    assert torch.equal(got["dw"], old[0] + plain["dw"])
    assert torch.equal(got["db"], old[1] + plain["db"])


@pytest.mark.parametrize("M,H", [(8, 64), (4, 2048)])
def test_gradient_against_differences(M, H):
    # f = <dy, y> along a direction of unit scale: a central difference of step h is off by h^2
    # times the third derivative over 6 (rstd and xhat are of order one: below 4 sqrt(M H)) and by
    # the rounding of y, 3 u sqrt(M H) over 2 h.
    a = make(M, H, F32, F32, False, shift=0.0)
    gen = torch.Generator(device="cuda").manual_seed(5)
    v = torch.randn((M, H), generator=gen, device="cuda")
    h = 2.0 ** -7
    got = run(a)

    def f(x, w):
        return float((run(dict(a, x=x, w=w))["y"].double() * a["dy"].double()).sum())

    tol = (M * H) ** 0.5 * (4 * h * h + 6 * U / h) + 1e-4
    slope = float((got["dx"].double() * v.double()).sum())
    assert abs((f(a["x"] + h * v, a["w"]) - f(a["x"] - h * v, a["w"])) / (2 * h) - slope) < tol
    vw = torch.randn(H, generator=gen, device="cuda")
    slope = float((got["dw"].double() * vw.double()).sum())
    assert abs((f(a["x"], a["w"] + vw) - f(a["x"], a["w"] - vw)) / 2 - slope) < tol


@pytest.mark.parametrize("residual", [True, False])
def test_autograd(residual):
    a = make(60, 512, BF, F32, residual)
    leaves = [a[k].clone().requires_grad_(True) for k in ("x", "w", "b")]
    r = a["r"].clone().requires_grad_(True) if residual else None
    shape = (3, 20, 512)
    out = m.layer_norm_func(leaves[0].view(shape), leaves[1], leaves[2],
                            None if r is None else r.view(shape))
    want = run(a)
    if residual:
        y, h = out
        assert torch.equal(h.view(60, 512), want["h"])
        g = torch.autograd.grad([y, h], leaves + [r], [a["dy"].view(shape), a["dh"].view(shape)])
        assert torch.equal(g[0], g[3])
    else:
        y = out
        g = torch.autograd.grad(y, leaves, a["dy"].view(shape))
    assert torch.equal(y.view(60, 512), want["y"])
    for got, name in zip(g, ("dx", "dw", "db")):
        assert torch.equal(got, want[name]), name


def test_autograd_forms():
    a = make(60, 512, BF, BF)
    w = a["w"].clone().requires_grad_(True)
    w.main_grad = torch.ones(512, device="cuda")
    y = m.layer_norm_func(a["x"], w, a["b"], fuse_grad_accum=True)
    y.backward(a["dy"])
    assert w.grad is None and (w.main_grad != 1).any()
    # h alone
    x = a["x"].clone().requires_grad_(True)
    _, h = m.layer_norm_func(x, w.detach(), None, a["r"])
    assert torch.equal(torch.autograd.grad(h, x, a["dh"])[0], a["dh"])
    # a transposed gradient, a pitched input, no rows
    y = m.layer_norm_func(x, w.detach())
    g, = torch.autograd.grad(y, x, a["dy"].t().contiguous().t())
    assert g.shape == x.shape
    wide = torch.randn(60, 1024, device="cuda").to(BF)
    u = wide[:, 512:].detach().requires_grad_(True)
    y = m.layer_norm_func(u, w.detach())
    g, = torch.autograd.grad(y, u, a["dy"])
    v = wide[:, 512:].contiguous().requires_grad_(True)
    y2 = m.layer_norm_func(v, w.detach())
    assert torch.equal(y, y2) and torch.equal(g, torch.autograd.grad(y2, v, a["dy"])[0])
    e = torch.zeros(0, 512, device="cuda", requires_grad=True)
    wf = w.detach().float().requires_grad_(True)
    ge = torch.autograd.grad(m.layer_norm_func(e, wf).sum(), [e, wf])
    assert ge[0].shape == (0, 512) and not ge[1].any()
    with pytest.raises(ValueError):
        m.layer_norm_func(a["x"].half())
    with pytest.raises(ValueError):
        m.layer_norm_func(a["x"], w, a["b"].float())
    with pytest.raises(ValueError):
        m.layer_norm_func(a["x"], w, residual=a["r"].float())
    with pytest.raises(m.MlpError):
        m.layer_norm_func(torch.zeros(2, 12, device="cuda"))


def test_replayed_graph_and_streams():
    a = make(2000, 2048, BF, F32)
    p = m.layernorm(2000, 2048, 1e-5, BF, F32)
    ws = m.alloc_layernorm_workspace(p)
    want = run(a)
    o = {k: torch.zeros_like(v) for k, v in want.items()}

    def call(**kw):
        m.mlp_layernorm_fwd(p, a["x"], a["r"], a["w"], a["b"], o["y"], o["h"], o["mean"], o["rstd"],
                            **kw)
        m.mlp_layernorm_bwd(p, a["dy"], o["h"], a["w"], o["mean"], o["rstd"], a["dh"], o["dx"],
                            o["dw"], o["db"], ws=ws, **kw)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        for v in o.values():
            v.zero_()
        graph.replay()
        for k, v in want.items():
            assert torch.equal(o[k], v), k
    side = torch.cuda.Stream()
    for v in o.values():
        v.zero_()
    torch.cuda.synchronize()
    call(stream=side)
    side.synchronize()
    for k, v in want.items():
        assert torch.equal(o[k], v), k
