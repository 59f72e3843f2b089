"""The linear layer (bias, activation, residual in the epilogue) and its
gradients against the formulas in fp64.

Tolerances, from the formats.  u = 2^-8 is bf16's unit roundoff.  An output
rounded once from fp32 errs by u |value| plus the fp32 sum's error, taken as
(4 sqrt(K) + K / 4) 2^-24 of the products' root sum of squares (random signs,
and K / 16 tensor-core steps that may each truncate), plus the activations'
own error (act.cuh: at most 1e-5 of max(1, |z|)).  The gradients
go through dz, which is rounded to bf16 and formed from z rounded to bf16:
each of its elements errs by u |dz| and by u |z| |dout| max|act''|, so a dot
product with random signs errs by about that over the products' root sum of
squares; the factor 4 covers the largest of the elements compared."""
import math

import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U = 2.0 ** -8
# max |act''| (relu's kink is handled where z is within the sum's error of 0)
CURVE = {"none": 0.0, "relu": 0.0, "relu_sq": 2.0, "gelu_tanh_approx": 0.85, "silu": 0.5,
         "sigmoid": 0.1}


def act_ref(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.relu(z)
    if name == "relu_sq":
        return torch.relu(z) ** 2
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "sigmoid":
        return torch.sigmoid(z)
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def inputs(M, N, K, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    return (rn(M, K).to(BF), (rn(N, K) / math.sqrt(K)).to(BF), rn(N).to(BF), rn(M, N).to(BF),
            rn(M, N).to(BF))


def rss(a, b):
    """Root sum of squares of the products of a @ b."""
    return ((a * a) @ (b * b)).sqrt()


def close(got, ref, tol):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got.double() - ref).abs() / tol)[bad].max()))


def nan(*s, dtype=BF):
    return torch.full(s, float("nan"), dtype=dtype, device="cuda")


def check(M, N, K, act, bias=True, residual=True, seed=0, rs=0.75):
    x, W, b, r, dout = inputs(M, N, K, seed)
    b = b if bias else None
    r = r if residual else None
    p = m.linear(M, N, K, act, rs)
    out, pre = nan(M, N), nan(M, N)
    ws = m.mlp_linear_fwd(p, x, W, b, r, out, pre)
    assert m.mlp_device_status(ws) == 0
    x64, W64, d64 = x.double(), W.double(), dout.double()
    z = (x64 @ W64.t() + (b.double() if bias else 0)).requires_grad_(True)
    a = act_ref(act, z)
    (da,) = torch.autograd.grad(a.sum(), z)
    z, a = z.detach(), a.detach()
    ref = a + (rs * r.double() if residual else 0)
    sums = (4 * math.sqrt(K) + K / 4) * 2.0 ** -24 * (rss(x64, W64.t()) + 1)
    close(pre, z, U * z.abs() + sums + 1e-30)
    slope = da.abs() + CURVE[act] * sums  # |act'| near z
    own = 0 if act in ("none", "relu", "relu_sq") else 1e-5 * z.abs().clamp(min=1)
    close(out, ref, U * ref.abs() + sums * slope + own + 2.0 ** -23 * (a.abs() + ref.abs()))
    # without pre_save
    out2 = nan(M, N)
    m.mlp_linear_fwd(p, x, W, b, r, out2)
    close(out2, ref, U * ref.abs() + sums * slope + own + 2.0 ** -23 * (a.abs() + ref.abs()))

    dx, dW, db = nan(M, K), nan(N, K), nan(N)
    keep = None if act == "none" else pre
    ws = m.mlp_linear_bwd(p, dout, x, W, keep, dx, dW, db)
    assert m.mlp_device_status(ws) == 0
    dz = d64 * da
    err = U * dz.abs() + d64.abs() * (CURVE[act] * (U * z.abs() + sums) + 2e-5)
    if act == "relu":
        err = err + d64.abs() * (z.abs() <= sums)
    fp = 4 * 2.0 ** -24
    close(dx, dz @ W64, U * (dz @ W64).abs() + 4 * rss(err, W64) + fp * math.sqrt(N) * rss(dz, W64)
          + 1e-30)
    rdW = dz.t() @ x64
    close(dW, rdW, U * rdW.abs() + 4 * rss(err.t(), x64) + fp * math.sqrt(M) * rss(dz.t(), x64)
          + 1e-30)
    rdb = dz.sum(0)
    tdb = 4 * err.square().sum(0).sqrt() + fp * math.sqrt(M) * dz.square().sum(0).sqrt()
    close(db, rdb, U * rdb.abs() + tdb + 1e-30)
    # fp32 accumulation into given gradients
    gW, gb = torch.ones(N, K, device="cuda"), torch.ones(N, device="cuda")
    m.mlp_linear_bwd(p, dout, x, W, keep, None, gW, gb, fuse_grad_accum=True)
    close(gW - 1, rdW, 4 * rss(err.t(), x64) + fp * math.sqrt(M) * (rss(dz.t(), x64) + 1) + 3e-7
          + 2.0 ** -23 * rdW.abs())
    close(gb - 1, rdb, tdb + 3e-7 + 2.0 ** -23 * rdb.abs())
    # each gradient alone
    dx2, dW2, db2 = nan(M, K), nan(N, K), nan(N)
    m.mlp_linear_bwd(p, dout, None, W, keep, dx=dx2)
    m.mlp_linear_bwd(p, dout, x, None, keep, dW=dW2)
    m.mlp_linear_bwd(p, dout, None, None, keep, db=db2)
    assert torch.equal(dW2, dW) and torch.equal(db2, db)
    close(dx2, dx.double(), 2 * U * dx.double().abs() + fp * math.sqrt(N) * rss(dz, W64) + 1e-30)


# rows: a stream, its edge, the skinny kernel, ragged tiles, pairs; widths off every tile edge
SHAPES = [(1, 8, 8), (1, 72, 4104), (3, 768, 768), (8, 264, 1032), (9, 264, 1032), (17, 520, 2056),
          (64, 4096, 1024), (128, 24, 4096), (129, 640, 72), (300, 1000, 328), (777, 4864, 512),
          (2049, 136, 2048), (1024, 2056, 1160)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", list(m.LINEAR_ACTS))
def test_against_formula(M, N, K, act):
    check(M, N, K, act, seed=M + N)


@pytest.mark.parametrize("M,N,K", [(9, 8, 8), (16, 136, 4096), (31, 520, 72), (100, 4096, 2056),
                                   (200, 264, 1160), (256, 128, 512), (588, 400, 1160),
                                   (700, 136, 2048)])
@pytest.mark.parametrize("policy", [0, 1, 2])
def test_few_rows_by_every_route(M, N, K, policy):
    """The skinny kernel (policy 0: alone, and with clusters sharing K) and the tiles."""
    m.mlp_set_tile_policy(policy)
    try:
        check(M, N, K, "gelu_tanh_approx", seed=M)
        check(M, N, K, "none", residual=False, seed=M)
    finally:
        m.mlp_set_tile_policy(0)


@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("M,N,K", [(5, 264, 520), (48, 520, 2048), (300, 264, 520)])
def test_optional_operands(M, N, K, bias, residual):
    check(M, N, K, "gelu_tanh_approx", bias, residual, seed=5)


@pytest.mark.parametrize("M", [1, 8, 40, 300])
def test_pitched_rows_and_in_place_residual(M):
    N, K = 264, 520
    x, W, b, r, dout = inputs(M, N, K, 9)
    p = m.linear(M, N, K, "silu", 0.5)
    want, pre = nan(M, N), nan(M, N)
    m.mlp_linear_fwd(p, x, W, b, r, want, pre)
    wide_x, wide_r, wide_o, wide_d = nan(M, K + 24), nan(M, N + 8), nan(M, N + 40), nan(M, N + 16)
    xv, rv, ov, dv = wide_x[:, 8:8 + K], wide_r[:, :N], wide_o[:, 16:16 + N], wide_d[:, 8:8 + N]
    xv.copy_(x), rv.copy_(r), dv.copy_(dout)
    got_pre = nan(M, N)
    m.mlp_linear_fwd(p, xv, W, b, rv, ov, got_pre)
    assert torch.equal(ov, want) and torch.equal(got_pre, pre)
    assert torch.isnan(wide_o[:, :16]).all() and torch.isnan(wide_o[:, 16 + N:]).all()
    m.mlp_linear_fwd(p, x, W, b, rv, rv)  # over the residual
    assert torch.equal(rv, want) and torch.isnan(wide_r[:, N:]).all()
    grads = [nan(M, K), nan(N, K), nan(N)]
    again = [nan(M, K), nan(N, K), nan(N)]
    m.mlp_linear_bwd(p, dout, x, W, pre, *grads)
    m.mlp_linear_bwd(p, dv, xv, W, pre, *again)
    for g, a in zip(grads, again):
        assert torch.equal(g, a)


@pytest.mark.parametrize("act", ["relu_sq", "gelu_tanh_approx", "silu", "sigmoid"])
def test_gradient_against_differences(act):
    """Central differences of sum(dout * out) in fp64 of the formula, at single
    elements of x, W and bias, against the kernels' gradients.  The step h leaves
    a truncation error of h^2 times the third derivative; what remains is the
    bf16 rounding of dz, z and the result (the bound of `check`, with every
    term's magnitude summed)."""
    M, N, K, h = 12, 16, 24, 1e-5
    x, W, b, r, dout = inputs(M, N, K, 21)
    p = m.linear(M, N, K, act)
    out, pre = nan(M, N), nan(M, N)
    m.mlp_linear_fwd(p, x, W, b, r, out, pre)
    g = [nan(M, K), nan(N, K), nan(N)]
    m.mlp_linear_bwd(p, dout, x, W, pre, *g)
    leaves = [t.double() for t in (x, W, b)]
    d64 = dout.double()
    z = leaves[0] @ leaves[1].t() + leaves[2]
    z.requires_grad_(True)
    (da,) = torch.autograd.grad(act_ref(act, z).sum(), z)
    z = z.detach()
    size = d64.abs() * (U * da.abs() + CURVE[act] * U * z.abs() + 2e-5)  # bounds |error of dz|

    def loss(v):
        return (act_ref(act, v[0] @ v[1].t() + v[2]) * d64).sum()

    bounds = [size @ leaves[1].abs(), size.t() @ leaves[0].abs(), size.sum(0)]
    for i, t in enumerate(leaves):
        for at in [0, t.numel() // 3, t.numel() - 1]:
            v = [u.clone() for u in leaves]
            v[i].view(-1)[at] += h
            up = loss(v)
            v[i].view(-1)[at] -= 2 * h
            slope = ((up - loss(v)) / (2 * h)).item()
            have = g[i].reshape(-1)[at].item()
            assert abs(have - slope) <= (2 * U * abs(slope) + bounds[i].reshape(-1)[at].item()
                                           + 1e-5)


def test_not_finite_stays_in_its_place():
    """A row with an infinity or a NaN leaves the other rows' outputs alone."""
    for M in (6, 40, 300):
        x, W, b, r, dout = inputs(M, 264, 520, 4)
        p = m.linear(M, 264, 520, "none")
        clean, got = nan(M, 264), nan(M, 264)
        m.mlp_linear_fwd(p, x, W, b, r, clean)
        x[2, 7], x[4, 0] = float("inf"), float("nan")
        m.mlp_linear_fwd(p, x, W, b, r, got)
        rows = [i for i in range(M) if i not in (2, 4)]
        assert torch.equal(got[rows], clean[rows])
        assert torch.isnan(got[4]).all() and not torch.isfinite(got[2]).any()


def test_stream_and_graph():
    """On a stream of its own, and replayed from a captured graph on new values."""
    M, N, K = 300, 520, 264
    x, W, b, r, dout = inputs(M, N, K, 2)
    p = m.linear(M, N, K, "gelu_tanh_approx")
    fw, bw = m.alloc_linear_workspace(p), m.alloc_linear_workspace(p, True)
    out, pre, dx, dW, db = nan(M, N), nan(M, N), nan(M, K), nan(N, K), nan(N)

    def step():
        m.mlp_linear_fwd(p, x, W, b, r, out, pre, ws=fw)
        m.mlp_linear_bwd(p, dout, x, W, pre, dx, dW, db, ws=bw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    x2 = inputs(M, N, K, 3)[0]
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (out, dx, dW, db)]
    step()
    torch.cuda.synchronize()
    for a, t in zip(got, (out, dx, dW, db)):
        assert torch.equal(a, t)
