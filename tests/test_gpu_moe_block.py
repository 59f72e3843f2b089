"""The differentiable linear layer and mixture of experts, alone and together in
the example's feed-forward block, against autograd of the formula in fp64 on the
same bf16 values.

Tolerance: relative to the largest reference value, 2e-2, the package's bound
for bf16 results that pass through several bf16-stored values (the layers' own
tests hold each kernel to its derived bound)."""
import importlib.util
import math
import os

import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TOL = 2e-2
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("moe_block",
                                                  os.path.join(ROOT, "examples", "moe_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rel(got, ref):
    ref = ref.detach()
    return float((got.detach().double() - ref).abs().max() / ref.abs().max().clamp(min=1e-30))


def gelu(z):
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def moe_ref(x, ids, w, Wg, Wu, Wd):
    out = torch.zeros_like(x)
    for e in range(Wg.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            g = x[t] @ Wg[e].t()
            y = (g * torch.sigmoid(g) * (x[t] @ Wu[e].t())) @ Wd[e].t()
            out = out.index_add(0, t, w[t, j][:, None] * y)
    return out


def leaf(t):
    return t.detach().double().requires_grad_(True)


@pytest.mark.parametrize("shape", [(3, 5), (40,), (2, 100)])
@pytest.mark.parametrize("act,scale", [("none", 1.0), ("gelu_tanh_approx", 0.5), ("silu", -2.0)])
def test_linear_func(shape, act, scale):
    K, N = 72, 136
    gen = torch.Generator(device="cuda").manual_seed(len(act))
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, W = rn(*shape, K).to(BF).requires_grad_(True), (rn(N, K) / 8).to(BF).requires_grad_(True)
    b, r = rn(N).to(BF).requires_grad_(True), rn(*shape, N).to(BF).requires_grad_(True)
    out = m.linear_func(x, W, b, r, act, scale)
    dout = rn(*shape, N).to(BF)
    got = torch.autograd.grad(out, (x, W, b, r), dout)
    lv = [leaf(t) for t in (x, W, b, r)]
    z = lv[0] @ lv[1].t() + lv[2]
    a = {"none": z, "gelu_tanh_approx": gelu(z), "silu": z * torch.sigmoid(z)}[act]
    ref = a + scale * lv[3]
    assert out.shape == ref.shape and rel(out, ref) < TOL
    for g, t in zip(got, torch.autograd.grad(ref, lv, dout.double())):
        assert g.shape == t.shape and rel(g, t) < TOL


@pytest.mark.parametrize("shape,wdt", [((3, 5), torch.float32), ((300,), BF)])
def test_moe_func(shape, wdt):
    E, k, H, inner = 6, 2, 72, 136
    gen = torch.Generator(device="cuda").manual_seed(7)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = rn(*shape, H).to(BF).requires_grad_(True)
    r = rn(*shape, H).to(BF).requires_grad_(True)
    Ws = [(rn(E, inner, H) / 8).to(BF).requires_grad_(True),
          (rn(E, inner, H) / 8).to(BF).requires_grad_(True),
          (rn(E, H, inner) / 12).to(BF).requires_grad_(True)]
    ids = torch.rand((*shape, E), generator=gen, device="cuda").topk(k, -1)[1].int()
    ids.view(-1)[1] = -1
    w = torch.rand((*shape, k), generator=gen, device="cuda").to(wdt).requires_grad_(True)
    out = m.moe_func(x, ids, w, *Ws, residual=r)
    dout = rn(*shape, H).to(BF)
    got = torch.autograd.grad(out, (x, w, *Ws, r), dout, retain_graph=True)
    lv = [leaf(t) for t in (x, w, *Ws, r)]
    ref = moe_ref(lv[0].reshape(-1, H), ids.view(-1, k), lv[1].reshape(-1, k), *lv[2:5])
    ref = ref.view(*shape, H) + lv[5]
    assert rel(out, ref) < TOL
    for g, t in zip(got, torch.autograd.grad(ref, lv, dout.double())):
        assert g.shape == t.shape and rel(g, t) < TOL
    with pytest.raises(RuntimeError):  # the preacts became their gradients
        torch.autograd.grad(out, x, dout)
    with torch.no_grad():
        assert rel(m.moe_func(x, ids, w, *Ws, residual=r), ref) < TOL


def test_only_the_gradients_asked_for():
    E, k, H, inner, T = 4, 2, 64, 72, 33
    gen = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, w = rn(T, H).to(BF), torch.rand((T, k), generator=gen, device="cuda")
    Ws = [(rn(E, inner, H) / 8).to(BF), (rn(E, inner, H) / 8).to(BF), (rn(E, H, inner) / 8).to(BF)]
    ids = torch.rand((T, E), generator=gen, device="cuda").topk(k, -1)[1].int()
    dout = rn(T, H).to(BF)
    args = [x, w, *Ws]
    everything = [t.clone().requires_grad_(True) for t in args]
    full = torch.autograd.grad(m.moe_func(everything[0], ids, *everything[1:]), everything, dout)
    for i in range(5):
        some = [t.clone().requires_grad_(i == j) for j, t in enumerate(args)]
        (one,) = torch.autograd.grad(m.moe_func(some[0], ids, *some[1:]), [some[i]], dout)
        assert torch.equal(one, full[i])


def test_fused_accumulation():
    """fp32 main_grad is added to, and no gradient is returned."""
    E, k, H, inner, T = 4, 2, 64, 72, 33
    gen = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = rn(T, H).to(BF).requires_grad_(True)
    ids = torch.rand((T, E), generator=gen, device="cuda").topk(k, -1)[1].int()
    w = torch.rand((T, k), generator=gen, device="cuda")
    Ws = [(rn(*s) / 8).to(BF).requires_grad_(True) for s in
          ((E, inner, H), (E, inner, H), (E, H, inner), (H, H), (H,))]
    dout = rn(T, H).to(BF)

    def run(fuse):
        y = m.moe_func(x, ids, w, *Ws[:3], fuse_grad_accum=fuse)
        return m.linear_func(y, Ws[3], Ws[4], activation="silu", fuse_grad_accum=fuse)

    plain = torch.autograd.grad(run(False), Ws, dout)
    for t in Ws:
        t.main_grad = torch.ones_like(t, dtype=torch.float32)
    run(True).backward(dout)
    for t, g in zip(Ws, plain):
        assert t.grad is None
        # the bf16 gradient is the fp32 one rounded (and fp32 sums may meet in any order)
        near = (t.main_grad - 1).double() - g.double()
        assert (near.abs() <= 2.0 ** -8 * g.double().abs() + 1e-4 * g.double().abs().max()).all()


def test_no_tokens():
    x = torch.zeros((0, 64), dtype=BF, device="cuda", requires_grad=True)
    W = torch.ones((72, 64), dtype=BF, device="cuda", requires_grad=True)
    out = m.linear_func(x, W, activation="relu")
    assert out.shape == (0, 72)
    gx, gW = torch.autograd.grad(out.sum(), (x, W))
    assert gx.shape == (0, 64) and (gW == 0).all()
    Ws = [torch.ones(s, dtype=BF, device="cuda", requires_grad=True)
          for s in ((4, 72, 64), (4, 72, 64), (4, 64, 72))]
    ids = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    y = m.moe_func(x, ids, torch.zeros((0, 2), device="cuda"), *Ws)
    assert y.shape == (0, 64)
    assert all((g == 0).all() for g in torch.autograd.grad(y.sum(), Ws))


def test_workspace_of_a_call_on_another_stream():
    # the call's own workspace is freed here while its kernels still wait on
    # their stream: memory allocated meanwhile must be other memory
    T, E, k, H, I = 300, 8, 2, 256, 512
    gen = torch.Generator(device="cuda").manual_seed(5)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(BF)  # noqa: E731
    p = m.moe(T, E, k, H, I)
    x, Wg, Wu, Wd = rn(T, H), rn(E, I, H) / 16, rn(E, I, H) / 16, rn(E, H, I) / 23
    ids = torch.rand(T, E, generator=gen, device="cuda").topk(k, -1)[1].int()
    w = torch.rand(T, k, generator=gen, device="cuda")
    want, got = torch.empty_like(x), torch.zeros_like(x)
    m.mlp_moe_fwd_infer(p, x, ids, w, Wg, Wu, Wd, None, want)
    n = m.mlp_moe_workspace_size(p, m.MODE_INFER)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        torch.cuda._sleep(20_000_000)
    m.mlp_moe_fwd_infer(p, x, ids, w, Wg, Wu, Wd, None, got, stream=other)
    mine = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all(bool((t == 7).all()) for t in mine)


@pytest.mark.parametrize("tokens", [1, 6, 200])
def test_block_of_the_example(tokens):
    ex = example()
    p = ex.make_params()
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((tokens, 256), generator=gen, device="cuda").to(BF).requires_grad_(True)
    out = ex.block(x, p)
    dout = torch.randn((tokens, 256), generator=gen, device="cuda").to(BF)
    names = ["Wg", "Wu", "Wd", "W1", "b1", "W2", "b2"]
    got = torch.autograd.grad(out, [x] + [p[n] for n in names], dout)
    q, x64 = {k: leaf(v) for k, v in p.items()}, leaf(x)
    # the router's choice and weights come from the kernel's own (rounded) logits
    logits = m.linear_func(x, p["Wr"], p["br"])
    top, ids = torch.topk(logits.float(), 2, dim=-1)
    exact = x64 @ q["Wr"].t() + q["br"]
    assert rel(logits, exact) < TOL
    w = torch.softmax(exact.gather(1, ids), -1)
    r = x64 + moe_ref(x64, ids, w, q["Wg"], q["Wu"], q["Wd"])
    ref = r + gelu(r @ q["W1"].t() + q["b1"]) @ q["W2"].t() + q["b2"]
    assert rel(out, ref) < TOL
    want = torch.autograd.grad(ref, [x64] + [q[n] for n in names], dout.double())
    for n, g, t in zip(["x"] + names, got, want):
        assert rel(g, t) < TOL, n


def test_example_trains(monkeypatch, capsys):
    ex = example()
    monkeypatch.setattr("sys.argv", ["moe_block.py", "--steps", "12", "--tokens", "256"])
    losses = ex.main()
    assert losses[-1] < 0.8 * losses[0]
