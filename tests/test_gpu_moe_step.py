"""The layer norm, the router with its balance loss, the experts and the orthogonalised update
as a training step uses them together (examples/moe_step.py), against autograd of the formula in
fp64 on the same values.

Tolerance: relative to the largest reference value, 2e-2, the package's bound for bf16 results
that pass through several bf16-stored values (the operators' own tests hold each kernel to its
derived bound)."""
import importlib.util
import os

import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TOL = 2e-2
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("moe_step",
                                                  os.path.join(ROOT, "examples", "moe_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rel(got, ref):
    ref = ref.detach()
    return float((got.detach().double() - ref).abs().max() / ref.abs().max().clamp(min=1e-30))


def reference(x, p, ids, mask, top_k):
    """The block in fp64 with the experts that the library chose."""
    mean, var = x.mean(1, keepdim=True), x.var(1, unbiased=False, keepdim=True)
    h = (x - mean) / torch.sqrt(var + 1e-5) * p["norm_w"] + p["norm_b"]
    logits = h @ p["Wr"].t()
    probs = torch.softmax(logits, 1)
    E = probs.shape[1]
    pick = torch.gather(probs, 1, ids.clamp(min=0))
    w = pick / pick.sum(1, keepdim=True) * (ids >= 0)
    y = x.clone()
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        g = h[t] @ p["Wg"][e].t()
        part = (g * torch.sigmoid(g) * (h[t] @ p["Wu"][e].t())) @ p["Wd"][e].t()
        y = y.index_add(0, t, w[t, j][:, None] * part)
    N = int(mask.sum())
    f = torch.bincount(ids[ids >= 0], minlength=E).double() / (top_k * N)
    return y, E * (f * probs[mask].sum(0) / N).sum()


@pytest.mark.parametrize("tokens,H,inner,E,top_k", [(70, 64, 96, 8, 2), (300, 256, 352, 16, 4),
                                                    (5, 128, 72, 8, 1)])
def test_gradients_of_the_block(tokens, H, inner, E, top_k):
    ex = example()
    p = ex.make_params(H, inner, E)
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((tokens, H), generator=gen, device="cuda").to(BF).requires_grad_(True)
    dy = torch.randn((tokens, H), generator=gen, device="cuda").to(BF)
    mask = torch.arange(tokens, device="cuda") < tokens - 2
    y, balance, counts = ex.block(x, p, top_k, mask)
    leaves = [x] + list(p.values())
    got = torch.autograd.grad([y, balance], leaves, [dy, torch.tensor(5.0, device="cuda")])
    assert torch.equal(y[~mask], x[~mask])
    # the library's choice, from its own logits
    with torch.no_grad():
        h = m.layer_norm_func(x, p["norm_w"], p["norm_b"])
        ids = m.router_func(m.linear_func(h, p["Wr"]), top_k, mask)[0].long()
    assert torch.equal(counts.long(), torch.bincount(ids[ids >= 0], minlength=E))
    wide = {k: v.detach().double().requires_grad_(True) for k, v in p.items()}
    xd = x.detach().double().requires_grad_(True)
    yd, bd = reference(xd, wide, ids, mask, top_k)
    want = torch.autograd.grad([yd, bd], [xd] + list(wide.values()),
                               [dy.double(), torch.tensor(5.0, dtype=torch.float64, device="cuda")])
    assert rel(y, yd) <= TOL and rel(balance, bd) <= TOL
    for (name, g), r in zip(zip(["x"] + list(p), got), want):
        assert rel(g, r) <= TOL, (name, rel(g, r))


def test_update():
    """A step of a matrix, of a stack and of a vector against the formula in fp64: the
    orthogonalised part to 7e-3 (its bound), the weights to a bf16 rounding more."""
    ex = example()
    gen = torch.Generator(device="cuda").manual_seed(9)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    for shape in ((64, 256), (8, 352, 256), (256,)):
        w, mom, g = rn(*shape).to(BF), rn(*shape), rn(*shape).to(BF)
        if len(shape) == 1:
            w = w.float()
        w0, m0 = w.double(), mom.double()
        ex.update(w, mom, g, 0.1, beta=0.5)
        M = 0.5 * m0 + g.double()
        step = M
        if len(shape) > 1:
            rows, cols = shape[-2:]
            X = M / M.square().sum((-2, -1), keepdim=True).sqrt()
            X = X.transpose(-2, -1) if rows > cols else X
            a, b, c = m.MUON_COEFFS
            for _ in range(5):
                A = X @ X.transpose(-2, -1)
                X = a * X + (b * A + c * A @ A) @ X
            X = X.transpose(-2, -1) if rows > cols else X
            step = max(1.0, rows / cols) ** 0.5 * X
        want = w0 - 0.1 * step
        assert rel(mom, M) < 1e-6
        eps = 0.1 * 7e-3 * step.norm() + 2.0 ** -8 * want.norm() * (len(shape) > 1)
        assert (w.double() - want).norm() <= eps + 1e-6 * want.norm()


def test_example_runs(monkeypatch, capsys):
    ex = example()
    monkeypatch.setattr("sys.argv", ["moe_step.py", "--steps", "3", "--tokens", "256"])
    losses = ex.main()
    assert len(losses) == 3 and all(v == v and abs(v) < 1e6 for v in losses)
    assert "slots" in capsys.readouterr().out
