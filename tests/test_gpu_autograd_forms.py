"""What linear_func and moe_func refuse, and how they behave under autograd's modes."""
import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def randn(seed, *shapes):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(s, generator=gen, device="cuda") / 8).to(BF) for s in shapes]


def moe_args(lead, k, E=4, H=64, inner=72):
    x, Wg, Wu, Wd = randn(1, (*lead, H), (E, inner, H), (E, inner, H), (E, H, inner))
    gen = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.rand((*lead, E), generator=gen, device="cuda").topk(k, -1)[1].int()
    w = torch.rand((*lead, k), generator=gen, device="cuda")
    return x, ids, w, Wg, Wu, Wd


def test_shapes_that_only_have_the_right_number_of_values():
    x, ids, w, *Ws = moe_args((6,), 2)
    with pytest.raises(ValueError, match="weights"):
        m.moe_func(x, ids, w.t().contiguous(), *Ws)
    with pytest.raises(ValueError, match="ids|weights"):
        m.moe_func(x, ids.t().contiguous(), w, *Ws)
    with pytest.raises(ValueError, match="residual"):
        m.moe_func(x, ids, w, *Ws, residual=x.t().contiguous())
    with pytest.raises(ValueError, match="x must"):
        m.moe_func(x.view(3, 128), ids, w, *Ws)
    with pytest.raises(ValueError, match="Wd"):
        m.moe_func(x, ids, w, Ws[0], Ws[1], Ws[0])
    x, W, b, r = randn(3, (6, 64), (8, 64), (8,), (6, 8))
    for bad in (dict(residual=r.t().contiguous()), dict(residual=r.view(8, 6)),
                dict(residual=r.view(2, 3, 8)), dict(bias=r), dict(bias=randn(4, (16,))[0])):
        with pytest.raises(ValueError, match=next(iter(bad))):
            m.linear_func(x, W, **bad)
    with pytest.raises(ValueError, match="x must"):
        m.linear_func(x.view(3, 128), W)


def test_flat_rows():
    # routing and residual of [tokens, .] beside x of more dimensions
    x, ids, w, *Ws = moe_args((2, 3), 2)
    r = randn(5, x.shape)[0]
    whole = m.moe_func(x, ids, w, *Ws, residual=r)
    assert torch.equal(m.moe_func(x, ids.view(6, 2), w.view(6, 2), *Ws, residual=r.view(6, 64)), whole)
    x, W, r = randn(6, (2, 3, 64), (8, 64), (2, 3, 8))
    flat = r.view(6, 8).clone().requires_grad_(True)
    r.requires_grad_(True)
    a, b = m.linear_func(x, W, residual=r, resid_scale=0.5), m.linear_func(x, W, residual=flat,
                                                                         resid_scale=0.5)
    assert torch.equal(a, b)
    ga, = torch.autograd.grad(a.float().sum(), r)
    gb, = torch.autograd.grad(b.float().sum(), flat)
    assert torch.equal(ga.view(6, 8), gb)


def test_second_derivatives_raise():
    # (a gradient without a graph would drop out of a sum with other terms)
    x, ids, w, *Ws = moe_args((6,), 2)
    W = randn(7, (8, 64))[0]
    forms = {"linear": lambda z: m.linear_func(z, W, activation="silu"),
             "moe": lambda z: m.moe_func(z, ids, w, *Ws),
             "mlp": lambda z: m.mlp_func(z, *(t[0] for t in Ws)),
             "block": lambda z: m.mlp_block_func(z, *(t[0] for t in Ws))}
    for name, f in forms.items():
        z = x.clone().requires_grad_(True)
        (g,) = torch.autograd.grad(f(z).float().square().sum(), z, create_graph=True)
        with pytest.raises(RuntimeError, match="twice"):
            (g.float().square().sum() + z.float().sum()).backward()


def test_preact_only_where_a_gradient_follows(monkeypatch):
    from activated_mlp_gemms_gb300 import autograd
    saved, real = [], autograd.mlp_linear_fwd

    def fwd(p, x, W, b, r, out, pre=None):
        saved.append(pre is not None)
        return real(p, x, W, b, r, out, pre)

    monkeypatch.setattr(autograd, "mlp_linear_fwd", fwd)
    x, W, b, r = randn(8, (6, 64), (8, 64), (8,), (6, 8))
    for t in (W, b, r):
        t.requires_grad_(True)
    with torch.no_grad():
        m.linear_func(x, W, b, r, "silu")
    with torch.inference_mode():
        m.linear_func(x, W, b, r, "silu")
    m.linear_func(x, W.detach(), None, r, "silu")  # the residual's gradient needs none
    assert saved == [False] * 3
    m.linear_func(x, W.detach(), b, None, "silu")
    assert saved[3]


def test_no_tokens_into_main_grad():
    # nothing to add, no gradient returned, and the weights are not read
    x, ids, w, *Ws = moe_args((6,), 2)
    Ws = [t.requires_grad_(True) for t in Ws]
    for t in Ws:
        t.main_grad = torch.ones_like(t, dtype=torch.float32)
    empty = x[:0].clone().requires_grad_(True)
    y = m.moe_func(empty, ids[:0], w[:0].requires_grad_(True), *Ws, residual=empty,
                   fuse_grad_accum=True)
    y.sum().backward()
    assert empty.grad.shape == (0, 64)
    assert all(t.grad is None and (t.main_grad == 1).all() for t in Ws)
    with torch.no_grad():
        assert m.moe_func(empty, ids[:0], w[:0], *Ws).shape == (0, 64)
