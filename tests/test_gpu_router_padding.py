"""Tokens that are not routed have a logits' gradient of exactly zero, whatever the gradients of
the loss and of the weights are: an overflowed loss scale must not reach padding."""
import math

import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF])
# (each number of lanes and values a lane; more slots than lanes)
@pytest.mark.parametrize("T,E,k", [(70, 20, 3), (70, 60, 4), (70, 64, 20), (37, 128, 6),
                                   (19, 250, 8), (9, 500, 8), (9, 1000, 40)])
def test_gradients_that_are_not_finite(T, E, k, dtype, renorm, bad):
    gen = torch.Generator(device="cuda").manual_seed(T + E)
    x = torch.randn((T, E), generator=gen, device="cuda").to(dtype)
    mask = torch.rand((T,), generator=gen, device="cuda") < 0.6
    mask[2:5] = True
    x[3] = -math.inf  # no expert left
    x[~mask] = math.nan  # what padding holds does not matter
    routed = mask.clone()
    routed[3] = False
    p = m.router(T, E, k, renorm, logits_dtype=dtype)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w, bal = torch.empty(T, k, device="cuda"), torch.empty(E + 1, device="cuda")
    m.mlp_moe_router_fwd(p, x, mask, ids, w, None, bal)
    assert not w[~routed].any() and (ids[~routed] == -1).all()
    one, dl = torch.tensor([bad], device="cuda"), torch.full_like(x, 7.0)
    finite = torch.randn((T, k), generator=gen, device="cuda")
    huge = torch.full_like(finite, bad)
    for dw, dloss in ((finite, one), (None, one), (huge, None), (huge, one)):
        m.mlp_moe_router_bwd(p, x, mask, ids, bal, dw, dloss, dl.fill_(7.0))
        assert not dl[~routed].any()  # (a NaN would be "any", too)
        assert dl[routed].isnan().any()


def test_a_padding_token_of_router_func():
    x = torch.randn(12, 16, device="cuda").requires_grad_(True)
    mask = torch.arange(12, device="cuda") < 7
    _, w, _, loss = m.router_func(x, 2, mask)
    g, = torch.autograd.grad([w, loss], [x], [torch.ones_like(w), torch.tensor(math.inf, device="cuda")])
    assert not g[7:].any() and g[:7].isnan().any()
