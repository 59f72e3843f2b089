"""The routing weights and the loss within the error that include/mlp_router.h states.

With u = 2^-24 and d a logit's distance from its token's largest: the difference rounds (u d), so
does its product with log2(e) (u d), whose constant is off by 0.23 u of itself (0.23 u d); the
hardware's base-2 exponential is within 2^-22 = 4 u of its value.  So e^-d is within
(2.3 d + 4) u of itself.  The softmax's sum is off by the mean of that over the token's experts
(the mean of d is at most ln E, the largest entropy: 2.3 * 6.94 = 16 for 1024 experts) and by its
chain of at most 32 / 2 + 1 + 5 = 22 additions; the reciprocal is within 2 u of its value, and the
product rounds once.  A weight is within (2.3 d + 4 + 16 + 4 + 22 + 2 + 1) u = (2.3 d + 49) u, and
its type's rounding, of its value; below 2^-126 it may be zero."""
import math

import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.mark.parametrize("scale", [0.01, 1.5, 12.0, 40.0])
@pytest.mark.parametrize("wt", [F32, BF])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(500, 8, 8), (300, 60, 8), (200, 64, 64), (200, 250, 8),
                                   (100, 512, 30), (100, 1024, 64)])
def test_weights(T, E, k, renorm, wt, scale):
    gen = torch.Generator(device="cuda").manual_seed(E + k)
    x = scale * torch.randn((T, E), generator=gen, device="cuda")
    p = m.router(T, E, k, renorm, weights_dtype=wt)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w, bal = torch.empty(T, k, dtype=wt, device="cuda"), torch.empty(E + 1, device="cuda")
    m.mlp_moe_router_fwd(p, x, None, ids, w, None, bal)
    z = x.double()
    prob = torch.softmax(z, 1)
    ref = torch.gather(prob, 1, ids.long())
    if renorm:
        ref = ref / ref.sum(1, keepdim=True)
    d = z.amax(1, keepdim=True) - torch.gather(z, 1, ids.long())
    tol = ((2.3 * d + 49) * U + (0 if wt == F32 else 2.0 ** -8)) * ref + 2.0 ** -126
    assert ((w.double() - ref).abs() <= tol).all()
    # the loss: sums of probabilities over at most T tokens, the coefficients' six roundings
    worst = 2.3 * math.log(E) + 49 + T + E + 6
    loss = (bal[1:].double() * prob.sum(0)).sum()
    assert abs(float(bal[0]) - float(loss)) <= worst * U * float(loss)
