"""A NaN stays one through max(z, 0): a row with one does not come out as zeros."""
import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def randn(seed, *shapes):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(s, generator=gen, device="cuda") / 8).to(BF) for s in shapes]


@pytest.mark.parametrize("act", ["relu", "relu_sq"])
@pytest.mark.parametrize("M", [6, 40, 300])
def test_linear(act, M):
    x, W, dout = randn(M, (M, 72), (136, 72), (M, 136))
    p = m.linear(M, 136, 72, act)
    clean, got, pre, dx = (torch.zeros((M, n), dtype=BF, device="cuda") for n in (136, 136, 136, 72))
    m.mlp_linear_fwd(p, x, W, None, None, clean)
    x[4, 1] = float("nan")
    m.mlp_linear_fwd(p, x, W, None, None, got, pre)
    assert torch.isnan(got[4]).all() and torch.isnan(pre[4]).all()
    rest = [i for i in range(M) if i != 4]
    assert torch.equal(got[rest], clean[rest])
    # the gradient of what is not finite
    dout[4] = float("nan")
    m.mlp_linear_bwd(p, dout, x, W, pre, dx=dx)
    assert torch.isnan(dx[4]).all() and torch.isfinite(dx[rest]).all()


@pytest.mark.parametrize("act", ["relu", "relu_sq", "reglu"])
@pytest.mark.parametrize("T", [4, 40, 600])
def test_experts(act, T):
    x, W1, Wu, Wd = randn(T, (T, 64), (3, 72, 64), (3, 72, 64), (3, 64, 72))
    Wu = Wu if act == "reglu" else None
    p = m.moe(T, 3, 1, 64, 72, act)
    ids = (torch.arange(T, device="cuda") % 3).int().view(T, 1)
    w, out = torch.ones((T, 1), device="cuda"), torch.zeros_like(x)
    x[2, 5] = float("nan")
    m.mlp_moe_fwd_infer(p, x, ids, w, W1, Wu, Wd, None, out)
    assert torch.isnan(out[2]).all() and torch.isfinite(out[:2]).all() and torch.isfinite(out[3:]).all()


@pytest.mark.parametrize("act", ["relu", "relu_sq", "reglu"])
@pytest.mark.parametrize("M", [1, 5, 12, 300])
def test_dense(act, M):
    x, W1, Wu, Wd = randn(M, (M, 64), (72, 64), (72, 64), (64, 72))
    p = m.problem(M, 64, 72, act, 1.0, 1.0)
    out = torch.zeros_like(x)
    x[M // 2, 5] = float("nan")
    m.mlp_fwd_infer(p, x, W1, Wu if act == "reglu" else None, Wd, out)
    assert torch.isnan(out[M // 2]).all() and torch.isnan(out).sum() == 64
