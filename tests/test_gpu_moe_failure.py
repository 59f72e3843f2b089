"""Bounded waits of the linear layer's and the experts' GEMMs: with the hook that
publishes no work every wait runs out, the status word says so, and the context
stays usable."""
import pytest
import torch

import activated_mlp_gemms_gb300 as m

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TIMEOUT = -6


@pytest.fixture
def no_work():
    m.mlp_set_wait_timeout_ms(20)
    m.mlp_debug_set_flags(m.DEBUG_NO_WORK)
    yield
    m.mlp_debug_set_flags(0)
    m.mlp_set_wait_timeout_ms(0)


@pytest.mark.parametrize("M", [40, 300])  # the skinny kernel, and the tiles
def test_linear(no_work, M):
    N, K = 264, 520
    t = lambda *s: torch.ones(s, dtype=BF, device="cuda")  # noqa: E731
    p = m.linear(M, N, K)
    out = t(M, N)
    ws = m.mlp_linear_fwd(p, t(M, K), t(N, K), None, None, out)
    assert m.mlp_device_status(ws) == TIMEOUT
    m.mlp_debug_set_flags(0)
    ws = m.mlp_linear_fwd(p, t(M, K), t(N, K), None, None, out)
    assert m.mlp_device_status(ws) == 0
    assert (out == K).all()


@pytest.mark.parametrize("policy", [1, 2])
def test_experts(no_work, policy):
    T, E, H, I = 600, 2, 264, 136
    t = lambda *s: torch.ones(s, dtype=BF, device="cuda")  # noqa: E731
    p = m.moe(T, E, 1, H, I, "relu")
    ids = (torch.arange(T, device="cuda") % E).int().view(T, 1)
    one = torch.ones(T, 1, device="cuda")
    x, W1, Wd, out = t(T, H), t(E, I, H), t(E, H, I), t(T, H)
    m.mlp_set_tile_policy(policy)
    try:
        ws = m.mlp_moe_fwd_infer(p, x, ids, one, W1, None, Wd, None, out)
        assert m.mlp_device_status(ws) == TIMEOUT
        m.mlp_debug_set_flags(0)
        ws = m.mlp_moe_fwd_infer(p, x, ids, one, W1, None, Wd, None, out)
        assert m.mlp_device_status(ws) == 0
    finally:
        m.mlp_set_tile_policy(0)
    assert (out == float(torch.tensor(float(H * I)).to(BF))).all()
