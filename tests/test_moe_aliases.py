"""Outputs over operands that other blocks still read are refused (no GPU needed:
fake, never-dereferenced pointers; nothing is enqueued on a refusal)."""
import ctypes
import os

import pytest

import activated_mlp_gemms_gb300 as m

A = [0x100000 * (i + 1) for i in range(16)]  # distinct operands


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(m.LIB_PATH):
        from activated_mlp_gemms_gb300 import _build
        _build.build()
    return m.lib()


def test_token_calls(L):
    b = ctypes.byref(m.moe(16, 8, 2, 64))
    assert L.mlp_moe_dispatch(b, A[0], A[1], A[1], None) == -1
    assert L.mlp_moe_dispatch_bwd(b, A[0], A[1], A[1], None) == -1
    assert L.mlp_moe_combine(b, A[0], A[1], A[2], None, A[1], None) == -1
    # dout, y, weights, dy, dweights
    assert L.mlp_moe_combine_bwd(b, A[0], A[1], A[2], A[3], A[1], None, None) == -1
    assert L.mlp_moe_combine_bwd(b, A[0], A[1], A[2], A[3], A[2], A[4], None) == -1


@pytest.mark.parametrize("over", ["dy", "xs"])
def test_experts_backward(L, over):
    p = m.moe(16, 8, 2, 64, 128)
    plan, dy, xs, Wg, Wu, Wd, G, U, dxs, dWg, dWu, dWd, ws = A[:13]
    dxs = dy if over == "dy" else xs
    wanted = [(dWg, dWu, dWd), (None, None, dWd) if over == "dy" else (None, dWu, None)]
    for grads in wanted:
        assert L.mlp_moe_experts_bwd(ctypes.byref(p), plan, dy, xs, Wg, Wu, Wd, G, U, dxs, *grads,
                                     0, ws, 1 << 40, None) == -1


def test_experts_forward(L):
    p = m.moe(16, 8, 2, 64, 128)
    plan, xs, Wg, Wu, Wd, ws = A[:6]
    assert L.mlp_moe_experts_fwd(ctypes.byref(p), plan, xs, Wg, Wu, Wd, xs, None, None, ws, 1 << 40,
                                 None) == -1
