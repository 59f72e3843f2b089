"""Outputs of the router's calls over operands that other tokens still read, or over each other,
are refused (no GPU needed: fake, never-dereferenced pointers; nothing is enqueued on a refusal)."""
import ctypes
import os

import pytest

import activated_mlp_gemms_gb300 as m

A = [0x100000 * (i + 1) for i in range(9)]  # distinct operands


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(m.LIB_PATH):
        from activated_mlp_gemms_gb300 import _build
        _build.build()
    return m.lib()


NAMES = ("logits", "mask", "ids", "weights", "counts", "balance")


@pytest.mark.parametrize("out,over", [(o, i) for o in NAMES[2:] for i in NAMES if i != o])
def test_forward(L, out, over):
    at = dict(zip(NAMES, A))
    at[out] = at[over]
    p = m.router(16, 8, 2)
    assert L.mlp_moe_router_fwd(ctypes.byref(p), *(at[n] for n in NAMES), A[7], 1 << 40, None) == -1


@pytest.mark.parametrize("over", ["mask", "ids", "balance", "dweights", "dloss"])
def test_backward(L, over):
    names = ("logits", "mask", "ids", "balance", "dweights", "dloss")
    at = dict(zip(names, A))
    p = m.router(16, 8, 2)
    assert L.mlp_moe_router_bwd(ctypes.byref(p), *(at[n] for n in names), at[over], None) == -1
