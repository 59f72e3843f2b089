"""Outputs of the layer norm's calls over operands that other rows still read, or over each other,
are refused (no GPU needed: fake, never-dereferenced pointers; nothing is enqueued on a refusal)."""
import ctypes
import os

import pytest

import activated_mlp_gemms_gb300 as m

A = [0x100000 * (i + 1) for i in range(12)]  # distinct operands
FWD = ("x", "residual", "weight", "bias", "y", "h", "mean", "rstd")
BWD = ("dy", "h", "weight", "mean", "rstd", "dh", "dx", "dweight", "dbias")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(m.LIB_PATH):
        from activated_mlp_gemms_gb300 import _build
        _build.build()
    return m.lib()


def place(names, out, over):
    at = dict(zip(names, A))
    at[out] = at[over]
    return [at[n] for n in names]


@pytest.mark.parametrize("out,over", [(o, i) for o in FWD[4:] for i in FWD if i != o and not (
    o in ("y", "h") and i in ("x", "residual"))])  # (these may be)
def test_forward(L, out, over):
    p = m.layernorm(16, 64)
    assert L.mlp_layernorm_fwd(ctypes.byref(p), *place(FWD, out, over), None) == -1


@pytest.mark.parametrize("out,over", [("dx", i) for i in ("h", "weight", "mean", "rstd", "dweight",
                                                          "dbias")] + [("dweight", "dbias")])
def test_backward(L, out, over):
    p = m.layernorm(16, 64)
    assert L.mlp_layernorm_bwd(ctypes.byref(p), *place(BWD, out, over), 0, A[10], 1 << 40,
                               None) == -1
