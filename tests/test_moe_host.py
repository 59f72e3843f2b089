"""Refusals of the mixture-of-experts entry points (no GPU needed: fake,
never-dereferenced pointers; nothing is enqueued on a refusal)."""
import ctypes
import os
import re

import pytest
import torch

import activated_mlp_gemms_gb300 as m
from activated_mlp_gemms_gb300 import experts as moe_mod

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(m.LIB_PATH):
        from activated_mlp_gemms_gb300 import _build
        _build.build()
    return m.lib()


def test_every_declared_symbol_is_exported(L):
    src = open(os.path.join(ROOT, "include", "mlp_moe.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = re.findall(r"^(?:int|long long|size_t) (mlp_moe_[a-z0-9_]+)\(", src, flags=re.M)
    assert len(names) >= 7
    for n in names:
        assert hasattr(L, n), n


@pytest.mark.parametrize("change,code", [
    (dict(T=0), -1), (dict(E=0), -1), (dict(top_k=0), -1), (dict(H=0), -1), (dict(T=-3), -1),
    (dict(weights_type=2), -1), (dict(H=12), -2), (dict(E=1025), -3), (dict(top_k=65), -3),
    (dict(T=1 << 30), -3)])
def test_problem_refusals(L, change, code):
    p = m.moe(16, 8, 2, 64)
    for k, v in change.items():
        setattr(p, k, v)
    b = ctypes.byref(p)
    assert L.mlp_moe_rows(b) == 0
    assert L.mlp_moe_plan_layout(b, ctypes.byref(moe_mod._Layout())) == code
    assert L.mlp_moe_sort(b, FAKE, FAKE, None) == code
    assert L.mlp_moe_dispatch(b, FAKE, FAKE, FAKE, None) == code
    assert L.mlp_moe_dispatch_bwd(b, FAKE, FAKE, FAKE, None) == code
    assert L.mlp_moe_combine(b, FAKE, FAKE, FAKE, None, FAKE, None) == code
    assert L.mlp_moe_combine_bwd(b, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == code
    with pytest.raises(m.MlpError):
        m.mlp_moe_rows(p)


def test_pointer_refusals(L):
    b = ctypes.byref(m.moe(16, 8, 2, 64))
    assert L.mlp_moe_rows(None) == 0
    assert L.mlp_moe_sort(None, FAKE, FAKE, None) == -1
    assert L.mlp_moe_sort(b, None, FAKE, None) == -1
    assert L.mlp_moe_sort(b, FAKE, None, None) == -1
    assert L.mlp_moe_sort(b, FAKE + 2, FAKE, None) == -2
    assert L.mlp_moe_sort(b, FAKE, FAKE + 4, None) == -2
    assert L.mlp_moe_plan_layout(b, None) == -1
    for i in range(3):
        for bad, code in ((None, -1), (FAKE + 2, -2)):
            a = [FAKE] * 3
            a[i] = bad
            assert L.mlp_moe_dispatch(b, *a, None) == code
            assert L.mlp_moe_dispatch_bwd(b, *a, None) == code
    assert L.mlp_moe_combine(b, FAKE, None, FAKE, None, FAKE, None) == -1
    assert L.mlp_moe_combine(b, FAKE, FAKE, None, None, FAKE, None) == -1
    assert L.mlp_moe_combine(b, FAKE, FAKE, FAKE, FAKE + 8, FAKE, None) == -2
    assert L.mlp_moe_combine(b, FAKE, FAKE, FAKE, None, None, None) == -1
    # dy needs the weights, dweights needs y; neither wanted: nothing to do
    assert L.mlp_moe_combine_bwd(b, FAKE, FAKE, FAKE, None, FAKE, None, None) == -1
    assert L.mlp_moe_combine_bwd(b, FAKE, FAKE, None, FAKE, None, FAKE, None) == -1
    assert L.mlp_moe_combine_bwd(b, FAKE, FAKE, None, None, None, None, None) == 0


def test_layout(L):
    p = m.moe(3, 5, 2, 64)
    assert m.mlp_moe_rows(p) == (6 + 5 * 15) // 16 * 16
    assert m.mlp_moe_rows(m.moe(1, 64, 1, 64)) == 16
    lay = moe_mod._layout(p)
    parts = sorted([(lay.offsets, 6), (lay.counts, 5), (lay.pos, 6), (lay.src, 80)])
    for (a, n), (b, _) in zip(parts, parts[1:] + [(lay.ints, 0)]):
        assert a % 4 == 0 and a + n <= b


def test_python_refusals(L):
    with pytest.raises(ValueError):
        m.moe(4, 4, 1, 64, act="tanh")
    with pytest.raises(ValueError):
        m.moe(4, 4, 1, 64, weights_dtype=torch.float16)
    p = m.moe(4, 4, 1, 64)
    with pytest.raises(ValueError):  # not on the GPU
        m.mlp_moe_sort(p, torch.zeros(4, 1, dtype=torch.int32),
                       torch.zeros(10, dtype=torch.int32))
