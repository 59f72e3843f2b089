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


def _experts(L, p, plan=FAKE, xs=FAKE, Wg=FAKE, Wu=FAKE, Wd=FAKE, y=FAKE, G=FAKE, U=FAKE, ws=FAKE,
             n=1 << 40):
    return L.mlp_moe_experts_fwd(ctypes.byref(p), plan, xs, Wg, Wu, Wd, y, G, U, ws, n, None)


def _experts_bwd(L, p, plan=FAKE, dy=FAKE, xs=FAKE, Wg=FAKE, Wu=FAKE, Wd=FAKE, G=FAKE, U=FAKE,
                 dxs=FAKE, dWg=FAKE, dWu=FAKE, dWd=FAKE, fuse=0, ws=FAKE, n=1 << 40):
    return L.mlp_moe_experts_bwd(ctypes.byref(p), plan, dy, xs, Wg, Wu, Wd, G, U, dxs, dWg, dWu,
                                 dWd, fuse, ws, n, None)


def _layer(L, p, x=FAKE, ids=FAKE, w=FAKE, Wg=FAKE, Wu=FAKE, Wd=FAKE, r=None, out=FAKE, ws=FAKE,
           n=1 << 40):
    return L.mlp_moe_fwd_infer(ctypes.byref(p), x, ids, w, Wg, Wu, Wd, r, out, ws, n, None)


def test_experts_refusals(L):
    ok = lambda **kw: m.moe(16, 8, 2, 64, 128, **kw)  # noqa: E731
    calls = (_experts, _experts_bwd, _layer)
    for change, code in ((dict(I=0), -1), (dict(act=7), -1), (dict(I=100), -2), (dict(H=20), -2),
                         (dict(gate_mult=float("nan")), -1), (dict(T=0), -1), (dict(E=2000), -3)):
        p = ok()
        for k, v in change.items():
            setattr(p, k, v)
        for call in calls:
            assert call(L, p) == code, (change, call)
        assert m.mlp_moe_workspace_size(p, m.MODE_FWD) == 0
    p, q = ok(), ok(act="relu_sq")
    for call in calls:
        assert call(L, q) == -1  # a non-gated MLP takes no Wu
        assert call(L, p, Wu=None) == -1
        assert call(L, p, Wg=FAKE + 8) == -2
        assert call(L, p, ws=None) == -1
        assert call(L, p, ws=FAKE + 16) == -2
        assert call(L, p, n=2048) == -4
    for name in ("plan", "xs", "Wg", "Wd", "y"):
        assert _experts(L, p, **{name: None}) == -1
    assert _experts(L, q, Wu=None, G=FAKE, U=FAKE) == -1  # no up preact without an up weight
    assert _experts(L, p, G=FAKE + 4) == -2
    for name in ("plan", "dy", "xs", "Wg", "Wd", "G", "U"):
        assert _experts_bwd(L, p, **{name: None}) == -1
    assert _experts_bwd(L, p, fuse=2) == -1
    assert _experts_bwd(L, p, dWd=FAKE + 4) == -2
    assert _experts_bwd(L, q, Wu=None, U=None, dWu=FAKE) == -1
    assert _experts_bwd(L, p, dxs=None, dWg=None, dWu=None, dWd=None) == 0  # nothing asked for
    for name in ("x", "ids", "w", "out"):
        assert _layer(L, p, **{name: None}) == -1
    assert _layer(L, p, r=FAKE + 8) == -2
    assert m.mlp_moe_workspace_size(p, m.MODE_BWD_RECOMPUTE) == 0
    rows = m.mlp_moe_rows(p)
    assert m.mlp_moe_workspace_size(p, m.MODE_FWD) == 1024 + rows * 128 * 2
