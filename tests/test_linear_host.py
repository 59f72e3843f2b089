"""Refusals of the linear layer's entry points (no GPU needed: fake,
never-dereferenced pointers; nothing is enqueued on a refusal)."""
import ctypes
import os
import re

import pytest
import torch

import activated_mlp_gemms_gb300 as m

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, BIG = 0x10000, 1 << 40


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(m.LIB_PATH):
        from activated_mlp_gemms_gb300 import _build
        _build.build()
    return m.lib()


def test_every_declared_symbol_is_exported(L):
    src = open(os.path.join(ROOT, "include", "mlp_linear.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = re.findall(r"^(?:int|size_t) (mlp_linear_[a-z0-9_]+)\(", src, flags=re.M)
    assert len(names) == 3
    for n in names:
        assert hasattr(L, n), n


OUT, PRE, DX = FAKE + 0x10000, FAKE + 0x20000, FAKE + 0x30000


def fwd(L, p, x=FAKE, W=FAKE, bias=FAKE, resid=FAKE, out=OUT, pre=PRE, ws=FAKE, n=BIG):
    return L.mlp_linear_fwd(ctypes.byref(p), x, W, bias, resid, out, pre, ws, n, None)


def bwd(L, p, dout=FAKE, x=FAKE, W=FAKE, pre=FAKE, dx=DX, dW=FAKE, db=FAKE, fuse=0, ws=FAKE,
        n=BIG):
    return L.mlp_linear_bwd(ctypes.byref(p), dout, x, W, pre, dx, dW, db, fuse, ws, n, None)


@pytest.mark.parametrize("change,code", [
    (dict(M=0), -1), (dict(N=-8), -1), (dict(K=0), -1), (dict(act=6), -1), (dict(act=-1), -1),
    (dict(resid_scale=float("inf")), -1), (dict(N=12), -2), (dict(K=100), -2), (dict(ldx=8), -1),
    (dict(ldx=132), -2), (dict(ldr=8), -1), (dict(ldo=258), -2), (dict(ldo=-256), -1),
    (dict(M=1 << 30, N=1 << 12), -3)])
def test_problem_refusals(L, change, code):
    p = m.linear(16, 256, 128, "silu")
    for k, v in change.items():
        setattr(p, k, v)
    assert m.mlp_linear_workspace_size(p) == 0 and m.mlp_linear_workspace_size(p, True) == 0
    assert fwd(L, p) == code and bwd(L, p) == code


def test_pointer_refusals(L):
    p = m.linear(16, 256, 128, "silu")
    for name in ("x", "W", "out"):
        assert fwd(L, p, **{name: None}) == -1
    for name in ("x", "W", "out", "bias", "resid", "pre"):
        assert fwd(L, p, **{name: FAKE + 8}) == -2
    for name in ("dout", "pre", "x", "W"):
        assert bwd(L, p, **{name: None}) == -1
    for name in ("dout", "pre", "x", "W", "dx", "dW", "db"):
        assert bwd(L, p, **{name: FAKE + 8}) == -2
    assert bwd(L, p, fuse=2) == -1
    # outputs over operands that are still read
    other = FAKE + 0x100000
    assert fwd(L, p, x=other, out=other) == -1 and fwd(L, p, x=other, pre=other) == -1
    assert bwd(L, p, dx=other, x=other) == -1 and bwd(L, p, dx=other, dout=other) == -1
    assert L.mlp_linear_fwd(None, FAKE, FAKE, None, None, FAKE, None, FAKE, BIG, None) == -1
    # nothing asked for: nothing to do
    assert bwd(L, p, x=None, W=None, dx=None, dW=None, db=None) == 0


def test_workspace(L):
    p = m.linear(16, 256, 128, "silu")
    for back, call in ((False, fwd), (True, bwd)):
        n = m.mlp_linear_workspace_size(p, back)
        assert n >= 1024
        assert call(L, p, n=n - 1) == -4
        assert call(L, p, ws=None) == -1
        assert call(L, p, ws=FAKE + 16) == -2
    assert L.mlp_linear_workspace_size(ctypes.byref(p), 2) == 0
    # large outputs need no split sums; an activation's backward holds dz
    big = m.linear(8192, 4096, 4096)
    assert m.mlp_linear_workspace_size(big) == 1024
    act = m.linear(8192, 4096, 4096, "relu")
    assert (m.mlp_linear_workspace_size(act, True) - m.mlp_linear_workspace_size(big, True)
            == 8192 * 4096 * 2)


def test_python_refusals():
    with pytest.raises(ValueError):
        m.linear(8, 8, 8, "tanh")
    p = m.linear(8, 8, 8)
    t = torch.zeros(8, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on the GPU
        m.mlp_linear_fwd(p, t, t, None, None, t)
