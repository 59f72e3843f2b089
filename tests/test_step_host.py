"""Refusals of the router's, the layer norm's and the orthogonalisation's entry points (no GPU
needed: fake, never-dereferenced pointers; nothing is enqueued on a refusal)."""
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


@pytest.mark.parametrize("header,prefix,n", [("mlp_router.h", "mlp_moe_router_", 3),
                                             ("mlp_norm.h", "mlp_layernorm_", 3),
                                             ("mlp_ortho.h", "mlp_ortho", 2)])
def test_every_declared_symbol_is_exported(L, header, prefix, n):
    src = open(os.path.join(ROOT, "include", header)).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = re.findall(rf"^(?:int|size_t) ({prefix}[a-z0-9_]+)\(", src, flags=re.M)
    assert len(names) == n
    for name in names:
        assert hasattr(L, name), name


# ------------------------------------------------------------------ router

def rfwd(L, p, logits=FAKE, mask=None, ids=FAKE, w=FAKE, counts=FAKE, balance=FAKE, ws=FAKE, n=BIG):
    return L.mlp_moe_router_fwd(ctypes.byref(p), logits, mask, ids, w, counts, balance, ws, n, None)


def rbwd(L, p, logits=FAKE, mask=None, ids=FAKE, balance=FAKE, dw=FAKE, dloss=FAKE,
         dlogits=FAKE + 0x10000):
    return L.mlp_moe_router_bwd(ctypes.byref(p), logits, mask, ids, balance, dw, dloss, dlogits,
                                None)


@pytest.mark.parametrize("change,code", [
    (dict(T=0), -1), (dict(T=-5), -1), (dict(E=0), -1), (dict(top_k=0), -1), (dict(top_k=9), -1),
    (dict(renormalize=2), -1), (dict(logits_type=2), -1), (dict(weights_type=-1), -1),
    (dict(ldl=7), -1), (dict(ldd=4), -1), (dict(ldl=-8), -1), (dict(E=1025), -3),
    (dict(E=128, top_k=65), -3), (dict(T=1 << 30), -3)])
def test_router_problem_refusals(L, change, code):
    p = m.router(16, 8, 2)
    for k, v in change.items():
        setattr(p, k, v)
    assert m.mlp_moe_router_workspace_size(p) == 0
    assert rfwd(L, p) == code and rbwd(L, p) == code
    with pytest.raises(m.MlpError):
        m.alloc_router_workspace(p)


def test_router_pointer_refusals(L):
    p = m.router(16, 8, 2)
    for name in ("logits", "ids", "w"):
        assert rfwd(L, p, **{name: None}) == -1
    for name in ("logits", "ids", "w", "counts", "balance"):
        assert rfwd(L, p, **{name: FAKE + 2}) == -2
    assert rfwd(L, p, ws=None) == -1 and rfwd(L, p, ws=FAKE + 64) == -2
    assert rfwd(L, p, n=m.mlp_moe_router_workspace_size(p) - 1) == -4
    half = m.router(16, 8, 2, logits_dtype=torch.bfloat16, weights_dtype=torch.bfloat16)
    assert rfwd(L, half, logits=FAKE + 1) == -2 and rfwd(L, half, w=FAKE + 1) == -2
    for name in ("logits", "ids", "balance", "dlogits"):
        assert rbwd(L, p, **{name: None}) == -1
    for name in ("logits", "ids", "balance", "dw", "dloss", "dlogits"):
        assert rbwd(L, p, **{name: FAKE + 2}) == -2
    # the gradient over the logits: rows at the same places only
    p.ldl = 16
    assert rbwd(L, p, dlogits=FAKE) == -1
    assert L.mlp_moe_router_fwd(None, FAKE, None, FAKE, FAKE, None, None, None, 0, None) == -1


# -------------------------------------------------------------- layer norm

def nfwd(L, p, x=FAKE, r=FAKE, w=FAKE, b=FAKE, y=FAKE + 0x10000, h=FAKE + 0x20000, mean=FAKE,
         rstd=FAKE):
    return L.mlp_layernorm_fwd(ctypes.byref(p), x, r, w, b, y, h, mean, rstd, None)


def nbwd(L, p, dy=FAKE, h=FAKE, w=FAKE, mean=FAKE, rstd=FAKE, dh=FAKE, dx=FAKE + 0x10000, dw=FAKE,
         db=FAKE, fuse=0, ws=FAKE, n=BIG):
    return L.mlp_layernorm_bwd(ctypes.byref(p), dy, h, w, mean, rstd, dh, dx, dw, db, fuse, ws, n,
                               None)


@pytest.mark.parametrize("change,code", [
    (dict(M=0), -1), (dict(H=0), -1), (dict(H=-8), -1), (dict(eps=-1e-5), -1),
    (dict(eps=float("nan")), -1), (dict(type=2), -1), (dict(weight_type=5), -1), (dict(ldx=56), -1),
    (dict(ldr=-64), -1), (dict(H=60), -2), (dict(ldx=68), -2), (dict(H=16392), -3)])
def test_norm_problem_refusals(L, change, code):
    p = m.layernorm(16, 64)
    for k, v in change.items():
        setattr(p, k, v)
    assert m.mlp_layernorm_workspace_size(p) == 0
    assert nfwd(L, p) == code and nbwd(L, p) == code
    with pytest.raises(m.MlpError):
        m.alloc_layernorm_workspace(p)


def test_norm_pointer_refusals(L):
    p = m.layernorm(16, 64)
    for name in ("x", "y"):
        assert nfwd(L, p, **{name: None}) == -1
    for name in ("x", "r", "w", "b", "y", "h"):
        assert nfwd(L, p, **{name: FAKE + 8}) == -2
    for name in ("mean", "rstd"):
        assert nfwd(L, p, **{name: FAKE + 2}) == -2
    other = FAKE + 0x100000
    assert nfwd(L, p, y=other, h=other) == -1
    q = m.layernorm(16, 64)
    q.ldx = 128  # a pitched input under a dense output
    assert nfwd(L, q, x=other, y=other) == -1 and nfwd(L, q, x=other, h=other) == -1
    for name in ("dy", "h", "mean", "rstd"):
        assert nbwd(L, p, **{name: None}) == -1
    for name in ("dy", "h", "w", "dh", "dx", "dw", "db"):
        assert nbwd(L, p, **{name: FAKE + 8}) == -2
    assert nbwd(L, p, fuse=2) == -1 and nbwd(L, p, h=other, dx=other) == -1
    assert nbwd(L, p, ws=None) == -1 and nbwd(L, p, ws=FAKE + 64) == -2
    assert nbwd(L, p, n=m.mlp_layernorm_workspace_size(p) - 1) == -4
    # nothing asked for: nothing to do
    assert nbwd(L, p, dx=None, dw=None, db=None, ws=None, n=0) == 0


# ------------------------------------------------------------------- python

def test_python_refusals():
    for bad in (dict(logits_dtype=torch.float16), dict(weights_dtype=torch.float64)):
        with pytest.raises(ValueError):
            m.router(4, 4, 1, **bad)
    with pytest.raises(ValueError):
        m.layernorm(4, 8, dtype=torch.float16)
    t = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        m.router_func([1.0], 1)
    with pytest.raises(ValueError):  # not on the GPU
        m.router_func(t, 2)
    with pytest.raises(ValueError):
        m.layer_norm_func(t)
    with pytest.raises(TypeError):
        m.layer_norm_func(None)


# ----------------------------------------------------------- orthogonalisation

def ortho(L, p, G=FAKE, out=FAKE + 0x10000, ws=FAKE, n=BIG):
    return L.mlp_orthogonalize(ctypes.byref(p), G, out, ws, n, None)


@pytest.mark.parametrize("change,code", [
    (dict(rows=0), -1), (dict(cols=-8), -1), (dict(batch=0), -1), (dict(steps=0), -1),
    (dict(steps=33), -1), (dict(coeff=(float("nan"), 0, 0)), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("inf")), -1), (dict(scale=float("nan")), -1), (dict(type=2), -1),
    (dict(out_type=-1), -1), (dict(rows=12), -2), (dict(cols=100), -2),
    (dict(rows=40000, cols=40000), -3), (dict(rows=8, cols=1 << 22), -3),
    (dict(batch=65536), -3), (dict(rows=32768, cols=32768, batch=65), -3)])
def test_ortho_problem_refusals(L, change, code):
    p = m.ortho(64, 128)
    for k, v in change.items():
        setattr(p, k, type(p.coeff)(*v) if k == "coeff" else v)
    assert m.mlp_ortho_workspace_size(p) == 0
    assert ortho(L, p) == code
    with pytest.raises(m.MlpError):
        m.alloc_ortho_workspace(p)


def test_ortho_pointer_refusals(L):
    p = m.ortho(64, 128)
    assert ortho(L, p, G=None) == -1 and ortho(L, p, out=None) == -1
    assert ortho(L, p, G=FAKE + 8) == -2 and ortho(L, p, out=FAKE + 8) == -2
    assert ortho(L, p, ws=None) == -1 and ortho(L, p, ws=FAKE + 64) == -2
    assert ortho(L, p, n=m.mlp_ortho_workspace_size(p) - 1) == -4
    q = m.ortho(64, 128, out_dtype=torch.float32)
    assert ortho(L, q, G=FAKE, out=FAKE) == -1  # the result over an update of another type
    assert L.mlp_orthogonalize(None, FAKE, FAKE, FAKE, BIG, None) == -1
    # X twice in two fp16 terms, A and the polynomial in one or two
    assert m.mlp_ortho_workspace_size(p) == 1024 + 1024 + 2 * 64 * 128 * 4 + 2 * 64 * 64 * 2
    assert m.mlp_ortho_workspace_size(q) == m.mlp_ortho_workspace_size(p) + 2 * 64 * 64 * 2
    with pytest.raises(ValueError):
        m.ortho(64, 64, dtype=torch.float16)
