"""The layer norm with the residual sum in front of it (include/mlp_norm.h), and its
gradients:

    h = x + residual,   y = (h - mean) * rstd * weight + bias

Argument marshalling only.  x and residual of the forward may be row-pitched
views; the other tensors are contiguous.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import MlpError, _check, _stream, lib
from .router_op import _F32, _device, _rows, _tensor, _ws

_DTYPES = (torch.float32, torch.bfloat16)
_TYPES = {t: i for i, t in enumerate(_DTYPES)}
NORM_MAX_H = 16384  # MLP_NORM_MAX_H


class LayerNorm(ctypes.Structure):
    """mlp_layernorm_t"""
    _fields_ = [("M", ctypes.c_int), ("H", ctypes.c_int), ("eps", ctypes.c_float),
                ("type", ctypes.c_int), ("weight_type", ctypes.c_int), ("ldx", ctypes.c_int),
                ("ldr", ctypes.c_int)]


def declare(L):
    """Argument types of mlp_norm.h's functions (called when the library is loaded)."""
    P, VP = ctypes.POINTER(LayerNorm), ctypes.c_void_p
    L.mlp_layernorm_workspace_size.argtypes = [P]
    L.mlp_layernorm_workspace_size.restype = ctypes.c_size_t
    L.mlp_layernorm_fwd.argtypes = [P] + [VP] * 9
    L.mlp_layernorm_fwd.restype = ctypes.c_int
    L.mlp_layernorm_bwd.argtypes = [P] + [VP] * 9 + [ctypes.c_int, VP, ctypes.c_size_t, VP]
    L.mlp_layernorm_bwd.restype = ctypes.c_int


def layernorm(M, H, eps=1e-5, dtype=torch.bfloat16, weight_dtype=torch.bfloat16) -> LayerNorm:
    """The problem: M rows of H values; the type of the rows, and of weight and bias.  (The row
    pitches come from the tensors of each call.)"""
    for t, name in ((dtype, "dtype"), (weight_dtype, "weight_dtype")):
        if t not in _TYPES:
            raise ValueError(f"{name} must be torch.float32 or torch.bfloat16")
    return LayerNorm(int(M), int(H), float(eps), _TYPES[dtype], _TYPES[weight_dtype], 0, 0)


def mlp_layernorm_workspace_size(p: LayerNorm) -> int:
    return int(lib().mlp_layernorm_workspace_size(ctypes.byref(p)))


@functools.lru_cache(maxsize=1024)
def _ws_size(M, H, kind):
    """The workspace size: a function of the sizes and the rows' type."""
    return mlp_layernorm_workspace_size(LayerNorm(M, H, 0.0, kind, 0, 0, 0))


def alloc_layernorm_workspace(p: LayerNorm, device=None) -> torch.Tensor:
    n = mlp_layernorm_workspace_size(p)
    if n == 0:
        raise MlpError(-1, "mlp_layernorm_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def mlp_layernorm_fwd(p: LayerNorm, x, residual, weight, bias, y, h=None, mean=None, rstd=None,
                      stream=None) -> None:
    """y = LayerNorm(x + residual) (residual, weight and bias may be None); h receives the sum,
    mean and rstd (fp32 [M]) the rows' statistics: what the backward takes."""
    dev, mh = _device(), (p.M, p.H)
    dt, wt = _DTYPES[p.type == 1], (_DTYPES[p.weight_type == 1],)
    f32 = _F32
    xp, ldx = _rows(x, mh, dt, "x", dev)
    rp, ldr = _rows(residual, mh, dt, "residual", dev)
    q = p
    if ldx or ldr or p.ldx or p.ldr:
        q = LayerNorm(p.M, p.H, p.eps, p.type, p.weight_type, ldx, ldr)
    rc = lib().mlp_layernorm_fwd(
        ctypes.byref(q), xp, rp, _tensor(weight, (p.H,), wt, "weight", dev),
        _tensor(bias, (p.H,), wt, "bias", dev), _tensor(y, mh, (dt,), "y", dev),
        _tensor(h, mh, (dt,), "h", dev), _tensor(mean, (p.M,), f32, "mean", dev),
        _tensor(rstd, (p.M,), f32, "rstd", dev), _stream(stream))
    _check(rc, "mlp_layernorm_fwd")


def mlp_layernorm_bwd(p: LayerNorm, dy, h, weight, mean, rstd, dh=None, dx=None, dweight=None,
                      dbias=None, fuse_grad_accum=False, ws=None, stream=None):
    """dx = dh + the gradient through the norm (of x and of residual alike), and the gradients
    of weight and bias: in their type, or added to fp32 with fuse_grad_accum.  h is the
    forward's (its x without a residual); outputs that are None are skipped.  Returns the
    workspace used (None without dweight and dbias)."""
    dev, mh = _device(), (p.M, p.H)
    dt, wt = (_DTYPES[p.type == 1],), (_DTYPES[p.weight_type == 1],)
    f32 = _F32
    gt = f32 if fuse_grad_accum else wt
    args = (_tensor(dy, mh, dt, "dy", dev), _tensor(h, mh, dt, "h", dev),
            _tensor(weight, (p.H,), wt, "weight", dev), _tensor(mean, (p.M,), f32, "mean", dev),
            _tensor(rstd, (p.M,), f32, "rstd", dev), _tensor(dh, mh, dt, "dh", dev),
            _tensor(dx, mh, dt, "dx", dev), _tensor(dweight, (p.H,), gt, "dweight", dev),
            _tensor(dbias, (p.H,), gt, "dbias", dev))
    if dweight is None and dbias is None:
        ws, at = None, (None, 0)
    else:
        ws = _ws(ws, _ws_size(p.M, p.H, p.type), dy.device, stream)
        at = (ws.data_ptr(), ws.numel())
    rc = lib().mlp_layernorm_bwd(ctypes.byref(p), *args, int(bool(fuse_grad_accum)), *at,
                                 _stream(stream))
    _check(rc, "mlp_layernorm_bwd")
    return ws
