"""An update made orthogonal by Newton-Schulz products (include/mlp_ortho.h), as the
Muon optimiser does with a linear layer's: one matrix, or a stack of them (the
experts').

Argument marshalling only.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import MlpError, _check, _stream, lib
from .router_op import _device, _tensor, _ws

_DTYPES = (torch.float32, torch.bfloat16)
_TYPES = {t: i for i, t in enumerate(_DTYPES)}
MUON_COEFFS = (3.4445, -4.7750, 2.0315)


class Ortho(ctypes.Structure):
    """mlp_ortho_t"""
    _fields_ = [("rows", ctypes.c_int), ("cols", ctypes.c_int), ("batch", ctypes.c_int),
                ("steps", ctypes.c_int), ("coeff", ctypes.c_float * 3), ("eps", ctypes.c_float),
                ("scale", ctypes.c_float), ("type", ctypes.c_int), ("out_type", ctypes.c_int)]


def declare(L):
    """Argument types of mlp_ortho.h's functions (called when the library is loaded)."""
    P, VP = ctypes.POINTER(Ortho), ctypes.c_void_p
    L.mlp_ortho_workspace_size.argtypes = [P]
    L.mlp_ortho_workspace_size.restype = ctypes.c_size_t
    L.mlp_orthogonalize.argtypes = [P, VP, VP, VP, ctypes.c_size_t, VP]
    L.mlp_orthogonalize.restype = ctypes.c_int


def ortho(rows, cols, batch=1, steps=5, coeffs=MUON_COEFFS, eps=1e-7, scale=1.0,
          dtype=torch.bfloat16, out_dtype=torch.bfloat16) -> Ortho:
    """The problem: a stack of `batch` matrices [rows, cols], `steps` Newton-Schulz steps with
    coefficients a, b, c; the types of the update and of the result."""
    for t, name in ((dtype, "dtype"), (out_dtype, "out_dtype")):
        if t not in _TYPES:
            raise ValueError(f"{name} must be torch.float32 or torch.bfloat16")
    a, b, c = (float(v) for v in coeffs)
    return Ortho(int(rows), int(cols), int(batch), int(steps), (a, b, c), float(eps),
                 float(scale), _TYPES[dtype], _TYPES[out_dtype])


def mlp_ortho_workspace_size(p: Ortho) -> int:
    return int(lib().mlp_ortho_workspace_size(ctypes.byref(p)))


@functools.lru_cache(maxsize=1024)
def _ws_size(rows, cols, batch, out_type):
    """The workspace size: a function of the sizes and the result's type."""
    return mlp_ortho_workspace_size(Ortho(rows, cols, batch, 1, (1, 0, 0), 0, 1, 0, out_type))


def alloc_ortho_workspace(p: Ortho, device=None) -> torch.Tensor:
    n = mlp_ortho_workspace_size(p)
    if n == 0:
        raise MlpError(-1, "mlp_ortho_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def mlp_orthogonalize(p: Ortho, G, out, ws=None, stream=None):
    """out = scale * X after the steps from X = G / (|G| + eps), for each matrix of the stack:
    G and out [batch, rows, cols], or [rows, cols] with a batch of one; out may be G itself
    where the types are the same.  Returns the workspace used."""
    dev = _device()
    shape = (p.batch, p.rows, p.cols)
    if p.batch == 1 and isinstance(G, torch.Tensor) and G.dim() == 2:
        shape = (p.rows, p.cols)
    args = (_tensor(G, shape, (_DTYPES[p.type == 1],), "G", dev),
            _tensor(out, shape, (_DTYPES[p.out_type == 1],), "out", dev))
    ws = _ws(ws, _ws_size(p.rows, p.cols, p.batch, p.out_type), G.device, stream)
    rc = lib().mlp_orthogonalize(ctypes.byref(p), *args, ws.data_ptr(), ws.numel(),
                                 _stream(stream))
    _check(rc, "mlp_orthogonalize")
    return ws
