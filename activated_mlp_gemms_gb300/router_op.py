"""The router of a mixture of experts (include/mlp_router.h): a token's experts and
their weights from its logits, the experts' counts, the balance loss, and the
logits' gradient.

Argument marshalling only.  logits and dlogits may be row-pitched views (unit
stride along the last dimension: the first E columns of a padded linear layer's
output); the other tensors are contiguous.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import MlpError, _call_workspace, _check, _stream, lib

_DTYPES = (torch.float32, torch.bfloat16)
_TYPES = {t: i for i, t in enumerate(_DTYPES)}
_T = torch.Tensor
_I32, _F32, _BOOL = (torch.int32,), (torch.float32,), (torch.bool, torch.uint8)


class Router(ctypes.Structure):
    """mlp_router_t"""
    _fields_ = [(n, ctypes.c_int) for n in ("T", "E", "top_k", "renormalize", "logits_type",
                                            "weights_type", "ldl", "ldd")]


def declare(L):
    """Argument types of mlp_router.h's functions (called when the library is loaded)."""
    P, VP = ctypes.POINTER(Router), ctypes.c_void_p
    L.mlp_moe_router_workspace_size.argtypes = [P]
    L.mlp_moe_router_workspace_size.restype = ctypes.c_size_t
    L.mlp_moe_router_fwd.argtypes = [P] + [VP] * 7 + [ctypes.c_size_t, VP]
    L.mlp_moe_router_fwd.restype = ctypes.c_int
    L.mlp_moe_router_bwd.argtypes = [P] + [VP] * 8
    L.mlp_moe_router_bwd.restype = ctypes.c_int


def router(T, E, top_k, renormalize=True, logits_dtype=torch.float32,
           weights_dtype=torch.float32) -> Router:
    """The problem: T tokens, E experts, top_k slots a token; whether a token's weights are
    divided by their sum; the types.  (The row pitches come from the tensors of each call.)"""
    for t, name in ((logits_dtype, "logits_dtype"), (weights_dtype, "weights_dtype")):
        if t not in _TYPES:
            raise ValueError(f"{name} must be torch.float32 or torch.bfloat16")
    return Router(int(T), int(E), int(top_k), int(bool(renormalize)), _TYPES[logits_dtype],
                  _TYPES[weights_dtype], 0, 0)


def _tensor(t, shape, dtypes, name, device):
    """The tensor's address (None stays None) once its type, device, shape and strides are
    right: dense."""
    if t is None:
        return None
    if (t.__class__ is _T and t.dtype in dtypes and t.shape == shape and t.get_device() == device
            and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda or t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor on the current device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, shape, dtype, name, device):
    """(address, row pitch or 0 when dense) of a matrix with unit column stride."""
    if (t.__class__ is _T and t.dtype is dtype and t.shape == shape and t.get_device() == device
            and t.is_contiguous()):
        return t.data_ptr(), 0
    if not isinstance(t, torch.Tensor) or t.is_contiguous() or t.shape != shape:
        return _tensor(t, shape, (dtype,), name, device), 0
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor on the current device")
    if (shape[1] > 1 and t.stride(1) != 1) or t.stride(0) < shape[1]:
        raise ValueError(f"{name} must have unit stride along its last dimension and rows "
                         "that do not overlap")
    if t.stride(0) > 0x7fffffff:  # the C ABI's int; ctypes would wrap it
        raise ValueError(f"{name}'s row stride of {t.stride(0)} passes 32 bits")
    return t.data_ptr(), t.stride(0)


def _pitched(p, ldl, ldd):
    if not (ldl or ldd or p.ldl or p.ldd):
        return p
    return Router(p.T, p.E, p.top_k, p.renormalize, p.logits_type, p.weights_type, ldl, ldd)


def _device():
    return torch._C._cuda_getDevice()


def mlp_moe_router_workspace_size(p: Router) -> int:
    return int(lib().mlp_moe_router_workspace_size(ctypes.byref(p)))


def alloc_router_workspace(p: Router, device=None) -> torch.Tensor:
    n = mlp_moe_router_workspace_size(p)
    if n == 0:
        raise MlpError(-1, "mlp_moe_router_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


@functools.lru_cache(maxsize=1024)
def _ws_size(T, E, top_k):
    """The workspace size: a function of the sizes alone."""
    return mlp_moe_router_workspace_size(Router(T, E, top_k, 0, 0, 0, 0, 0))


def _ws(ws, size, device, stream):
    if ws is None:  # (of a problem that the call refuses: any)
        return _call_workspace(size or 256, device, stream)
    if not (ws.is_cuda and ws.dtype == torch.uint8 and ws.is_contiguous()
            and ws.get_device() == device.index):
        raise ValueError("workspace must be a contiguous CUDA uint8 tensor on the current device")
    return ws


def mlp_moe_router_fwd(p: Router, logits, mask, ids, weights, counts=None, balance=None, ws=None,
                       stream=None):
    """ids int32 [T, top_k] and weights [T, top_k] of the top_k largest logits [T, E]; mask
    (bool or uint8 [T], or None) is zero for tokens that are not routed: ids -1, weights 0.
    counts int32 [E] receives the slots of each expert, balance fp32 [E + 1] the balance loss
    and, behind it, its derivative by each expert's probability (for the backward).  Returns
    the workspace used (None without counts and balance)."""
    dev = _device()
    ld, wd = _DTYPES[p.logits_type == 1], _DTYPES[p.weights_type == 1]
    slots = (p.T, p.top_k)
    lp, ldl = _rows(logits, (p.T, p.E), ld, "logits", dev)
    q = _pitched(p, ldl, 0)
    args = (lp, _tensor(mask, (p.T,), _BOOL, "mask", dev),
            _tensor(ids, slots, _I32, "ids", dev),
            _tensor(weights, slots, (wd,), "weights", dev),
            _tensor(counts, (p.E,), _I32, "counts", dev),
            _tensor(balance, (p.E + 1,), _F32, "balance", dev))
    if counts is None and balance is None:
        ws, at = None, (None, 0)
    else:
        ws = _ws(ws, _ws_size(p.T, p.E, p.top_k), ids.device, stream)
        at = (ws.data_ptr(), ws.numel())
    _check(lib().mlp_moe_router_fwd(ctypes.byref(q), *args, *at, _stream(stream)),
           "mlp_moe_router_fwd")
    return ws


def mlp_moe_router_bwd(p: Router, logits, mask, ids, balance, dweights, dloss, dlogits,
                       stream=None) -> None:
    """dlogits [T, E] from the gradients of the weights (dweights [T, top_k] or None) and of the
    loss (dloss fp32 [1] on the device, or None; it needs the forward's balance)."""
    dev = _device()
    ld, wd = _DTYPES[p.logits_type == 1], _DTYPES[p.weights_type == 1]
    slots = (p.T, p.top_k)
    lp, ldl = _rows(logits, (p.T, p.E), ld, "logits", dev)
    dp, ldd = _rows(dlogits, (p.T, p.E), ld, "dlogits", dev)
    q = _pitched(p, ldl, ldd)
    if dloss is not None and dloss.dim() == 0:
        dloss = dloss.reshape(1)
    rc = lib().mlp_moe_router_bwd(
        ctypes.byref(q), lp, _tensor(mask, (p.T,), _BOOL, "mask", dev),
        _tensor(ids, slots, _I32, "ids", dev),
        _tensor(balance, (p.E + 1,), _F32, "balance", dev),
        _tensor(dweights, slots, (wd,), "dweights", dev),
        _tensor(dloss, (1,), _F32, "dloss", dev), dp, _stream(stream))
    _check(rc, "mlp_moe_router_bwd")
