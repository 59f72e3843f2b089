"""The linear layer with bias, activation and residual in its epilogue
(include/mlp_linear.h), and its gradients.

    z = x W^T + bias,   out = act(z) + resid_scale * residual

Argument marshalling only.  x, residual, out and dout may be row-pitched
views (unit stride along the last dimension, a row stride that is a multiple
of 8); the other tensors are contiguous.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import MlpError, _call_workspace, _check, _ptr, _stream, lib

LINEAR_ACTS = {"none": 0, "relu": 1, "relu_sq": 2, "gelu_tanh_approx": 3, "silu": 4, "sigmoid": 5}


class Linear(ctypes.Structure):
    """mlp_linear_t"""
    _fields_ = [("M", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("act", ctypes.c_int), ("resid_scale", ctypes.c_float), ("ldx", ctypes.c_int),
                ("ldr", ctypes.c_int), ("ldo", ctypes.c_int)]


def declare(L):
    """Argument types of mlp_linear.h's functions (called when the library is loaded)."""
    P, VP = ctypes.POINTER(Linear), ctypes.c_void_p
    L.mlp_linear_workspace_size.argtypes = [P, ctypes.c_int]
    L.mlp_linear_workspace_size.restype = ctypes.c_size_t
    L.mlp_linear_fwd.argtypes = [P] + [VP] * 7 + [ctypes.c_size_t, VP]
    L.mlp_linear_fwd.restype = ctypes.c_int
    L.mlp_linear_bwd.argtypes = [P] + [VP] * 7 + [ctypes.c_int, VP, ctypes.c_size_t, VP]
    L.mlp_linear_bwd.restype = ctypes.c_int


def linear(M, N, K, act="none", resid_scale=1.0) -> Linear:
    """The problem: x [M, K], W [N, K], out [M, N].  (The row pitches come from the
    tensors of each call.)"""
    if act not in LINEAR_ACTS:
        raise ValueError(f"unknown activation {act!r}; one of {list(LINEAR_ACTS)}")
    return Linear(int(M), int(N), int(K), LINEAR_ACTS[act], float(resid_scale), 0, 0, 0)


def _dense(t, shape, name, dtype=torch.bfloat16):
    """The tensor's address (None stays None) once its type, device and shape are right."""
    if t is None:
        return None
    if (t.__class__ is torch.Tensor and t.dtype is dtype and t.is_cuda and t.shape == shape
            and t.is_contiguous()):
        return t.data_ptr()
    p = _ptr(t, dtype, name)  # says what is wrong (or passes a subclass)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    return p


def _pitched(t, shape, name):
    """(address, row pitch or 0 when dense) of a bf16 matrix with unit column stride."""
    if t is None:
        return None, 0
    if (t.__class__ is torch.Tensor and t.dtype is torch.bfloat16 and t.is_cuda
            and t.shape == shape and t.is_contiguous()):
        return t.data_ptr(), 0
    if not isinstance(t, torch.Tensor) or t.is_contiguous():
        return _dense(t, shape, name), 0
    if not t.is_cuda or t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be a CUDA bfloat16 tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.stride(1) != 1 or t.stride(0) < shape[1]:
        raise ValueError(f"{name} must have unit stride along its last dimension and rows "
                         "that do not overlap")
    if t.stride(0) > 0x7fffffff:  # the C ABI's int; ctypes would wrap it
        raise ValueError(f"{name}'s row stride of {t.stride(0)} passes 32 bits")
    return t.data_ptr(), t.stride(0)


def _problem(p, x, r, o):
    """`p` with the call's row pitches."""
    if not (x or r or o or p.ldx or p.ldr or p.ldo):
        return p
    return Linear(p.M, p.N, p.K, p.act, p.resid_scale, x, r, o)


def mlp_linear_workspace_size(p: Linear, backward=False) -> int:
    return int(lib().mlp_linear_workspace_size(ctypes.byref(p), int(bool(backward))))


@functools.lru_cache(maxsize=1024)
def _ws_size(M, N, K, act, backward):
    """The workspace size: a function of the sizes alone."""
    return mlp_linear_workspace_size(Linear(M, N, K, act), backward)


def alloc_linear_workspace(p: Linear, backward=False, device=None) -> torch.Tensor:
    n = mlp_linear_workspace_size(p, backward)
    if n == 0:
        raise MlpError(-1, "mlp_linear_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _ws(ws, p, backward, device, stream):
    if ws is None:  # (of a problem that the call refuses: any)
        return _call_workspace(_ws_size(p.M, p.N, p.K, p.act, backward) or 256, device, stream)
    if not (ws.is_cuda and ws.dtype == torch.uint8 and ws.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA uint8 tensor")
    return ws


def mlp_linear_fwd(p: Linear, x, W, bias, residual, out, pre_save=None, ws=None, stream=None):
    """out = act(x W^T + bias) + resid_scale * residual; bias and residual may be None.
    pre_save (bf16 [M, N]) receives x W^T + bias for the backward of an activation.
    Returns the workspace used (given none, a small one that later calls of this thread on
    this stream use too, and then hold their status)."""
    M, N, K = p.M, p.N, p.K
    xp, ldx = _pitched(x, (M, K), "x")
    rp, ldr = _pitched(residual, (M, N), "residual")
    op, ldo = _pitched(out, (M, N), "out")
    q = _problem(p, ldx, ldr, ldo)
    ws = _ws(ws, q, False, out.device, stream)
    rc = lib().mlp_linear_fwd(ctypes.byref(q), xp, _dense(W, (N, K), "W"),
                              _dense(bias, (N,), "bias"), rp, op,
                              _dense(pre_save, (M, N), "pre_save"), ws.data_ptr(), ws.numel(),
                              _stream(stream))
    _check(rc, "mlp_linear_fwd")
    return ws


def mlp_linear_bwd(p: Linear, dout, x, W, pre=None, dx=None, dW=None, db=None,
                   fuse_grad_accum=False, ws=None, stream=None):
    """dz = dout * act'(pre), dx = dz W, dW = dz^T x, db = sum of dz over the rows; outputs
    that are None are skipped.  dW and db are bf16 (overwritten) or fp32 (+= in place) when
    fuse_grad_accum.  (The residual's gradient is resid_scale * dout.)"""
    dp, ldd = _pitched(dout, (p.M, p.N), "dout")
    xp, ldx = _pitched(x, (p.M, p.K), "x")
    wd = torch.float32 if fuse_grad_accum else torch.bfloat16
    q = _problem(p, ldx, 0, ldd)
    ws = _ws(ws, q, True, dout.device, stream)
    rc = lib().mlp_linear_bwd(ctypes.byref(q), dp, xp, _dense(W, (p.N, p.K), "W"),
                              _dense(pre, (p.M, p.N), "pre"), _dense(dx, (p.M, p.K), "dx"),
                              _dense(dW, (p.N, p.K), "dW", wd), _dense(db, (p.N,), "db", wd),
                              int(bool(fuse_grad_accum)), ws.data_ptr(), ws.numel(),
                              _stream(stream))
    _check(rc, "mlp_linear_bwd")
    return ws
