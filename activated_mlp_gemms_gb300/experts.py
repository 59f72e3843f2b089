"""The mixture-of-experts MLP (include/mlp_moe.h): tokens sorted by expert and
back with their routing weights, and the gradients.

Calls return the workspace that they used: given none, a small one that later calls
of the same thread on the same stream use too, and then hold their status.

Argument marshalling only, as in the package's other calls: outputs are
tensors that the caller passes.  Every shape is checked, because the kernels
take their row numbers from the plan.
"""
from __future__ import annotations

import ctypes
import functools
from collections.abc import Mapping

import torch

from . import (ACTS, MODE_BWD, MODE_FWD, MODE_INFER, MlpError, _call_workspace, _check, _ptr,
               _stream, _wdt, lib)

ROW_ALIGN = 16  # MLP_MOE_ROW_ALIGN
MAX_EXPERTS = 1024  # MLP_MOE_MAX_EXPERTS
MAX_TOP_K = 64  # MLP_MOE_MAX_TOP_K
_W_DTYPES = (torch.float32, torch.bfloat16)
_W_TYPES = {t: i for i, t in enumerate(_W_DTYPES)}


class Moe(ctypes.Structure):
    """mlp_moe_t"""
    _fields_ = [("T", ctypes.c_int), ("E", ctypes.c_int), ("top_k", ctypes.c_int),
                ("H", ctypes.c_int), ("I", ctypes.c_int), ("act", ctypes.c_int),
                ("gate_mult", ctypes.c_float), ("down_mult", ctypes.c_float),
                ("weights_type", ctypes.c_int)]


class _Layout(ctypes.Structure):
    """mlp_moe_plan_t"""
    _fields_ = [(n, ctypes.c_longlong) for n in ("ints", "offsets", "counts", "pos", "src")]


def declare(L):
    """Argument types of mlp_moe.h's functions (called when the library is loaded)."""
    P, VP = ctypes.POINTER(Moe), ctypes.c_void_p
    L.mlp_moe_rows.argtypes = [P]
    L.mlp_moe_rows.restype = ctypes.c_longlong
    L.mlp_moe_plan_layout.argtypes = [P, ctypes.POINTER(_Layout)]
    L.mlp_moe_sort.argtypes = [P] + [VP] * 3
    L.mlp_moe_dispatch.argtypes = [P] + [VP] * 4
    L.mlp_moe_dispatch_bwd.argtypes = [P] + [VP] * 4
    L.mlp_moe_combine.argtypes = [P] + [VP] * 6
    L.mlp_moe_combine_bwd.argtypes = [P] + [VP] * 7
    L.mlp_moe_workspace_size.argtypes = [P, ctypes.c_int]
    L.mlp_moe_workspace_size.restype = ctypes.c_size_t
    L.mlp_moe_experts_fwd.argtypes = [P] + [VP] * 9 + [ctypes.c_size_t, VP]
    L.mlp_moe_experts_bwd.argtypes = [P] + [VP] * 12 + [ctypes.c_int, VP, ctypes.c_size_t, VP]
    L.mlp_moe_fwd_infer.argtypes = [P] + [VP] * 9 + [ctypes.c_size_t, VP]
    for n in ("experts_fwd", "experts_bwd", "fwd_infer"):
        getattr(L, "mlp_moe_" + n).restype = ctypes.c_int
    for n in ("plan_layout", "sort", "dispatch", "dispatch_bwd", "combine", "combine_bwd"):
        getattr(L, "mlp_moe_" + n).restype = ctypes.c_int


def moe(T, E, top_k, H, I=0, act="swiglu", gate_mult=1.0, down_mult=1.0,
        weights_dtype=torch.float32) -> Moe:
    """The problem: T tokens of H values, E experts, top_k slots a token; the experts'
    intermediate size I, activation and multipliers; the routing weights' type."""
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r}; one of {list(ACTS)}")
    if weights_dtype not in _W_TYPES:
        raise ValueError("weights_dtype must be torch.float32 or torch.bfloat16")
    return Moe(int(T), int(E), int(top_k), int(H), int(I), ACTS[act], float(gate_mult),
               float(down_mult), _W_TYPES[weights_dtype])


def _shaped(t, shape, name, dtype=torch.bfloat16):
    """The tensor's address (None stays None) once its type, device and shape are right."""
    if t is None:
        return None
    if (t.__class__ is torch.Tensor and t.dtype is dtype and t.is_cuda and t.shape == shape
            and t.is_contiguous()):
        return t.data_ptr()
    p = _ptr(t, dtype, name)  # says what is wrong (or passes a subclass)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return p


class _Sizes:
    """What the calls need to know of a problem's sizes: the shapes of the tensors, and the
    plan's public parts as (shape, strides, first value)."""

    def __init__(self, T, E, top_k, H, weights_type):
        p, out = Moe(T, E, top_k, H, weights_type=weights_type), _Layout()
        _check(lib().mlp_moe_plan_layout(ctypes.byref(p), ctypes.byref(out)),
               "mlp_moe_plan_layout")
        rows = int(lib().mlp_moe_rows(ctypes.byref(p)))
        self.tokens, self.slots, self.rows = (T, H), (T, top_k), (rows, H)
        self.layout, self.plan = out, (int(out.ints),)
        self.views = {"offsets": ((E + 1,), (1,), out.offsets), "counts": ((E,), (1,), out.counts),
                      "pos": ((T, top_k), (top_k, 1), out.pos), "src": ((rows,), (1,), out.src)}
        self.w_dtype = _W_DTYPES[weights_type]


_sizes_of = functools.lru_cache(maxsize=1024)(_Sizes)


def _sizes(p: Moe) -> _Sizes:
    return _sizes_of(p.T, p.E, p.top_k, p.H, p.weights_type)


def _layout(p: Moe) -> _Layout:
    return _sizes(p).layout


def mlp_moe_rows(p: Moe) -> int:
    """Rows of the sorted layout's buffers (xs, y, dxs, dy, G, U)."""
    return _sizes(p).rows[0]


def alloc_moe_plan(p: Moe, device=None) -> torch.Tensor:
    return torch.empty(_sizes(p).plan, dtype=torch.int32, device=device or "cuda")


def _plan(s: _Sizes, plan):
    return _shaped(plan, s.plan, "plan", torch.int32)


class _PlanViews(Mapping):
    """The plan's public parts, each made a view when it is asked for."""

    def __init__(self, views, plan):
        self._views, self._plan = views, plan

    def __getitem__(self, name):
        size, stride, first = self._views[name]
        return self._plan.as_strided(size, stride, self._plan.storage_offset() + first)

    def __iter__(self):
        return iter(self._views)

    def __len__(self):
        return len(self._views)


def moe_plan_views(p: Moe, plan) -> Mapping:
    """The plan's public parts as views: offsets [E + 1] (first row of each expert),
    counts [E], pos [T, top_k] (row of each slot, -1 when dropped), src [rows] (slot of
    each row, -1 for padding)."""
    s = _sizes(p)
    _plan(s, plan)
    return _PlanViews(s.views, plan)


def mlp_moe_sort(p: Moe, ids, plan, stream=None) -> None:
    """Fills the plan from ids (int32 [T, top_k]; an id outside [0, E) drops the slot)."""
    s = _sizes(p)
    rc = lib().mlp_moe_sort(ctypes.byref(p), _shaped(ids, s.slots, "ids", torch.int32),
                            _plan(s, plan), _stream(stream))
    _check(rc, "mlp_moe_sort")


def mlp_moe_dispatch(p: Moe, plan, x, xs, stream=None) -> None:
    """xs[pos[t, j]] = x[t]; the other rows of xs become zero."""
    s = _sizes(p)
    rc = lib().mlp_moe_dispatch(ctypes.byref(p), _plan(s, plan), _shaped(x, s.tokens, "x"),
                                _shaped(xs, s.rows, "xs"), _stream(stream))
    _check(rc, "mlp_moe_dispatch")


def mlp_moe_dispatch_bwd(p: Moe, plan, dxs, dx, stream=None) -> None:
    """dx[t] = sum_j dxs[pos[t, j]]."""
    s = _sizes(p)
    rc = lib().mlp_moe_dispatch_bwd(ctypes.byref(p), _plan(s, plan), _shaped(dxs, s.rows, "dxs"),
                                    _shaped(dx, s.tokens, "dx"), _stream(stream))
    _check(rc, "mlp_moe_dispatch_bwd")


def mlp_moe_combine(p: Moe, plan, y, weights, residual, out, stream=None) -> None:
    """out[t] = residual[t] + sum_j weights[t, j] y[pos[t, j]] (residual may be None)."""
    s = _sizes(p)
    rc = lib().mlp_moe_combine(ctypes.byref(p), _plan(s, plan), _shaped(y, s.rows, "y"),
                               _shaped(weights, s.slots, "weights", s.w_dtype),
                               _shaped(residual, s.tokens, "residual"),
                               _shaped(out, s.tokens, "out"), _stream(stream))
    _check(rc, "mlp_moe_combine")


def mlp_moe_combine_bwd(p: Moe, plan, dout, y, weights, dy=None, dweights=None,
                        stream=None) -> None:
    """dy[pos[t, j]] = weights[t, j] dout[t] (the other rows zero) and
    dweights[t, j] = <dout[t], y[pos[t, j]]>; either may be None."""
    s = _sizes(p)
    rc = lib().mlp_moe_combine_bwd(ctypes.byref(p), _plan(s, plan),
                                   _shaped(dout, s.tokens, "dout"), _shaped(y, s.rows, "y"),
                                   _shaped(weights, s.slots, "weights", s.w_dtype),
                                   _shaped(dy, s.rows, "dy"),
                                   _shaped(dweights, s.slots, "dweights", s.w_dtype),
                                   _stream(stream))
    _check(rc, "mlp_moe_combine_bwd")


def mlp_moe_workspace_size(p: Moe, mode: int) -> int:
    return int(lib().mlp_moe_workspace_size(ctypes.byref(p), int(mode)))


@functools.lru_cache(maxsize=1024)
def _ws_size(T, E, top_k, H, I, act, mode):
    """The workspace size: a function of the sizes alone."""
    return mlp_moe_workspace_size(Moe(T, E, top_k, H, I, act, 1.0, 1.0, 0), mode)


def alloc_moe_workspace(p: Moe, mode: int, device=None) -> torch.Tensor:
    n = mlp_moe_workspace_size(p, mode)
    if n == 0:
        raise MlpError(-1, "mlp_moe_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _ws(ws, p, mode, device, stream):
    if ws is None:  # (of a problem that the call refuses: any)
        n = _ws_size(p.T, p.E, p.top_k, p.H, p.I, p.act, mode)
        return _call_workspace(n or 256, device, stream)
    if not (ws.is_cuda and ws.dtype == torch.uint8 and ws.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA uint8 tensor")
    return ws


def _weights(p: Moe, Wg, Wu, Wd, dtype=torch.bfloat16, names=("Wg", "Wu", "Wd")):
    up, down = (p.E, p.I, p.H), (p.E, p.H, p.I)
    return (_shaped(Wg, up, names[0], dtype), _shaped(Wu, up, names[1], dtype),
            _shaped(Wd, down, names[2], dtype))


def mlp_moe_experts_fwd(p: Moe, plan, xs, Wg, Wu, Wd, y, G_save=None, U_save=None, ws=None,
                        stream=None):
    """Each expert's MLP over its rows of xs: y[r] = MLP_e(xs[r]); optionally stores the
    preacts (bf16 [rows, I]) for the backward.  Wg, Wu [E, I, H] (Wu None when non-gated),
    Wd [E, H, I].  Rows of y past the plan's offsets[E] are not written.  Up to
    MLP_MOE_FINE_SLOTS slots the plan receives y in fp32 too, for dweights of
    mlp_moe_combine_bwd.  Returns the workspace used."""
    s = _sizes(p)
    inter = (s.rows[0], p.I)
    ws = _ws(ws, p, MODE_FWD, y.device, stream)
    rc = lib().mlp_moe_experts_fwd(ctypes.byref(p), _plan(s, plan), _shaped(xs, s.rows, "xs"),
                                   *_weights(p, Wg, Wu, Wd), _shaped(y, s.rows, "y"),
                                   _shaped(G_save, inter, "G_save"),
                                   _shaped(U_save, inter, "U_save"), ws.data_ptr(),
                                   ws.numel(), _stream(stream))
    _check(rc, "mlp_moe_experts_fwd")
    return ws


def mlp_moe_experts_bwd(p: Moe, plan, dy, xs, Wg, Wu, Wd, G, U, dxs=None, dWg=None, dWu=None,
                        dWd=None, fuse_grad_accum=False, ws=None, stream=None):
    """Gradients of mlp_moe_experts_fwd from its saved G, U (overwritten with dG, dU).
    Outputs that are None are skipped; weight gradients are bf16 (overwritten) or fp32
    (+= in place) when fuse_grad_accum.  The padding rows of dy and xs are zero."""
    s = _sizes(p)
    inter = (s.rows[0], p.I)
    ws = _ws(ws, p, MODE_BWD, dy.device, stream)
    rc = lib().mlp_moe_experts_bwd(ctypes.byref(p), _plan(s, plan), _shaped(dy, s.rows, "dy"),
                                   _shaped(xs, s.rows, "xs"), *_weights(p, Wg, Wu, Wd),
                                   _shaped(G, inter, "G"), _shaped(U, inter, "U"),
                                   _shaped(dxs, s.rows, "dxs"),
                                   *_weights(p, dWg, dWu, dWd, _wdt(fuse_grad_accum),
                                             ("dWg", "dWu", "dWd")),
                                   int(bool(fuse_grad_accum)), ws.data_ptr(), ws.numel(),
                                   _stream(stream))
    _check(rc, "mlp_moe_experts_bwd")
    return ws


def mlp_moe_fwd_infer(p: Moe, x, ids, weights, Wg, Wu, Wd, residual, out, ws=None, stream=None):
    """The whole layer without gradients: out[t] = residual[t] + sum_j weights[t, j]
    MLP_{ids[t, j]}(x[t]) (residual may be None).  Returns the workspace used."""
    ws = _ws(ws, p, MODE_INFER, out.device, stream)
    th, tk = (p.T, p.H), (p.T, p.top_k)
    rc = lib().mlp_moe_fwd_infer(ctypes.byref(p), _shaped(x, th, "x"),
                                 _shaped(ids, tk, "ids", torch.int32),
                                 _shaped(weights, tk, "weights", _W_DTYPES[bool(p.weights_type)]),
                                 *_weights(p, Wg, Wu, Wd), _shaped(residual, th, "residual"),
                                 _shaped(out, th, "out"), ws.data_ptr(), ws.numel(),
                                 _stream(stream))
    _check(rc, "mlp_moe_fwd_infer")
    return ws
