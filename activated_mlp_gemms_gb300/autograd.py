"""mlp_func / mlp_block_func: the fused MLP (and the MLP block with its RMS
norm and scaled residual) as differentiable PyTorch functions, on the
library's entry points (quack mlp.py's mlp_func and MLPRecomputeFunc: the
forward saves the preacts, or only x with recompute=True; the backward skips
the gradients autograd does not ask for; fuse_grad_accum adds the weight
gradients in place into fp32 buffers instead of returning them).

Argument marshalling only: the forward is one mlp_fwd call and the backward
one mlp_bwd or mlp_bwd_recompute call; nothing runs outside the library's
kernels.  Tensors are CUDA and bf16: x [..., H], Wg and Wu [I, H] (Wu None
for the non-gated activations), Wd [H, I].

With fuse_grad_accum=True every weight that needs a gradient carries an
fp32 tensor of its own shape as `main_grad`; the backward adds its gradient
there (dW += grad, as quack's _compute_weight_grad adds into the existing
gradient) and returns no gradient for it.

The saved-preact backward writes dG, dU over the saved G, U (the library's
in-place stage), so a graph built with recompute=False can be
differentiated once; recompute=True keeps only x and may be run again.

mlp_block_func is modded-nanogpt gpt.py's "process mlp" step, y =
resid_lambda x + post_lambda MLP(norm(x)), as one mlp_block_fwd and one
mlp_block_bwd call (saved preacts and the per-token 1/rms).

None of them can be differentiated twice: a second derivative raises.

linear_func is the linear layer with bias, activation and residual, and
moe_func the mixture-of-experts MLP (at the end of this file).
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import (GATED_ACTS, block, mlp_block_bwd, mlp_block_fwd, mlp_bwd, mlp_bwd_recompute,
               mlp_fwd, problem)
from .experts import (alloc_moe_plan, mlp_moe_combine, mlp_moe_combine_bwd, mlp_moe_dispatch,
                      mlp_moe_dispatch_bwd, mlp_moe_experts_bwd, mlp_moe_experts_fwd,
                      mlp_moe_fwd_infer, mlp_moe_rows, mlp_moe_sort, moe)
from .linear_op import linear, mlp_linear_bwd, mlp_linear_fwd


def _check_operand(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")


def _grad_buffers(ctx, x2, weights):
    """dx and the three weight-gradient buffers autograd asks for (None where
    it does not): fresh bf16 tensors, or each weight's fp32 main_grad when
    fusing the accumulation."""
    need = ctx.needs_input_grad
    dx = torch.empty_like(x2) if need[0] else None
    bufs = [None, None, None]
    for i, w in enumerate(weights):
        if w is None or not need[i + 1]:
            continue
        if ctx.fuse:
            g = getattr(w, "main_grad", None)
            if (g is None or g.dtype != torch.float32 or g.shape != w.shape
                    or not g.is_contiguous() or g.device != w.device):
                raise ValueError("fuse_grad_accum: each weight needs a contiguous fp32 "
                                 "`main_grad` of its own shape")
            bufs[i] = g
        else:
            bufs[i] = torch.empty_like(w)
    return dx, bufs


def _check_weights(act, Wg, Wu, Wd):
    gated = act in GATED_ACTS
    for t, name in ((Wg, "Wg"), (Wd, "Wd")):
        _check_operand(t, name)
    if gated:
        _check_operand(Wu, "Wu")
    elif Wu is not None:
        raise ValueError(f"{act} is not gated: Wu must be None")
    return gated


class _MlpFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, Wg, Wu, Wd, act, gate_mult, down_mult, recompute, fuse_grad_accum):
        _check_operand(x, "x")
        gated = _check_weights(act, Wg, Wu, Wd)
        shape = x.shape
        H = shape[-1]
        I = Wd.shape[1]
        x2 = x.reshape(-1, H).contiguous()
        M = x2.shape[0]
        ctx.shape, ctx.recompute, ctx.fuse, ctx.gated = shape, recompute, fuse_grad_accum, gated
        ctx.spent = False
        out = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
        if M == 0:
            ctx.prob = None
            ctx.save_for_backward(x2, Wg, Wu, Wd, None, None)
            return out.view(shape)
        prob = problem(M, H, I, act, gate_mult, down_mult)
        ctx.prob = prob
        if recompute:
            G = U = None
            mlp_fwd(prob, x2, Wg, Wu, Wd, out)
        else:
            G = torch.empty((M, I), dtype=torch.bfloat16, device=x.device)
            U = torch.empty_like(G) if gated else None
            mlp_fwd(prob, x2, Wg, Wu, Wd, out, G, U)
        ctx.save_for_backward(x2, Wg, Wu, Wd, G, U)
        return out.view(shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        x2, Wg, Wu, Wd, G, U = ctx.saved_tensors
        if ctx.spent and not ctx.recompute:
            raise RuntimeError("mlp_func: the saved preacts were overwritten by the first "
                               "backward; use recompute=True to differentiate twice")
        ctx.spent = True
        M, H = x2.shape
        dx, bufs = _grad_buffers(ctx, x2, (Wg, Wu, Wd))
        if M == 0:
            if dx is not None:
                dx = dx.view(ctx.shape)
            grads = [None if ctx.fuse or b is None else b.zero_() for b in bufs]
            return (dx, *grads, None, None, None, None, None)
        dout2 = dout.reshape(-1, H)
        if dout2.dtype != torch.bfloat16:
            dout2 = dout2.to(torch.bfloat16)
        dout2 = dout2.contiguous()
        if any(b is not None for b in bufs) or dx is not None:
            if ctx.recompute:
                mlp_bwd_recompute(ctx.prob, dout2, x2, Wg, Wu, Wd, dx, *bufs,
                                  fuse_grad_accum=ctx.fuse)
            else:
                mlp_bwd(ctx.prob, dout2, x2, Wg, Wu, Wd, G, U, dx, *bufs,
                        fuse_grad_accum=ctx.fuse)
        grads = [None if ctx.fuse else b for b in bufs]
        return (dx.view(ctx.shape) if dx is not None else None, *grads,
                None, None, None, None, None)


def mlp_func(x, Wg, Wu, Wd, activation="swiglu", gate_mult=1.0, down_mult=1.0,
             recompute=False, fuse_grad_accum=False):
    """out = down_mult * Wd (gate_mult * act(x Wg^T) * (x Wu^T)) over the last
    dimension of x, differentiable with respect to x and the weights."""
    return _MlpFunction.apply(x, Wg, Wu, Wd, activation, gate_mult, down_mult, bool(recompute),
                              bool(fuse_grad_accum))


class _MlpBlockFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, Wg, Wu, Wd, act, gate_mult, down_mult, resid_lambda, post_lambda, eps,
                fuse_grad_accum):
        _check_operand(x, "x")
        gated = _check_weights(act, Wg, Wu, Wd)
        shape = x.shape
        H = shape[-1]
        I = Wd.shape[1]
        x2 = x.reshape(-1, H).contiguous()
        M = x2.shape[0]
        ctx.shape, ctx.fuse = shape, fuse_grad_accum
        ctx.spent = False
        y = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
        if M == 0:
            ctx.prob = None
            ctx.save_for_backward(x2, Wg, Wu, Wd, None, None, None)
            return y.view(shape)
        prob = problem(M, H, I, act, gate_mult, down_mult)
        blk = block(resid_lambda, post_lambda, eps)
        ctx.prob, ctx.blk = prob, blk
        G = torch.empty((M, I), dtype=torch.bfloat16, device=x.device)
        U = torch.empty_like(G) if gated else None
        rstd, _ = mlp_block_fwd(prob, blk, x2, Wg, Wu, Wd, y, G, U)
        ctx.save_for_backward(x2, Wg, Wu, Wd, G, U, rstd)
        return y.view(shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x2, Wg, Wu, Wd, G, U, rstd = ctx.saved_tensors
        if ctx.spent:
            raise RuntimeError("mlp_block_func: the saved preacts were overwritten by the "
                               "first backward")
        ctx.spent = True
        M, H = x2.shape
        dx, bufs = _grad_buffers(ctx, x2, (Wg, Wu, Wd))
        rest = (None,) * 7
        if M == 0:
            grads = [None if ctx.fuse or b is None else b.zero_() for b in bufs]
            return (dx.view(ctx.shape) if dx is not None else None, *grads, *rest)
        dy2 = dy.reshape(-1, H)
        if dy2.dtype != torch.bfloat16:
            dy2 = dy2.to(torch.bfloat16)
        dy2 = dy2.contiguous()
        if any(b is not None for b in bufs) or dx is not None:
            mlp_block_bwd(ctx.prob, ctx.blk, dy2, x2, Wg, Wu, Wd, G, U, rstd, dx, *bufs,
                          fuse_grad_accum=ctx.fuse)
        grads = [None if ctx.fuse else b for b in bufs]
        return (dx.view(ctx.shape) if dx is not None else None, *grads, *rest)


def mlp_block_func(x, Wg, Wu, Wd, activation="swiglu", gate_mult=1.0, down_mult=1.0,
                   resid_lambda=1.0, post_lambda=1.0, eps=2.0 ** -7, fuse_grad_accum=False):
    """y = resid_lambda x + post_lambda MLP(x / rms(x)) over the last
    dimension of x (rms with eps inside the root), differentiable with
    respect to x and the weights."""
    return _MlpBlockFunction.apply(x, Wg, Wu, Wd, activation, gate_mult, down_mult,
                                   float(resid_lambda), float(post_lambda), float(eps),
                                   bool(fuse_grad_accum))


def _grad_like(t, fuse, name):
    """Where a weight's gradient goes: a fresh bf16 tensor, or its fp32 main_grad."""
    if not fuse:
        return torch.empty_like(t)
    g = getattr(t, "main_grad", None)
    if (g is None or g.dtype != torch.float32 or g.shape != t.shape or not g.is_contiguous()
            or g.device != t.device):
        raise ValueError(f"fuse_grad_accum: {name} needs a contiguous fp32 `main_grad` of its "
                         "own shape")
    return g


def _check_shape(t, shape, name):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _check_rows(t, lead, last, name):
    """A row of `last` values for each of x's rows: x's own leading dimensions, or flat."""
    if t.dim() != 2 or t.shape != (math.prod(lead), last):
        _check_shape(t, (*lead, last), name)


class _LinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, bias, residual, act, resid_scale, fuse_grad_accum, keep_pre):
        for t, name in ((x, "x"), (W, "W")) + (((bias, "bias"),) if bias is not None else ()) + (
                ((residual, "residual"),) if residual is not None else ()):
            _check_operand(t, name)
        if W.dim() != 2:
            raise ValueError(f"W must be [N, K], got {tuple(W.shape)}")
        N, K = W.shape
        shape = x.shape
        if x.dim() == 0 or shape[-1] != K:
            raise ValueError(f"x must have {K} values in its last dimension, got {tuple(shape)}")
        if bias is not None:
            _check_shape(bias, (N,), "bias")
        if residual is not None:
            _check_rows(residual, shape[:-1], N, "residual")
        x2 = x.reshape(-1, K).contiguous()
        M = x2.shape[0]
        ctx.x_shape, ctx.fuse, ctx.scale = shape, fuse_grad_accum, resid_scale
        ctx.r_shape = residual.shape if residual is not None else None
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
        ctx.prob = linear(M, N, K, act, resid_scale)
        pre = None
        if M:
            r2 = residual.reshape(M, N).contiguous() if residual is not None else None
            if act != "none" and keep_pre:
                pre = torch.empty_like(out)
            mlp_linear_fwd(ctx.prob, x2, W, bias, r2, out, pre)
        ctx.save_for_backward(x2, W, bias, pre)
        return out.view(*shape[:-1], N)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        x2, W, bias, pre = ctx.saved_tensors
        need = ctx.needs_input_grad
        M, N = x2.shape[0], W.shape[0]
        d2 = dout.reshape(M, N)
        if d2.dtype != torch.bfloat16:
            d2 = d2.to(torch.bfloat16)
        d2 = d2.contiguous()
        dx = torch.empty_like(x2) if need[0] else None
        dW = _grad_like(W, ctx.fuse, "W") if need[1] else None
        db = _grad_like(bias, ctx.fuse, "bias") if bias is not None and need[2] else None
        if M == 0:
            if not ctx.fuse:
                for g in (dW, db):
                    if g is not None:
                        g.zero_()
        elif dx is not None or dW is not None or db is not None:
            mlp_linear_bwd(ctx.prob, d2, x2, W, pre, dx, dW, db, fuse_grad_accum=ctx.fuse)
        dr = None
        if ctx.r_shape is not None and need[3]:
            dr = (dout if ctx.scale == 1.0 else dout * ctx.scale).reshape(ctx.r_shape)
        return (dx.view(ctx.x_shape) if dx is not None else None, None if ctx.fuse else dW,
                None if ctx.fuse else db, dr, None, None, None, None)


def linear_func(x, W, bias=None, residual=None, activation="none", resid_scale=1.0,
                fuse_grad_accum=False):
    """out = act(x W^T + bias) + resid_scale * residual over the last dimension of x,
    differentiable with respect to x, W, bias and residual (one mlp_linear_fwd and one
    mlp_linear_bwd call)."""
    # (ctx.needs_input_grad stays true for parameters where gradients are off)
    keep_pre = torch.is_grad_enabled() and any(
        isinstance(t, torch.Tensor) and t.requires_grad for t in (x, W, bias))
    return _LinearFunction.apply(x, W, bias, residual, activation, float(resid_scale),
                                 bool(fuse_grad_accum), keep_pre)


class _MoeFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weights, Wg, Wu, Wd, residual, ids, prob, fuse_grad_accum):
        T, H = x.shape
        new = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=x.device)  # noqa: E731
        ctx.prob, ctx.fuse, ctx.spent = prob, fuse_grad_accum, False
        if prob is None:  # no tokens
            ctx.save_for_backward(x, weights, Wg, Wu, Wd)
            return new(0, H)
        rows = mlp_moe_rows(prob)
        plan = alloc_moe_plan(prob, x.device)
        xs, y, G = new(rows, H), new(rows, H), new(rows, prob.I)
        U = new(rows, prob.I) if Wu is not None else None
        out = new(T, H)
        mlp_moe_sort(prob, ids, plan)
        mlp_moe_dispatch(prob, plan, x, xs)
        mlp_moe_experts_fwd(prob, plan, xs, Wg, Wu, Wd, y, G, U)
        mlp_moe_combine(prob, plan, y, weights, residual, out)
        keep_y = y if ctx.needs_input_grad[1] else None  # only the weights' gradient reads it
        ctx.save_for_backward(plan, xs, weights, Wg, Wu, Wd, G, U, keep_y)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        need = ctx.needs_input_grad
        if ctx.prob is None:
            grads = [torch.zeros_like(t) if t is not None and n and not (ctx.fuse and i >= 2) else None
                     for i, (t, n) in enumerate(zip(ctx.saved_tensors, need))]
            return (*grads, dout if need[5] else None, None, None, None)
        plan, xs, weights, Wg, Wu, Wd, G, U, y = ctx.saved_tensors
        p = ctx.prob
        experts = need[0] or any(need[2:5])
        if ctx.spent and experts:
            raise RuntimeError("moe_func: the saved preacts were overwritten by the first backward")
        d = dout if dout.dtype == torch.bfloat16 else dout.to(torch.bfloat16)
        d = d.contiguous()
        dy = torch.empty_like(xs) if experts else None
        dw = torch.empty_like(weights) if need[1] else None
        mlp_moe_combine_bwd(p, plan, d, y, weights, dy, dw)
        dx = dxs = None
        dW = [None, None, None]
        if experts:
            ctx.spent = True
            for i, (w, name) in enumerate(((Wg, "Wg"), (Wu, "Wu"), (Wd, "Wd"))):
                if w is not None and need[2 + i]:
                    dW[i] = _grad_like(w, ctx.fuse, name)
            if need[0]:
                dxs = torch.empty_like(xs)
            mlp_moe_experts_bwd(p, plan, dy, xs, Wg, Wu, Wd, G, U, dxs, *dW,
                                fuse_grad_accum=ctx.fuse)
            if need[0]:
                dx = torch.empty((p.T, p.H), dtype=torch.bfloat16, device=xs.device)
                mlp_moe_dispatch_bwd(p, plan, dxs, dx)
        dW = [None if ctx.fuse else g for g in dW]
        return (dx, dw, *dW, dout if need[5] else None, None, None, None)


def moe_func(x, ids, weights, Wg, Wu, Wd, activation="swiglu", residual=None, gate_mult=1.0,
             down_mult=1.0, fuse_grad_accum=False):
    """The mixture-of-experts MLP, out[t] = residual[t] + sum_j weights[t, j]
    MLP_{ids[t, j]}(x[t]), over the last dimension of x: ids int32 and weights (fp32 or
    bf16) [..., top_k], Wg and Wu [E, I, H] (Wu None when non-gated), Wd [E, H, I].  A slot
    whose id is outside [0, E) is dropped.  Differentiable with respect to x, weights, the
    experts' weights and residual; without gradients to take it is one mlp_moe_fwd_infer
    call.  The graph can be differentiated once (the saved preacts become their
    gradients)."""
    gated = _check_weights(activation, Wg, Wu, Wd)
    _check_operand(x, "x")
    if Wg.dim() != 3:
        raise ValueError(f"Wg must be [E, I, H], got {tuple(Wg.shape)}")
    E, inner, H = Wg.shape
    if x.dim() == 0 or x.shape[-1] != H:
        raise ValueError(f"x must have {H} values in its last dimension, got {tuple(x.shape)}")
    if ids.dim() == 0:
        raise ValueError("ids must be [..., top_k]")
    shape, k = x.shape, ids.shape[-1]
    _check_rows(ids, shape[:-1], k, "ids")
    _check_rows(weights, shape[:-1], k, "weights")
    if gated:
        _check_shape(Wu, (E, inner, H), "Wu")
    _check_shape(Wd, (E, H, inner), "Wd")
    x2 = x.reshape(-1, H).contiguous()
    T = x2.shape[0]
    r2 = None
    if residual is not None:
        _check_operand(residual, "residual")
        _check_rows(residual, shape[:-1], H, "residual")
        r2 = residual.reshape(T, H).contiguous()
    i2, w2 = ids.reshape(T, k).contiguous(), weights.reshape(T, k).contiguous()
    prob = moe(T, E, k, H, inner, activation, gate_mult, down_mult,
               weights_dtype=w2.dtype) if T else None
    args = [t for t in (x2, w2, Wg, Wu, Wd, r2) if t is not None]
    if torch.is_grad_enabled() and any(t.requires_grad for t in args):
        out = _MoeFunction.apply(x2, w2, Wg, Wu, Wd, r2, i2, prob, bool(fuse_grad_accum))
    else:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
        if T:
            mlp_moe_fwd_infer(prob, x2, i2, w2, Wg, Wu, Wd, r2, out)
    return out.view(shape)
