/*
 * mlp_norm.h -- C ABI of the layer norm with the residual sum in front of it, of
 * libmlp.so:
 *
 *   h = x + residual                               [M,H] (rounded to its type)
 *   y = (h - mean) * rstd * weight + bias          [M,H]
 *   mean = sum_i h[m,i] / H,  rstd = 1 / sqrt(sum_i (h[m,i] - mean)^2 / H + eps)
 *
 * and its gradients.  Sums and statistics in fp32, one rounding of each output.
 * An addition of this library; the conventions of mlp.h (ownership, streams,
 * alignment, return values, workspace, determinism) hold here.  (The RMS norm of
 * mlp_block_fwd is part of that call.)
 */
#ifndef MLP_GB300_NORM_H
#define MLP_GB300_NORM_H

#include "mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLP_NORM_MAX_H 16384

typedef enum { MLP_NORM_F32 = 0, MLP_NORM_BF16 = 1 } mlp_norm_type_t;

/* M rows of H values, H a multiple of 8 and at most MLP_NORM_MAX_H; eps >= 0. */
typedef struct {
  int M, H;
  float eps;
  int type;         /* mlp_norm_type_t: of x, residual, h, y and their gradients */
  int weight_type;  /* mlp_norm_type_t: of weight and bias */
  int ldx, ldr;     /* row pitch in values of x and of residual (the forward's inputs), 0 for
                     * dense; at least H, multiples of 8 */
} mlp_layernorm_t;

/* Bytes of workspace of mlp_layernorm_bwd with dweight or dbias; 0 on invalid
 * arguments. */
size_t mlp_layernorm_workspace_size(const mlp_layernorm_t* p);

/* Forward.
 *   x, residual  [M,H] (pitches ldx, ldr); residual NULL: h is x
 *   weight, bias [H] (weight_type); NULL: ones, zeros
 *   y            [M,H] out, dense; may be x or residual itself (dense)
 *   h            [M,H] out, dense, or NULL; with a residual, what the backward takes (it may
 *                be x or residual itself (dense), not y)
 *   mean, rstd   fp32 [M] out or NULL: for the backward
 * (No other output overlaps an operand or another output.) */
int mlp_layernorm_fwd(const mlp_layernorm_t* p, const void* x, const void* residual,
                      const void* weight, const void* bias, void* y, void* h, float* mean,
                      float* rstd, void* stream);

/* Backward (ldx, ldr are not read: every operand is dense).
 *   dy       [M,H];  h  [M,H] the forward's h (its x without a residual)
 *   mean, rstd  the forward's;  weight as in the forward
 *   dh       [M,H] or NULL: a gradient that reaches h from elsewhere, added to dx
 *   dx       [M,H] out or NULL: the gradient of h, so of x and of residual alike; may be
 *            dy or dh itself, not h
 *   dweight, dbias  [H] out or NULL: in weight_type, or with fuse_grad_accum = 1 fp32 that
 *            the gradient is added to
 *   ws       NULL where dweight and dbias both are
 * (No other output overlaps an operand or another output.) */
int mlp_layernorm_bwd(const mlp_layernorm_t* p, const void* dy, const void* h, const void* weight,
                      const float* mean, const float* rstd, const void* dh, void* dx,
                      void* dweight, void* dbias, int fuse_grad_accum, void* ws, size_t ws_bytes,
                      void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MLP_GB300_NORM_H */
