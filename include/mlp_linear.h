/*
 * mlp_linear.h -- C ABI of the linear layer with its epilogue, of libmlp.so:
 *
 *   z   = x W^T + bias                       [M,N]
 *   out = act(z) + resid_scale * residual    [M,N]
 *
 * and its gradients.  x [M,K], W [N,K] (nn.Linear layout), bias [N],
 * residual [M,N]; bf16 storage, fp32 accumulation and epilogue, one rounding
 * to bf16.  An addition of this library; the conventions of mlp.h
 * (ownership, streams, alignment, return values, workspace, device-side
 * errors, determinism) hold here.
 */
#ifndef MLP_GB300_LINEAR_H
#define MLP_GB300_LINEAR_H

#include "mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The functions of mlp.h's activations: relu, relu^2, the tanh GELU, silu, sigmoid
 * (the last three with relative errors below 2e-5 before the rounding, down to
 * the smallest results). */
typedef enum {
  MLP_LINEAR_NONE = 0,
  MLP_LINEAR_RELU = 1,
  MLP_LINEAR_RELU_SQ = 2,
  MLP_LINEAR_GELU_TANH = 3,
  MLP_LINEAR_SILU = 4,
  MLP_LINEAR_SIGMOID = 5
} mlp_linear_act_t;

/* M, N, K > 0; N and K multiples of 8.  ldx, ldr, ldo: row pitch in elements
 * of x, of residual and of out (and of dout), 0 for dense; at least the row's
 * length, multiples of 8. */
typedef struct {
  int M, N, K;
  int act;            /* mlp_linear_act_t */
  float resid_scale;
  int ldx, ldr, ldo;
} mlp_linear_t;

/* Bytes of workspace of the forward (backward = 0) or the backward (1); 0 on
 * invalid arguments.  The backward's does not depend on which gradients are
 * asked for. */
size_t mlp_linear_workspace_size(const mlp_linear_t* p, int backward);

/* Forward.
 *   bias      bf16 [N] or NULL
 *   residual  bf16 [M,N] or NULL (pitch ldr); may be out itself
 *   out       bf16 [M,N] (pitch ldo); must not overlap x
 *   pre_save  bf16 [M,N] dense or NULL: z, which the backward of an
 *             activation needs (with MLP_LINEAR_NONE it is not)
 * With one to eight rows the weights are streamed on the warp-level MMA; up to
 * a few hundred run on the tensor cores with the weight rows as the MMA's M
 * (K shared by a cluster of CTAs where the blocks alone are too few); more rows
 * run as 128 x 256 or 256 x 256 output tiles.  A tile policy
 * (mlp_set_tile_policy) of 1 or 2 keeps every size above eight rows on those
 * tiles.  Two calls with the same operands and policy give the same bits. */
int mlp_linear_fwd(const mlp_linear_t* p, const void* x, const void* W, const void* bias,
                   const void* residual, void* out, void* pre_save, void* ws, size_t ws_bytes,
                   void* stream);

/* Backward:  dz = dout * act'(z),  dx = dz W,  dW = dz^T x,  db = sum_m dz.
 * (The residual's gradient is resid_scale * dout.)
 *   dout  bf16 [M,N] (pitch ldo)     pre  the forward's pre_save (NULL with MLP_LINEAR_NONE)
 *   dx    bf16 [M,K] dense, neither dout nor x;  dW [N,K], db [N]: bf16, or with fuse_grad_accum = 1
 *                                    fp32 that the gradient is added to
 * Each of dx, dW, db is NULL to skip; x and W may be NULL when what reads them
 * (dW, dx) is skipped.  dW may run on the library's second stream, as in
 * mlp_bwd. */
int mlp_linear_bwd(const mlp_linear_t* p, const void* dout, const void* x, const void* W,
                   const void* pre, void* dx, void* dW, void* db, int fuse_grad_accum, void* ws,
                   size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MLP_GB300_LINEAR_H */
