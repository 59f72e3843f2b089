/*
 * mlp_moe.h -- C ABI of the mixture-of-experts MLP of libmlp.so: tokens
 * sorted by expert and back with their routing weights, each expert's MLP
 * over its own rows, and the gradients.  An addition of this library; the
 * conventions of mlp.h (ownership, streams, alignment, return values,
 * workspace, device-side errors) hold for every call here.
 *
 * A token t has top_k slots; slot (t, j) names an expert ids[t, j] and
 * carries a weight w[t, j].  A slot whose id is not in [0, E) is dropped: it
 * takes no row, and contributes nothing.  With MLP_e the expert's MLP of
 * mlp.h (bias-free, gated or not):
 *
 *   out[t] = residual[t] + sum_j w[t, j] * MLP_{ids[t, j]}(x[t])
 *
 * The sorted layout.  Every expert owns a contiguous block of rows that
 * begins at a multiple of MLP_MOE_ROW_ALIGN (16, the K step of a bf16
 * tensor-core instruction: a weight gradient sums over an expert's rows, so
 * whole steps belong to one expert).  Inside the block the slots come in
 * the order of t, then j; the rows that fill up the block's last 16 are
 * padding.  mlp_moe_rows gives the most rows any assignment can need, and
 * the row buffers have that many.
 */
#ifndef MLP_GB300_MOE_H
#define MLP_GB300_MOE_H

#include "mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLP_MOE_ROW_ALIGN 16
#define MLP_MOE_MAX_EXPERTS 1024
#define MLP_MOE_MAX_TOP_K 64
#define MLP_MOE_FINE_SLOTS 64

typedef enum { MLP_MOE_W_F32 = 0, MLP_MOE_W_BF16 = 1 } mlp_moe_weight_t;

/* T tokens of H values, E experts, top_k slots a token; the experts' MLPs:
 * intermediate size I, activation and multipliers as mlp_problem_t's (I and
 * act are read by the calls that run the experts only).  weights_type: the
 * type of the routing weights and of their gradient. */
typedef struct {
  int T, E, top_k, H, I;
  int act;           /* mlp_act_t */
  float gate_mult, down_mult;
  int weights_type;  /* mlp_moe_weight_t */
} mlp_moe_t;

/* Rows of the sorted layout's buffers: n + 15 min(E, n), rounded down to a
 * multiple of 16, with n = T top_k.  0 on invalid arguments. */
long long mlp_moe_rows(const mlp_moe_t* p);

/* The plan: one caller-owned int32 device buffer (16-byte aligned) that
 * mlp_moe_sort fills and every other call reads.  Up to MLP_MOE_FINE_SLOTS slots
 * (T top_k) it also has room for the experts' results in fp32, rows x H values:
 * mlp_moe_experts_fwd writes them beside y, and dweights of mlp_moe_combine_bwd
 * reads them. */
typedef struct {
  long long ints;     /* size of the plan, in int32 values */
  long long offsets;  /* [E + 1]: first row of each expert; [E] = rows in use */
  long long counts;   /* [E]: slots of each expert */
  long long pos;      /* [T, top_k]: row of each slot, -1 when dropped */
  long long src;      /* [rows]: slot t * top_k + j of each row, -1 for padding and past the end */
} mlp_moe_plan_t;     /* the last four: where in the plan, in int32 values */
int mlp_moe_plan_layout(const mlp_moe_t* p, mlp_moe_plan_t* layout);

/* Fills the plan from ids (int32 [T, top_k], 4-byte aligned).  Stable and
 * deterministic. */
int mlp_moe_sort(const mlp_moe_t* p, const int* ids, void* plan, void* stream);

/* xs[pos[t, j]] = x[t]; every other row of xs is zero.
 *   x bf16 [T,H] in, xs bf16 [rows,H] out, not x */
int mlp_moe_dispatch(const mlp_moe_t* p, const void* plan, const void* x, void* xs, void* stream);

/* Its gradient: dx[t] = sum_j dxs[pos[t, j]] (fp32 sum, rounded once).
 *   dxs bf16 [rows,H] in, dx bf16 [T,H] out, not dxs */
int mlp_moe_dispatch_bwd(const mlp_moe_t* p, const void* plan, const void* dxs, void* dx,
                         void* stream);

/* out[t] = residual[t] + sum_j weights[t, j] y[pos[t, j]] (fp32, rounded once).
 *   y bf16 [rows,H], weights [T,top_k] (weights_type, aligned as that type),
 *   residual bf16 [T,H] or NULL, out bf16 [T,H] (may be residual itself, not y) */
int mlp_moe_combine(const mlp_moe_t* p, const void* plan, const void* y, const void* weights,
                    const void* residual, void* out, void* stream);

/* Its gradients: dy[pos[t, j]] = weights[t, j] dout[t], every other row of dy
 * zero; dweights[t, j] = sum_h dout[t,h] y[pos[t, j],h] (fp32 sum; 0 for a
 * dropped slot).  The sum cancels, and over a handful of slots y's rounding to
 * bf16 shows in it: up to MLP_MOE_FINE_SLOTS slots, after mlp_moe_experts_fwd
 * with this plan, it takes that call's fp32 values wherever they round to the y
 * given.  dy NULL: weights may be NULL; dweights NULL: y may be NULL.  dy is
 * neither dout nor y. */
int mlp_moe_combine_bwd(const mlp_moe_t* p, const void* plan, const void* dout, const void* y,
                        const void* weights, void* dy, void* dweights, void* stream);

/* Bytes of workspace of a call (0 on invalid arguments): MLP_MODE_FWD for
 * mlp_moe_experts_fwd, MLP_MODE_BWD for mlp_moe_experts_bwd, MLP_MODE_INFER
 * for mlp_moe_fwd_infer. */
size_t mlp_moe_workspace_size(const mlp_moe_t* p, int mode);

/* The experts' MLPs over the sorted rows, y[r] = MLP_e(xs[r]) for the rows r of
 * expert e (padding rows as any other).
 *   xs  bf16 [rows,H];  Wg, Wu bf16 [E,I,H] (Wu NULL when non-gated);
 *   Wd  bf16 [E,H,I];   y bf16 [rows,H] out
 *   G_save, U_save  bf16 [rows,I] out, optional: the preacts, for the backward
 * Rows from offsets[E] on are not written; y is not xs.  Up to MLP_MOE_FINE_SLOTS
 * slots the plan receives y in fp32, from a postact in two bf16 terms (calls with
 * such a plan do not run at the same time). */
int mlp_moe_experts_fwd(const mlp_moe_t* p, void* plan, const void* xs, const void* Wg,
                        const void* Wu, const void* Wd, void* y, void* G_save, void* U_save,
                        void* ws, size_t ws_bytes, void* stream);

/* Its gradients, from the saved preacts (which become dG, dU, as in mlp_bwd):
 *   dy   bf16 [rows,H] in, with zero padding rows (mlp_moe_combine_bwd's)
 *   dxs  bf16 [rows,H] out, neither dy nor xs where weight gradients are asked
 *        for; dWg, dWu [E,I,H], dWd [E,H,I]: bf16, or with
 *        fuse_grad_accum = 1 fp32 that the gradients are added to; each NULL
 *        to skip.  An expert without rows gets a zero gradient.
 * xs has zero padding rows (mlp_moe_dispatch's).  dxs is not written from
 * offsets[E] on. */
int mlp_moe_experts_bwd(const mlp_moe_t* p, const void* plan, const void* dy, const void* xs,
                        const void* Wg, const void* Wu, const void* Wd, void* G, void* U,
                        void* dxs, void* dWg, void* dWu, void* dWd, int fuse_grad_accum, void* ws,
                        size_t ws_bytes, void* stream);

/* The whole layer without gradients: sort, dispatch, experts, combine, with
 * everything between in the workspace.  Up to eight tokens (with at
 * most 128 slots and 1 GB of the experts' weights between them) stream the
 * weights of the experts they use instead, in two kernels.
 *   x bf16 [T,H], ids int32 [T,top_k], weights [T,top_k] (weights_type),
 *   residual bf16 [T,H] or NULL, out bf16 [T,H] (may be residual itself) */
int mlp_moe_fwd_infer(const mlp_moe_t* p, const void* x, const int* ids, const void* weights,
                      const void* Wg, const void* Wu, const void* Wd, const void* residual,
                      void* out, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MLP_GB300_MOE_H */
