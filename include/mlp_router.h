/*
 * mlp_router.h -- C ABI of the router of a mixture of experts, of libmlp.so:
 * which experts a token's slots take, their routing weights, how many slots
 * each expert gets, the balance loss, and the logits' gradient.  Its ids and
 * weights are what mlp_moe_sort and the calls after it take (mlp_moe.h).  An
 * addition of this library; the conventions of mlp.h (ownership, streams,
 * return values, workspace, determinism) hold here.
 *
 *   p[t,:]    = softmax(logits[t,:])
 *   ids[t,:]  = the top_k largest logits' experts, the largest first, of equals
 *               the lowest
 *   w[t,j]    = p[t, ids[t,j]], with renormalize divided by their sum over j
 *   counts[e] = slots whose id is e
 *   loss      = E sum_e f[e] P[e],  f[e] = counts[e] / (top_k N) (a constant for
 *               the gradient), P[e] = sum_t p[t,e] / N, N the routed tokens
 *
 * A token is routed unless its mask is 0 or all its logits are -inf; one that
 * is not has ids -1 and weights 0, adds nothing to counts, loss and N, and its
 * logits' gradient is 0.  An expert at -inf is never chosen: a routed token
 * with fewer than top_k experts left has ids -1 and weights 0 behind them.  A
 * NaN counts as the largest value and makes its token's weights NaN.
 *
 * Arithmetic in fp32, with the hardware's base-2 exponential (within 2^-22 of its
 * value) and reciprocal (2^-23).  A weight is within (2.3 d + 49) 2^-24 of its value,
 * beside its type's rounding, where d is its logit's distance from the token's
 * largest (measured 3e-8 to 9e-8 of it in the mean square); one below 2^-126 may be
 * zero.  Sums over tokens are sums of fp32; the derivatives behind the loss have six
 * roundings.
 */
#ifndef MLP_GB300_ROUTER_H
#define MLP_GB300_ROUTER_H

#include "mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MLP_ROUTER_F32 = 0, MLP_ROUTER_BF16 = 1 } mlp_router_type_t;

/* T tokens, E experts (at most 1024), top_k slots a token (at most E and 64). */
typedef struct {
  int T, E, top_k;
  int renormalize;   /* 0 or 1 */
  int logits_type;   /* mlp_router_type_t: of logits and dlogits */
  int weights_type;  /* mlp_router_type_t: of weights and dweights */
  int ldl, ldd;      /* row pitch in values of logits and of dlogits, 0 for dense; at least E */
} mlp_router_t;

/* Bytes of workspace of mlp_moe_router_fwd with counts or balance; 0 on invalid
 * arguments. */
size_t mlp_moe_router_workspace_size(const mlp_router_t* p);

/* Forward.  Every pointer is aligned as its type.
 *   logits   [T,E] (logits_type, pitch ldl)
 *   mask     uint8 [T] or NULL: 0 for a token that is not routed (padding)
 *   ids      int32 [T,top_k] out;  weights [T,top_k] (weights_type) out
 *   counts   int32 [E] out or NULL
 *   balance  fp32 [E + 1] out or NULL: the loss, then d loss / d p[t,e] for each
 *            expert (the same for every routed token), which the backward takes
 *   ws       256-byte aligned; NULL where counts and balance both are
 * No output may overlap an operand or another output.  The sums over tokens do not
 * depend on any order of arrival: two calls with the same operands give the same bits. */
int mlp_moe_router_fwd(const mlp_router_t* p, const void* logits, const unsigned char* mask,
                       int* ids, void* weights, int* counts, float* balance, void* ws,
                       size_t ws_bytes, void* stream);

/* Backward: the gradient of logits from those of weights and of the loss.
 *   ids      the forward's
 *   balance  the forward's, or NULL with dloss
 *   dweights [T,top_k] (weights_type) or NULL;  dloss fp32 [1] (on the device) or NULL
 *   dlogits  [T,E] (logits_type, pitch ldd) out; may be logits itself (then ldd = ldl),
 *            and overlaps no other operand
 * (An id outside [0, E) takes no part.) */
int mlp_moe_router_bwd(const mlp_router_t* p, const void* logits, const unsigned char* mask,
                       const int* ids, const float* balance, const void* dweights,
                       const float* dloss, void* dlogits, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MLP_GB300_ROUTER_H */
