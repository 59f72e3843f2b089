/*
 * mlp_ortho.h -- C ABI of the orthogonalised update of libmlp.so: a gradient or
 * momentum G of a weight matrix, or of a stack of them (the experts'), brought
 * near the orthogonal matrix of its own singular vectors by Newton-Schulz
 * products, as the Muon optimiser does with a linear layer's update (the
 * optimiser of modded-nanogpt's training script):
 *
 *   X = G / (|G| + eps)                      |G| the Frobenius norm of one matrix
 *   X <- a X + (b A + c A A) X,  A = X X^T   `steps` times
 *   out = scale * X
 *
 * (G with more rows than columns: the same with X^T X on the other side.)  An
 * addition of this library; the conventions of mlp.h (ownership, streams,
 * alignment, return values, workspace, device-side errors, determinism) hold
 * here.
 */
#ifndef MLP_GB300_ORTHO_H
#define MLP_GB300_ORTHO_H

#include "mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MLP_ORTHO_F32 = 0, MLP_ORTHO_BF16 = 1 } mlp_ortho_type_t;

/* A stack of `batch` matrices [rows, cols] (dense), rows and cols multiples of
 * 8, the lesser of them at most 32768.  coeff: a, b, c; they keep every singular
 * value s below 2 and |b s^2 + c s^4| below 8 (those of the Muon optimiser, 3.4445,
 * -4.7750, 2.0315, below 1.3 and 2.8; what leaves that range comes out infinite or
 * NaN).  steps 1 to 32; eps >= 0.
 *
 * Arithmetic: X and A are held as fp16 at fixed powers of two, X with the remainder
 * of its rounding beside it, the products summed in fp32.  A bf16 out takes the
 * products of the leading terms, and up to 128 rows (the lesser side) both terms in the
 * last product of a step.  Its rounding alone is 1.7e-3 of its Frobenius norm; the result
 * is off by 1.7e-3 to 2.2e-3 up to 128 rows (up to 3.5e-3 below 64), by 2.0e-3 to 3.4e-3
 * above (4.4e-3 where all singular values are equal), whichever way it is computed, alone
 * or in a stack.  An fp32 out takes those with the remainders too: 22 bits of X, A and P.  It
 * is off by 0.5e-6 to 5e-6 for momenta, as products of fp32 are (at most 1.8 times those: 64 x
 * 4096 1.7e-6 and 1.0e-6); by 5e-5 where a few directions stand over 1e-2 of noise, and by
 * 1.6e-4 where all but a few singular values are zero (fp32 products: 3e-5 to 6e-5, 4e-4).
 * |G| is summed in fp32: entries above 1e19 overflow
 * it, and of a G whose entries are all below 1e-19 it is lost (the result is then G / eps's:
 * zero, but not with an eps of 0). */
typedef struct {
  int rows, cols, batch;
  int steps;
  float coeff[3];
  float eps, scale;
  int type;      /* mlp_ortho_type_t of G */
  int out_type;  /* mlp_ortho_type_t of out */
} mlp_ortho_t;

/* Bytes of workspace; 0 on invalid arguments. */
size_t mlp_ortho_workspace_size(const mlp_ortho_t* p);

/*   G [batch, rows, cols] in;  out [batch, rows, cols] out (may be G itself where the
 *   types are the same) */
int mlp_orthogonalize(const mlp_ortho_t* p, const void* G, void* out, void* ws, size_t ws_bytes,
                      void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MLP_GB300_ORTHO_H */
