// ortho.h -- launchers of the orthogonalised update's kernels (mlp_ortho.h).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mlpk {

// X, A and P = b A + c A A are fp16 at these powers of two.  With singular values s below 2 X's
// entries stay below 2^15, A's too, and P's below 2^16 where |b s^2 + c s^4| < 8 (Muon's
// coefficients: s < 1.3, P < 2.8).  At the other end, what a matrix's typical entry is (1 / sqrt(m
// n) of X at the start, 1 / (m sqrt(n)) of A off its diagonal) and the second terms, 2^-11 of it,
// should stay above fp16's smallest steps, 2^-24: with A at 2^11 an fp32 result of 4864 x 2048
// was off by 1.0e-5.
constexpr float ORTHO_X = 16384.f, ORTHO_A = 8192.f;

constexpr int ORTHO_PARTS = 256;  // partial sums of a matrix's norm

// One product D = alpha in + beta P Q of a stack, P [M, K] K-major, Q [N, K] K-major or
// [K, N]; the three products hi lo + lo hi + hi hi with `terms` 2.
enum OrthoKind : int {
  ORTHO_SYM = 0,   // D symmetric (P is Q), in d_terms terms: the tiles on and below the diagonal,
                   // and their mirror images
  ORTHO_STEP = 1,  // Q is [K, N]; in and D in two terms
  ORTHO_LAST = 2   // the same, D the result: bf16 or fp32, as it is or transposed
};
struct OrthoGemm {
  CUtensorMap p, q;   // depth terms x batch
  CUtensorMap in, d;  // in 32 x 32 boxes
  const void* in_ptr;  // the same, for the kernel of few units
  void* d_ptr;
  int ld_in, ld_d;     // their row pitches
  int M, N, kblocks, terms, batch;
  int d_terms;  // of D where it is symmetric
  int chunk;    // with two terms: k-blocks that an accumulator sums up
  int tiles_m, tiles_n, units;
  float alpha, beta;  // alpha 0: no `in`
  int out_bf16, transposed;
  int backwards;  // the stack from its last matrix to its first
  int* status;
  unsigned long long timeout_ns;
  int debug_flags;
};
// cg 2: CTA pairs, 256 x 256 tiles; 1: single CTAs, 128 x 128 tiles.
cudaError_t launch_ortho_gemm(const OrthoGemm& g, int cg, OrthoKind kind, cudaStream_t stream);
// 256 x 256 tiles of a symmetric product, the k-blocks (at least two) shared by two CTA pairs; how
// many of their clusters are resident together (0: not known).
cudaError_t launch_ortho_pairs(const OrthoGemm& g, cudaStream_t stream);
int ortho_pairs_clusters();
// 128 x 128 tiles whose k-blocks are shared by clusters of `share` CTAs (2, 4 or 8, at most
// half of the k-blocks).
cudaError_t launch_ortho_split(const OrthoGemm& g, int share, OrthoKind kind, cudaStream_t stream);

// The whole call for matrices whose lesser side is at most 128: a cluster of CTAs keeps a matrix's
// X in shared memory, `width` (128 or 256) columns each, from G to the result.
constexpr int ORTHO_SMALL_M = 128, ORTHO_SMALL_CTAS = 8;
struct OrthoSmall {
  const void* G;
  void* out;
  int m, n, batch, steps, terms, transposed;  // transposed: G and out are [n, m]
  int bf16, out_bf16;
  float a, b, c, eps, scale;
  int* status;
  unsigned long long timeout_ns;
  int debug_flags;
};
cudaError_t launch_ortho_small(const OrthoSmall& g, int width, cudaStream_t stream);

// part [batch, ORTHO_PARTS] = sums of squares of G's matrices; clears *status.
cudaError_t launch_ortho_norm(const void* G, bool bf16, long long size, int batch, float* part,
                              int* status, cudaStream_t stream);
// X = ORTHO_X G / (|G| + eps) in two fp16 terms [2, batch, m, n] with a row pitch, transposed
// where rows > cols.
cudaError_t launch_ortho_scale(const void* G, bool bf16, int rows, int cols, int batch, int pitch,
                               const float* part, float eps, void* X, cudaStream_t stream);

}  // namespace mlpk
