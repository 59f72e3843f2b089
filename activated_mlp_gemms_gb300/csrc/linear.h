// linear.h -- launchers of the linear layer's own kernels (the GEMM instances
// with its epilogue are launch_gemm<EPI_LINEAR, ...>).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>

#include "gemm_params.h"

namespace mlpk {

// out = act(x W^T + bias) + rs * resid for 1 <= M <= LINEAR_STREAM_MAX_M rows
// (`act` a device activation; bias, resid, pre may be null).  Clears *status.
constexpr int LINEAR_STREAM_MAX_M = 8;
cudaError_t launch_linear_stream(const void* x, int ldx, const void* W, const void* bias,
                                 const void* resid, int ldr, float rs, void* out, int ldo,
                                 void* pre, int M, int N, int K, int act, cudaStream_t stream,
                                 bool pdl, int* status);

// The same on the tensor cores with the operands' places changed
// (k_linear_skinny.cu): CTAs of 128 features by up to 256 rows.  map_w: W [N, K]
// in boxes {64, 128}; w_mn (dx = dz W, with ACT_NONE and no bias or residual):
// W [K, N], N its contiguous features, in boxes {64, 64}; map_x: x [M, K] in boxes
// {64, mp}.  clear: clears *status; no_work: the bounded waits run out (testing).
struct SkinnyShape {
  int blocks, tiles, mp;  // blocks of 128 features; tiles of mp rows
  int share;              // CTAs that share a block's K, at most
};
SkinnyShape linear_skinny_shape(int M, int N, int K);
cudaError_t launch_linear_skinny(const CUtensorMap& map_w, const CUtensorMap& map_x,
                                 const void* bias, const void* resid, int ldr, float rs, void* out,
                                 int ldo, void* pre, int M, int N, int K, int act, bool w_mn,
                                 bool clear, int no_work, int* status, unsigned long long limit_ns,
                                 cudaStream_t stream, bool pdl);

// dz = dout * act'(pre) into dz (bf16 [M, N] dense; null: not written) and the
// column sums of dz over each chunk of rows into part fp32 [chunks, N] (null:
// not formed); then db[n] = sum over chunks (bf16), or db[n] += (fp32).  With
// one chunk the first writes db itself.  Clears *status (null: not).
int linear_db_chunks(int M, int N);
cudaError_t launch_linear_dact(const void* dout, int ldd, const void* pre, void* dz, float* part,
                               void* db, bool accum, int M, int N, int act, int* status,
                               cudaStream_t stream, bool pdl);
cudaError_t launch_linear_db(const float* part, int chunks, void* db, int N, bool accum,
                             cudaStream_t stream, bool pdl);

}  // namespace mlpk
