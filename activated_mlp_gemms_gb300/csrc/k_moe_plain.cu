// The experts' down projection (bf16, or fp32 for the inference layer's sum over
// a token's experts), input gradient and weight gradients (bf16 store, or added to
// fp32 gradients).
#include "gemm.cuh"

namespace mlpk {
template cudaError_t launch_gemm<EPI_STORE_BF16, false, false, 1, 0, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_STORE_BF16, false, false, 1, 0, true>();
template cudaError_t launch_gemm<EPI_STORE_BF16, false, false, 2, 0, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_STORE_BF16, false, false, 2, 0, true>();
template cudaError_t launch_gemm<EPI_STORE_BF16, false, true, 1, 0, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_STORE_BF16, false, true, 1, 0, true>();
template cudaError_t launch_gemm<EPI_STORE_BF16, false, true, 2, 0, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_STORE_BF16, false, true, 2, 0, true>();
template cudaError_t launch_gemm<EPI_STORE_BF16, true, true, 1, 0, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_STORE_BF16, true, true, 1, 0, true>();
template cudaError_t launch_gemm<EPI_STORE_BF16, true, true, 2, 0, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_STORE_BF16, true, true, 2, 0, true>();
template cudaError_t launch_gemm<EPI_ACCUM_F32, true, true, 1, 0, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_ACCUM_F32, true, true, 1, 0, true>();
template cudaError_t launch_gemm<EPI_ACCUM_F32, true, true, 2, 0, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_ACCUM_F32, true, true, 2, 0, true>();
template cudaError_t launch_gemm<EPI_STORE_F32, false, false, 1, 0, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_STORE_F32, false, false, 1, 0, true>();
template cudaError_t launch_gemm<EPI_STORE_F32, false, false, 2, 0, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_STORE_F32, false, false, 2, 0, true>();
}  // namespace mlpk
