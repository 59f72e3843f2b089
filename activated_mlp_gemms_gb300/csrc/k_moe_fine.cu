// The experts' GEMM instances for few slots: the postact in two bf16 terms, and the
// down projection that adds to y's fp32 rows.
#include "gemm.cuh"

namespace mlpk {
template cudaError_t launch_gemm<EPI_GATED_FINE, false, false, 1, ACT_SILU, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_GATED_FINE, false, false, 1, ACT_SILU, true>();
template cudaError_t launch_gemm<EPI_GATED_FINE, false, false, 1, ACT_RELU, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_GATED_FINE, false, false, 1, ACT_RELU, true>();
template cudaError_t launch_gemm<EPI_GATED_FINE, false, false, 1, ACT_GELU_EXP, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_GATED_FINE, false, false, 1, ACT_GELU_EXP, true>();
template cudaError_t launch_gemm<EPI_GATED_FINE, false, false, 1, ACT_SIGMOID, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_GATED_FINE, false, false, 1, ACT_SIGMOID, true>();
template cudaError_t launch_gemm<EPI_ACT_FINE, false, false, 1, ACT_RELU_SQ, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_ACT_FINE, false, false, 1, ACT_RELU_SQ, true>();
template cudaError_t launch_gemm<EPI_ACT_FINE, false, false, 1, ACT_GELU_EXP, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_ACT_FINE, false, false, 1, ACT_GELU_EXP, true>();
template cudaError_t launch_gemm<EPI_ACT_FINE, false, false, 1, ACT_RELU, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_ACT_FINE, false, false, 1, ACT_RELU, true>();
template cudaError_t launch_gemm<EPI_ACCUM_F32, false, false, 1, 0, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_ACCUM_F32, false, false, 1, 0, true>();
}  // namespace mlpk
