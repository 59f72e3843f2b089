// The experts' GEMM instances over the sorted rows: gate/up and fc1 with their
// activation epilogues.
#include "gemm.cuh"

namespace mlpk {
template cudaError_t launch_gemm<EPI_GATED_FWD, false, false, 1, ACT_SILU, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_GATED_FWD, false, false, 1, ACT_SILU, true>();
template cudaError_t launch_gemm<EPI_GATED_FWD, false, false, 2, ACT_SILU, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_GATED_FWD, false, false, 2, ACT_SILU, true>();
template cudaError_t launch_gemm<EPI_GATED_FWD, false, false, 1, ACT_RELU, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_GATED_FWD, false, false, 1, ACT_RELU, true>();
template cudaError_t launch_gemm<EPI_GATED_FWD, false, false, 2, ACT_RELU, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_GATED_FWD, false, false, 2, ACT_RELU, true>();
template cudaError_t launch_gemm<EPI_GATED_FWD, false, false, 1, ACT_GELU_EXP, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_GATED_FWD, false, false, 1, ACT_GELU_EXP, true>();
template cudaError_t launch_gemm<EPI_GATED_FWD, false, false, 2, ACT_GELU_EXP, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_GATED_FWD, false, false, 2, ACT_GELU_EXP, true>();
template cudaError_t launch_gemm<EPI_GATED_FWD, false, false, 1, ACT_SIGMOID, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_GATED_FWD, false, false, 1, ACT_SIGMOID, true>();
template cudaError_t launch_gemm<EPI_GATED_FWD, false, false, 2, ACT_SIGMOID, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_GATED_FWD, false, false, 2, ACT_SIGMOID, true>();
template cudaError_t launch_gemm<EPI_ACT_FWD, false, false, 1, ACT_RELU_SQ, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_ACT_FWD, false, false, 1, ACT_RELU_SQ, true>();
template cudaError_t launch_gemm<EPI_ACT_FWD, false, false, 2, ACT_RELU_SQ, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_ACT_FWD, false, false, 2, ACT_RELU_SQ, true>();
template cudaError_t launch_gemm<EPI_ACT_FWD, false, false, 1, ACT_GELU_EXP, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_ACT_FWD, false, false, 1, ACT_GELU_EXP, true>();
template cudaError_t launch_gemm<EPI_ACT_FWD, false, false, 2, ACT_GELU_EXP, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_ACT_FWD, false, false, 2, ACT_GELU_EXP, true>();
template cudaError_t launch_gemm<EPI_ACT_FWD, false, false, 1, ACT_RELU, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_ACT_FWD, false, false, 1, ACT_RELU, true>();
template cudaError_t launch_gemm<EPI_ACT_FWD, false, false, 2, ACT_RELU, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_ACT_FWD, false, false, 2, ACT_RELU, true>();
}  // namespace mlpk
