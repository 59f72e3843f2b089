// The experts' derivative GEMM instances (dy Wd with the dgated / dact epilogue).
#include "gemm.cuh"

namespace mlpk {
template cudaError_t launch_gemm<EPI_DGATED, false, true, 1, ACT_SILU, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_DGATED, false, true, 1, ACT_SILU, true>();
template cudaError_t launch_gemm<EPI_DGATED, false, true, 2, ACT_SILU, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_DGATED, false, true, 2, ACT_SILU, true>();
template cudaError_t launch_gemm<EPI_DGATED, false, true, 1, ACT_RELU, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_DGATED, false, true, 1, ACT_RELU, true>();
template cudaError_t launch_gemm<EPI_DGATED, false, true, 2, ACT_RELU, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_DGATED, false, true, 2, ACT_RELU, true>();
template cudaError_t launch_gemm<EPI_DGATED, false, true, 1, ACT_GELU_EXP, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_DGATED, false, true, 1, ACT_GELU_EXP, true>();
template cudaError_t launch_gemm<EPI_DGATED, false, true, 2, ACT_GELU_EXP, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_DGATED, false, true, 2, ACT_GELU_EXP, true>();
template cudaError_t launch_gemm<EPI_DGATED, false, true, 1, ACT_SIGMOID, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_DGATED, false, true, 1, ACT_SIGMOID, true>();
template cudaError_t launch_gemm<EPI_DGATED, false, true, 2, ACT_SIGMOID, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_DGATED, false, true, 2, ACT_SIGMOID, true>();
template cudaError_t launch_gemm<EPI_DACT, false, true, 1, ACT_RELU_SQ, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_DACT, false, true, 1, ACT_RELU_SQ, true>();
template cudaError_t launch_gemm<EPI_DACT, false, true, 2, ACT_RELU_SQ, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_DACT, false, true, 2, ACT_RELU_SQ, true>();
template cudaError_t launch_gemm<EPI_DACT, false, true, 1, ACT_GELU_EXP, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_DACT, false, true, 1, ACT_GELU_EXP, true>();
template cudaError_t launch_gemm<EPI_DACT, false, true, 2, ACT_GELU_EXP, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_DACT, false, true, 2, ACT_GELU_EXP, true>();
template cudaError_t launch_gemm<EPI_DACT, false, true, 1, ACT_RELU, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_DACT, false, true, 1, ACT_RELU, true>();
template cudaError_t launch_gemm<EPI_DACT, false, true, 2, ACT_RELU, true>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_DACT, false, true, 2, ACT_RELU, true>();
}  // namespace mlpk
