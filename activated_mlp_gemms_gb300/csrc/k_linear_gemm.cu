// GEMM instances of the linear layer: bias, activation and residual in the
// epilogue; operands K-major.
#include "gemm.cuh"

namespace mlpk {
template cudaError_t launch_gemm<EPI_LINEAR, false, false, 1, ACT_NONE>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_LINEAR, false, false, 1, ACT_NONE>();
template cudaError_t launch_gemm<EPI_LINEAR, false, false, 2, ACT_NONE>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_LINEAR, false, false, 2, ACT_NONE>();
template cudaError_t launch_gemm<EPI_LINEAR, false, false, 1, ACT_RELU>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_LINEAR, false, false, 1, ACT_RELU>();
template cudaError_t launch_gemm<EPI_LINEAR, false, false, 2, ACT_RELU>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_LINEAR, false, false, 2, ACT_RELU>();
template cudaError_t launch_gemm<EPI_LINEAR, false, false, 1, ACT_RELU_SQ>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_LINEAR, false, false, 1, ACT_RELU_SQ>();
template cudaError_t launch_gemm<EPI_LINEAR, false, false, 2, ACT_RELU_SQ>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_LINEAR, false, false, 2, ACT_RELU_SQ>();
template cudaError_t launch_gemm<EPI_LINEAR, false, false, 1, ACT_GELU_EXP>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_LINEAR, false, false, 1, ACT_GELU_EXP>();
template cudaError_t launch_gemm<EPI_LINEAR, false, false, 2, ACT_GELU_EXP>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_LINEAR, false, false, 2, ACT_GELU_EXP>();
template cudaError_t launch_gemm<EPI_LINEAR, false, false, 1, ACT_SILU_EXP>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_LINEAR, false, false, 1, ACT_SILU_EXP>();
template cudaError_t launch_gemm<EPI_LINEAR, false, false, 2, ACT_SILU_EXP>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_LINEAR, false, false, 2, ACT_SILU_EXP>();
template cudaError_t launch_gemm<EPI_LINEAR, false, false, 1, ACT_SIGMOID_EXP>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_LINEAR, false, false, 1, ACT_SIGMOID_EXP>();
template cudaError_t launch_gemm<EPI_LINEAR, false, false, 2, ACT_SIGMOID_EXP>(const Params&, int, cudaStream_t, bool);
template int max_groups<EPI_LINEAR, false, false, 2, ACT_SIGMOID_EXP>();
}  // namespace mlpk
