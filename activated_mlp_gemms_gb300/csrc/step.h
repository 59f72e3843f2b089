// step.h -- launchers of the kernels around the experts' MLP in a training step:
// the router and the layer norm.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

namespace mlpk {

// A kernel as a type, so that what is set up once for it has a place.
template <auto KERNEL>
struct KernelOf {
  static constexpr auto kernel = KERNEL;
  // Allows `most` bytes of dynamic shared memory, once a device.
  static cudaError_t allow_smem(int most) {
    static std::atomic<unsigned long long> done{0};  // devices
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load() >> dev & 1))) return e;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev);
    return e;
  }
};

// ------------------------------------------------------------------ router
constexpr int ROUTER_MAX_EXPERTS = 1024;
constexpr int ROUTER_MAX_TOP_K = 64;
struct RouterArgs {
  const void* logits;
  const unsigned char* mask;
  int T, E, top_k, renorm;
  bool l_bf16, w_bf16;
  int ldl, ldd;
};
// Partial sums over the tokens, one set a block (blocks = router_blocks): the routed
// tokens [blocks], the slots of each expert [blocks, E], the probabilities' sums [blocks, E].
int router_blocks(int T, int E);
struct RouterParts {
  int* n;
  int* c;
  float* p;
};
// parts.n null: neither counts nor balance are wanted
cudaError_t launch_router_fwd(const RouterArgs& a, int* ids, void* weights, int* counts,
                              float* balance, const RouterParts& parts, int* status,
                              cudaStream_t stream);
cudaError_t launch_router_finish(int T, int E, int top_k, const RouterParts& parts, int* counts,
                                 float* balance, cudaStream_t stream);
cudaError_t launch_router_bwd(const RouterArgs& a, const int* ids, const float* balance,
                              const void* dweights, const float* dloss, void* dlogits,
                              cudaStream_t stream);

// -------------------------------------------------------------- layer norm
constexpr int NORM_MAX_H = 16384;
struct NormArgs {
  int M, H;
  float eps;
  bool bf16, w_bf16;
  long long ldx, ldr;
};
cudaError_t launch_layernorm_fwd(const NormArgs& a, const void* x, const void* residual,
                                 const void* weight, const void* bias, void* y, void* h,
                                 float* mean, float* rstd, cudaStream_t stream);
// Blocks of the backward where dweight or dbias is wanted: each leaves its rows' sums in
// part fp32 [blocks, 2, H] (dweight's, dbias's), which the second kernel adds up.
int layernorm_blocks(int M, int H, bool bf16);
cudaError_t launch_layernorm_bwd(const NormArgs& a, const void* dy, const void* h,
                                 const void* weight, const float* mean, const float* rstd,
                                 const void* dh, void* dx, float* part, int* status,
                                 cudaStream_t stream);
cudaError_t launch_layernorm_sums(int H, int blocks, const float* part, void* dweight, void* dbias,
                                  bool w_bf16, bool accum, cudaStream_t stream);

}  // namespace mlpk
