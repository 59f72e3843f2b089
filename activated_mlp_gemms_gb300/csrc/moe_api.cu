// moe_api.cu -- the C entry points of mlp_moe.h: argument validation and the
// launch sequences of the mixture-of-experts MLP.
#include "mlp_moe.h"

#include "host.h"
#include "moe.h"

using namespace mlpk;

namespace {

int check_moe(const mlp_moe_t* p) {
  if (!p) return MLP_ERR_INVALID_ARG;
  if (p->T <= 0 || p->E <= 0 || p->top_k <= 0 || p->H <= 0) return MLP_ERR_INVALID_ARG;
  if (p->weights_type != MLP_MOE_W_F32 && p->weights_type != MLP_MOE_W_BF16)
    return MLP_ERR_INVALID_ARG;
  if (p->H % 8) return MLP_ERR_ALIGNMENT;
  if (p->E > MLP_MOE_MAX_EXPERTS || p->top_k > MLP_MOE_MAX_TOP_K) return MLP_ERR_UNSUPPORTED;
  // rows and slots are 32-bit; the token kernels' grids too
  if ((long long)p->T * p->top_k > (1LL << 30) || (long long)p->T * p->H >= (1LL << 40))
    return MLP_ERR_UNSUPPORTED;
  return MLP_OK;
}

MoePlan plan_of(const mlp_moe_t* p) { return moe_plan(p->T, p->E, p->top_k); }

// int32 ids and the routing weights: 4-byte aligned
int need4(const void* ptr) {
  if (!ptr) return MLP_ERR_INVALID_ARG;
  return (reinterpret_cast<uintptr_t>(ptr) & 3u) ? MLP_ERR_ALIGNMENT : MLP_OK;
}

bool w_bf16(const mlp_moe_t* p) { return p->weights_type == MLP_MOE_W_BF16; }

}  // namespace

extern "C" {

long long mlp_moe_rows(const mlp_moe_t* p) {
  return check_moe(p) == MLP_OK ? plan_of(p).rows : 0;
}

int mlp_moe_plan_layout(const mlp_moe_t* p, mlp_moe_plan_t* layout) {
  MLP_TRY(check_moe(p));
  if (!layout) return MLP_ERR_INVALID_ARG;
  const MoePlan L = plan_of(p);
  layout->ints = L.ints;
  layout->offsets = L.offsets;
  layout->counts = L.counts;
  layout->pos = L.pos;
  layout->src = L.src;
  return MLP_OK;
}

int mlp_moe_sort(const mlp_moe_t* p, const int* ids, void* plan, void* stream) {
  MLP_TRY(check_moe(p));
  MLP_TRY(need4(ids));
  MLP_TRY(need(plan));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(MLP_KERNEL_MOE_SORT, s, [&] {
    return launch_moe_sort(ids, static_cast<int*>(plan), plan_of(p), p->E, s, false);
  });
}

int mlp_moe_dispatch(const mlp_moe_t* p, const void* plan, const void* x, void* xs, void* stream) {
  MLP_TRY(check_moe(p));
  MLP_TRY(need(plan));
  MLP_TRY(need(x));
  MLP_TRY(need(xs));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(MLP_KERNEL_MOE_DISPATCH, s, [&] {
    return launch_moe_dispatch(x, static_cast<const int*>(plan), plan_of(p), p->T, p->top_k, p->H,
                               xs, s, false);
  });
}

int mlp_moe_dispatch_bwd(const mlp_moe_t* p, const void* plan, const void* dxs, void* dx,
                         void* stream) {
  MLP_TRY(check_moe(p));
  MLP_TRY(need(plan));
  MLP_TRY(need(dxs));
  MLP_TRY(need(dx));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(MLP_KERNEL_MOE_COMBINE, s, [&] {
    return launch_moe_combine(dxs, static_cast<const int*>(plan), plan_of(p), p->T, p->top_k, p->H,
                              nullptr, false, nullptr, dx, s, false);
  });
}

int mlp_moe_combine(const mlp_moe_t* p, const void* plan, const void* y, const void* weights,
                    const void* residual, void* out, void* stream) {
  MLP_TRY(check_moe(p));
  MLP_TRY(need(plan));
  MLP_TRY(need(y));
  MLP_TRY(need4(weights));
  MLP_TRY(opt(residual));
  MLP_TRY(need(out));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(MLP_KERNEL_MOE_COMBINE, s, [&] {
    return launch_moe_combine(y, static_cast<const int*>(plan), plan_of(p), p->T, p->top_k, p->H,
                              weights, w_bf16(p), residual, out, s, false);
  });
}

int mlp_moe_combine_bwd(const mlp_moe_t* p, const void* plan, const void* dout, const void* y,
                        const void* weights, void* dy, void* dweights, void* stream) {
  MLP_TRY(check_moe(p));
  MLP_TRY(need(plan));
  MLP_TRY(need(dout));
  if (dy) {
    MLP_TRY(need(dy));
    MLP_TRY(need4(weights));
  }
  if (dweights) {
    MLP_TRY(need4(dweights));
    MLP_TRY(need(y));
  }
  if (!dy && !dweights) return MLP_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(MLP_KERNEL_MOE_COMBINE_BWD, s, [&] {
    return launch_moe_combine_bwd(dout, y, static_cast<const int*>(plan), plan_of(p), p->T,
                                  p->top_k, p->H, weights, w_bf16(p), dy, dweights, s, false);
  });
}

}  // extern "C"
