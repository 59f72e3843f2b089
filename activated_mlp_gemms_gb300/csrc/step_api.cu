// step_api.cu -- the C entry points of mlp_router.h and mlp_norm.h: argument
// validation, workspace layout and launch sequences.
#include <algorithm>
#include <initializer_list>

#include "host.h"
#include "mlp_norm.h"
#include "mlp_router.h"
#include "step.h"

using namespace mlpk;

namespace {

int need_as(const void* ptr, uintptr_t size) {
  if (!ptr) return MLP_ERR_INVALID_ARG;
  return reinterpret_cast<uintptr_t>(ptr) % size ? MLP_ERR_ALIGNMENT : MLP_OK;
}
int opt_as(const void* ptr, uintptr_t size) { return ptr ? need_as(ptr, size) : MLP_OK; }

// Whether an output (or NULL) is one of the others.
bool any(const void* o, std::initializer_list<const void*> of) {
  return o && std::find(of.begin(), of.end(), o) != of.end();
}

int check_ws(size_t total, const void* ws, size_t ws_bytes) {
  if (!ws) return MLP_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return MLP_ERR_ALIGNMENT;
  return ws_bytes < total ? MLP_ERR_WORKSPACE_TOO_SMALL : MLP_OK;
}

// ------------------------------------------------------------------ router
int check_router(const mlp_router_t* p) {
  if (!p) return MLP_ERR_INVALID_ARG;
  if (p->T <= 0 || p->E <= 0 || p->top_k <= 0 || p->top_k > p->E) return MLP_ERR_INVALID_ARG;
  if (p->renormalize != 0 && p->renormalize != 1) return MLP_ERR_INVALID_ARG;
  auto type = [](int t) { return t == MLP_ROUTER_F32 || t == MLP_ROUTER_BF16; };
  if (!type(p->logits_type) || !type(p->weights_type)) return MLP_ERR_INVALID_ARG;
  if ((p->ldl && p->ldl < p->E) || (p->ldd && p->ldd < p->E)) return MLP_ERR_INVALID_ARG;
  if (p->E > ROUTER_MAX_EXPERTS || p->top_k > ROUTER_MAX_TOP_K) return MLP_ERR_UNSUPPORTED;
  // as mlp_moe.h's slots
  if ((long long)p->T * p->top_k > (1LL << 30)) return MLP_ERR_UNSUPPORTED;
  return MLP_OK;
}
RouterArgs args_of(const mlp_router_t* p, const void* logits, const unsigned char* mask) {
  return RouterArgs{logits,
                    mask,
                    p->T,
                    p->E,
                    p->top_k,
                    p->renormalize,
                    p->logits_type == MLP_ROUTER_BF16,
                    p->weights_type == MLP_ROUTER_BF16,
                    p->ldl ? p->ldl : p->E,
                    p->ldd ? p->ldd : p->E};
}
uintptr_t size_of(int type) { return type == MLP_ROUTER_BF16 ? 2 : 4; }

// After the control block (of which only the status word is used): one set of sums a block.
struct RouterLayout {
  size_t n, c, p, total;
};
RouterLayout router_layout(const mlp_router_t* p) {
  const size_t blocks = router_blocks(p->T, p->E);
  RouterLayout w;
  w.n = CTRL_BYTES;
  w.c = w.n + round256(blocks * 4);
  w.p = w.c + round256(blocks * p->E * 4);
  w.total = w.p + round256(blocks * p->E * 4);
  return w;
}

// -------------------------------------------------------------- layer norm
int check_norm(const mlp_layernorm_t* p) {
  if (!p) return MLP_ERR_INVALID_ARG;
  if (p->M <= 0 || p->H <= 0) return MLP_ERR_INVALID_ARG;
  if (!std::isfinite(p->eps) || p->eps < 0.f) return MLP_ERR_INVALID_ARG;
  auto type = [](int t) { return t == MLP_NORM_F32 || t == MLP_NORM_BF16; };
  if (!type(p->type) || !type(p->weight_type)) return MLP_ERR_INVALID_ARG;
  if ((p->ldx && p->ldx < p->H) || (p->ldr && p->ldr < p->H)) return MLP_ERR_INVALID_ARG;
  if (p->H % 8 || p->ldx % 8 || p->ldr % 8) return MLP_ERR_ALIGNMENT;
  if (p->H > NORM_MAX_H) return MLP_ERR_UNSUPPORTED;
  return MLP_OK;
}
static_assert(NORM_MAX_H == MLP_NORM_MAX_H, "one limit");

NormArgs norm_args(const mlp_layernorm_t* p) {
  return NormArgs{p->M,
                  p->H,
                  p->eps,
                  p->type == MLP_NORM_BF16,
                  p->weight_type == MLP_NORM_BF16,
                  p->ldx ? p->ldx : p->H,
                  p->ldr ? p->ldr : p->H};
}
size_t norm_total(const mlp_layernorm_t* p) {
  return CTRL_BYTES + round256((size_t)layernorm_blocks(p->M, p->H, p->type == MLP_NORM_BF16) * 2 * p->H * 4);
}

}  // namespace

extern "C" {

size_t mlp_moe_router_workspace_size(const mlp_router_t* p) {
  return check_router(p) == MLP_OK ? router_layout(p).total : 0;
}

int mlp_moe_router_fwd(const mlp_router_t* p, const void* logits, const unsigned char* mask,
                       int* ids, void* weights, int* counts, float* balance, void* ws,
                       size_t ws_bytes, void* stream) {
  MLP_TRY(check_router(p));
  MLP_TRY(need_as(logits, size_of(p->logits_type)));
  MLP_TRY(need_as(ids, 4));
  MLP_TRY(need_as(weights, size_of(p->weights_type)));
  MLP_TRY(opt_as(counts, 4));
  MLP_TRY(opt_as(balance, 4));
  const bool sums = counts || balance;
  const RouterLayout w = router_layout(p);
  if (sums) MLP_TRY(check_ws(w.total, ws, ws_bytes));
  // one token's results over another's logits, or over each other
  if (any(ids, {logits, mask, weights, counts, balance}) ||
      any(weights, {logits, mask, counts, balance}) || any(counts, {logits, mask, balance}) ||
      any(balance, {logits, mask}))
    return MLP_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* at = static_cast<char*>(ws);
  RouterParts parts = {};
  if (sums)
    parts = {reinterpret_cast<int*>(at + w.n), reinterpret_cast<int*>(at + w.c),
             reinterpret_cast<float*>(at + w.p)};
  MLP_TRY(traced(MLP_KERNEL_ROUTER, s, [&] {
    return launch_router_fwd(args_of(p, logits, mask), ids, weights, counts, balance, parts,
                             sums ? static_cast<int*>(ws) : nullptr, s);
  }));
  if (!sums || router_blocks(p->T, p->E) == 1) return MLP_OK;
  return traced(MLP_KERNEL_ROUTER, s, [&] {
    return launch_router_finish(p->T, p->E, p->top_k, parts, counts, balance, s);
  });
}

int mlp_moe_router_bwd(const mlp_router_t* p, const void* logits, const unsigned char* mask,
                       const int* ids, const float* balance, const void* dweights,
                       const float* dloss, void* dlogits, void* stream) {
  MLP_TRY(check_router(p));
  MLP_TRY(need_as(logits, size_of(p->logits_type)));
  MLP_TRY(need_as(dlogits, size_of(p->logits_type)));
  MLP_TRY(opt_as(dweights, size_of(p->weights_type)));
  MLP_TRY(opt_as(dloss, 4));
  if (dweights) MLP_TRY(need_as(ids, 4));
  if (dloss) MLP_TRY(need_as(balance, 4));
  const RouterArgs a = args_of(p, logits, mask);
  if (dlogits == logits && a.ldl != a.ldd) return MLP_ERR_INVALID_ARG;
  // one token's gradient over what another's is computed from
  if (any(dlogits, {mask, ids, balance, dweights, dloss})) return MLP_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(MLP_KERNEL_ROUTER_BWD, s, [&] {
    return launch_router_bwd(a, ids, balance, dweights, dloss, dlogits, s);
  });
}

size_t mlp_layernorm_workspace_size(const mlp_layernorm_t* p) {
  return check_norm(p) == MLP_OK ? norm_total(p) : 0;
}

int mlp_layernorm_fwd(const mlp_layernorm_t* p, const void* x, const void* residual,
                      const void* weight, const void* bias, void* y, void* h, float* mean,
                      float* rstd, void* stream) {
  MLP_TRY(check_norm(p));
  MLP_TRY(need(x));
  MLP_TRY(opt(residual));
  MLP_TRY(opt(weight));
  MLP_TRY(opt(bias));
  MLP_TRY(need(y));
  MLP_TRY(opt(h));
  MLP_TRY(opt_as(mean, 4));
  MLP_TRY(opt_as(rstd, 4));
  const NormArgs a = norm_args(p);
  // a pitched input is read while other rows of a dense output are written
  auto over = [&](const void* o) {
    return (o == x && a.ldx != p->H) || (o == residual && a.ldr != p->H);
  };
  if (y == h || over(y) || (h && over(h))) return MLP_ERR_INVALID_ARG;
  // one row's results over what another row reads
  if (any(y, {weight, bias}) || any(h, {weight, bias}) ||
      any(mean, {x, residual, weight, bias, y, h, rstd}) ||
      any(rstd, {x, residual, weight, bias, y, h}))
    return MLP_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(MLP_KERNEL_LAYERNORM, s, [&] {
    return launch_layernorm_fwd(a, x, residual, weight, bias, y, h, mean, rstd, s);
  });
}

int mlp_layernorm_bwd(const mlp_layernorm_t* p, const void* dy, const void* h, const void* weight,
                      const float* mean, const float* rstd, const void* dh, void* dx,
                      void* dweight, void* dbias, int fuse_grad_accum, void* ws, size_t ws_bytes,
                      void* stream) {
  MLP_TRY(check_norm(p));
  if (fuse_grad_accum != 0 && fuse_grad_accum != 1) return MLP_ERR_INVALID_ARG;
  MLP_TRY(need(dy));
  MLP_TRY(need(h));
  MLP_TRY(opt(weight));
  MLP_TRY(need_as(mean, 4));
  MLP_TRY(need_as(rstd, 4));
  MLP_TRY(opt(dh));
  MLP_TRY(opt(dx));
  MLP_TRY(opt(dweight));
  MLP_TRY(opt(dbias));
  const bool sums = dweight || dbias;
  if (sums) MLP_TRY(check_ws(norm_total(p), ws, ws_bytes));
  if (!dx && !sums) return MLP_OK;
  if (dx == h) return MLP_ERR_INVALID_ARG;
  // (a weight's gradient may go over the weight: it is written when all rows are done)
  if (any(dx, {weight, mean, rstd, dweight, dbias}) || any(dweight, {dbias}))
    return MLP_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* part = sums ? reinterpret_cast<float*>(static_cast<char*>(ws) + CTRL_BYTES) : nullptr;
  MLP_TRY(traced(MLP_KERNEL_LAYERNORM_BWD, s, [&] {
    return launch_layernorm_bwd(norm_args(p), dy, h, weight, mean, rstd, dh, dx, part,
                                sums ? static_cast<int*>(ws) : nullptr, s);
  }));
  if (!sums) return MLP_OK;
  return traced(MLP_KERNEL_LAYERNORM_SUMS, s, [&] {
    return launch_layernorm_sums(p->H, layernorm_blocks(p->M, p->H, p->type == MLP_NORM_BF16), part, dweight, dbias,
                                 p->weight_type == MLP_NORM_BF16, fuse_grad_accum == 1, s);
  });
}

}  // extern "C"
