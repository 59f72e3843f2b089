// Token rows to their places in the sorted layout and back:
//   k_moe_dispatch     xs[pos[t, j]] = x[t], zeros in the other rows
//   k_moe_combine      out[t] = residual[t] + sum_j w[t, j] y[pos[t, j]]
//                      (without weights: the gradient of the dispatch)
//   k_moe_combine_bwd  dy[pos[t, j]] = w[t, j] dout[t] (zeros in the other
//                      rows), dw[t, j] = sum_h dout[t, h] y[pos[t, j], h]
// All are bound by HBM: every row is read once and written once.  The work
// goes by token, not by sorted row, so that a token's row (or its gradient)
// is read once for all its slots and the sum over its slots needs no atomic
// (the same bits on every run).  Sums are fp32 and rounded once.
#include "moe.h"
#include "ptx.cuh"

namespace mlpk {

namespace {

constexpr int TOK_THREADS = 128;
constexpr int TOK_COLS = 8 * TOK_THREADS;  // columns a block covers in one step

template <bool W_BF16>
__device__ __forceinline__ float ld_weight(const void* w, size_t i) {
  if constexpr (W_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
  else return static_cast<const float*>(w)[i];
}

// Rows of the sorted layout that hold no slot (padding, and past the end)
// become zero: warp `group` looks at `per` rows and writes those that src
// marks.  (They come in runs, the rows past the end in one: with few rows a
// warp there are enough warps to write a run at HBM's rate.)
__device__ __forceinline__ void zero_empty_rows(const int* src, long long rows, long long group,
                                                int per, __nv_bfloat16* out, int H) {
  const int lane = threadIdx.x & 31;
  const long long r0 = group * per, r = r0 + lane;
  unsigned empty = __ballot_sync(0xffffffffu, lane < per && r < rows && src[r < rows ? r : 0] < 0);
  while (empty) {
    const int i = __ffs(empty) - 1;
    empty &= empty - 1;
    __nv_bfloat16* o = out + static_cast<size_t>(r0 + i) * H;
    for (int c = 8 * lane; c < H; c += 256) st_global_v4(o + c, make_uint4(0, 0, 0, 0));
  }
}

// Blocks [0, T segs): one column segment of one token each; the blocks after
// them clear the empty rows (TOK_THREADS / 32 groups of `per` rows a block).
__global__ void __launch_bounds__(TOK_THREADS)
    k_moe_dispatch(const __nv_bfloat16* __restrict__ x, const int* __restrict__ pos,
                   const int* __restrict__ src, __nv_bfloat16* __restrict__ xs, long long rows,
                   int top_k, int H, int segs, long long token_blocks, int per) {
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x >= token_blocks) {
    const long long group = (blockIdx.x - token_blocks) * (TOK_THREADS / 32) + (threadIdx.x >> 5);
    zero_empty_rows(src, rows, group, per, xs, H);
    return;
  }
  const int t = blockIdx.x / segs, c = (blockIdx.x % segs) * TOK_COLS + 8 * threadIdx.x;
  if (c >= H) return;
  const uint4 v = ld_global_v4(x + static_cast<size_t>(t) * H + c);
  const int* p = pos + static_cast<size_t>(t) * top_k;
  for (int j = 0; j < top_k; ++j) {
    const int r = p[j];
    if (r >= 0) st_global_v4(xs + static_cast<size_t>(r) * H + c, v);
  }
}

__device__ __forceinline__ void fma8(float (&a)[8], float w, const uint4& v) {
  const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_bf16x2(q[i]);
    a[2 * i] = fmaf(w, f.x, a[2 * i]);
    a[2 * i + 1] = fmaf(w, f.y, a[2 * i + 1]);
  }
}

template <bool HAS_W, bool W_BF16>
__global__ void __launch_bounds__(TOK_THREADS)
    k_moe_combine(const __nv_bfloat16* __restrict__ y, const int* __restrict__ pos,
                  const void* __restrict__ weights, const __nv_bfloat16* residual,
                  __nv_bfloat16* out, int top_k, int H, int segs) {
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x / segs, c = (blockIdx.x % segs) * TOK_COLS + 8 * threadIdx.x;
  if (c >= H) return;
  const size_t s0 = static_cast<size_t>(t) * top_k, o = static_cast<size_t>(t) * H + c;
  float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (residual) fma8(a, 1.f, ld_global_v4(residual + o));
  // four slots' rows in flight at a time
  for (int j0 = 0; j0 < top_k; j0 += 4) {
    uint4 v[4];
    float w[4];
    int r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = j0 + j < top_k ? pos[s0 + j0 + j] : -1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = 1.f;
      if (r[j] >= 0) {
        v[j] = ld_global_v4(y + static_cast<size_t>(r[j]) * H + c);
        if constexpr (HAS_W) w[j] = ld_weight<W_BF16>(weights, s0 + j0 + j);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (r[j] >= 0) fma8(a, w[j], v[j]);
  }
  st_global_v4(out + o, make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                   pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7])));
}

constexpr int BWD_SLOTS = 4;  // slots of a token in one walk over its columns

// One block per token (and the blocks that clear dy's empty rows): the
// token's gradient row against the rows of up to BWD_SLOTS slots at a time.
template <bool W_BF16>
__global__ void __launch_bounds__(TOK_THREADS)
    k_moe_combine_bwd(const __nv_bfloat16* __restrict__ dout, const __nv_bfloat16* __restrict__ y,
                      const int* __restrict__ pos, const int* __restrict__ src,
                      const void* __restrict__ weights, __nv_bfloat16* __restrict__ dy,
                      void* __restrict__ dweights, long long rows, int T, int top_k, int H,
                      int per) {
  __shared__ float part[TOK_THREADS / 32][BWD_SLOTS];
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x >= T) {
    const long long group = (blockIdx.x - T) * (TOK_THREADS / 32) + (threadIdx.x >> 5);
    zero_empty_rows(src, rows, group, per, dy, H);
    return;
  }
  const size_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const __nv_bfloat16* d = dout + t * H;
  for (int j0 = 0; j0 < top_k; j0 += BWD_SLOTS) {
    int r[BWD_SLOTS];
    float w[BWD_SLOTS], acc[BWD_SLOTS];
#pragma unroll
    for (int j = 0; j < BWD_SLOTS; ++j) {
      const size_t s = t * top_k + j0 + j;
      r[j] = j0 + j < top_k ? pos[s] : -1;
      w[j] = dy != nullptr && r[j] >= 0 ? ld_weight<W_BF16>(weights, s) : 0.f;
      acc[j] = 0.f;
    }
    for (int c = 8 * threadIdx.x; c < H; c += TOK_COLS) {
      const uint4 dv = ld_global_v4(d + c);
      const uint32_t dq[4] = {dv.x, dv.y, dv.z, dv.w};
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 u = unpack_bf16x2(dq[i]);
        f[2 * i] = u.x;
        f[2 * i + 1] = u.y;
      }
      uint4 v[BWD_SLOTS];
      if (dweights) {
#pragma unroll
        for (int j = 0; j < BWD_SLOTS; ++j)
          if (r[j] >= 0) v[j] = ld_global_v4(y + static_cast<size_t>(r[j]) * H + c);
      }
#pragma unroll
      for (int j = 0; j < BWD_SLOTS; ++j) {
        if (r[j] < 0) continue;
        if (dweights) {
          const uint32_t q[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 u = unpack_bf16x2(q[i]);
            acc[j] = fmaf(f[2 * i], u.x, acc[j]);
            acc[j] = fmaf(f[2 * i + 1], u.y, acc[j]);
          }
        }
        if (dy)
          st_global_v4(dy + static_cast<size_t>(r[j]) * H + c,
                       make_uint4(pack_bf16x2(w[j] * f[0], w[j] * f[1]),
                                  pack_bf16x2(w[j] * f[2], w[j] * f[3]),
                                  pack_bf16x2(w[j] * f[4], w[j] * f[5]),
                                  pack_bf16x2(w[j] * f[6], w[j] * f[7])));
      }
    }
    if (!dweights) continue;
#pragma unroll
    for (int j = 0; j < BWD_SLOTS; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
      if (lane == 0) part[warp][j] = acc[j];
    }
    __syncthreads();
    if (threadIdx.x < BWD_SLOTS && j0 + threadIdx.x < top_k) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < TOK_THREADS / 32; ++k) sum += part[k][threadIdx.x];
      const size_t s = t * top_k + j0 + threadIdx.x;
      if constexpr (W_BF16) static_cast<__nv_bfloat16*>(dweights)[s] = __float2bfloat16_rn(sum);
      else static_cast<float*>(dweights)[s] = sum;
    }
    __syncthreads();
  }
}

template <class... Args, class... Given>
cudaError_t launch_tok(void (*kern)(Args...), long long blocks, cudaStream_t stream, bool pdl,
                       Given... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(TOK_THREADS, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Args>(args)...);
}

using bf = __nv_bfloat16;

// Rows a warp looks at for empty ones: one while that leaves few warps (up to
// about 64 an SM), at most four.
int zero_rows(const MoePlan& L) { return L.rows <= 10240 ? 1 : L.rows <= 20480 ? 2 : 4; }
long long zero_blocks(const MoePlan& L) {
  const long long groups = (L.rows + zero_rows(L) - 1) / zero_rows(L);
  return (groups + TOK_THREADS / 32 - 1) / (TOK_THREADS / 32);
}

}  // namespace

cudaError_t launch_moe_dispatch(const void* x, const int* plan, const MoePlan& L, int T, int top_k,
                                int H, void* xs, cudaStream_t stream, bool pdl) {
  const int segs = (H + TOK_COLS - 1) / TOK_COLS;
  const long long tokens = static_cast<long long>(T) * segs;
  return launch_tok(k_moe_dispatch, tokens + zero_blocks(L), stream, pdl,
                    static_cast<const bf*>(x), plan + L.pos, plan + L.src, static_cast<bf*>(xs),
                    L.rows, top_k, H, segs, tokens, zero_rows(L));
}

cudaError_t launch_moe_combine(const void* y, const int* plan, const MoePlan& L, int T, int top_k,
                               int H, const void* weights, bool w_bf16, const void* residual,
                               void* out, cudaStream_t stream, bool pdl) {
  const int segs = (H + TOK_COLS - 1) / TOK_COLS;
  auto kern = weights == nullptr ? k_moe_combine<false, false>
              : w_bf16           ? k_moe_combine<true, true>
                                 : k_moe_combine<true, false>;
  return launch_tok(kern, static_cast<long long>(T) * segs, stream, pdl, static_cast<const bf*>(y),
                    plan + L.pos, weights, static_cast<const bf*>(residual), static_cast<bf*>(out),
                    top_k, H, segs);
}

cudaError_t launch_moe_combine_bwd(const void* dout, const void* y, const int* plan,
                                   const MoePlan& L, int T, int top_k, int H, const void* weights,
                                   bool w_bf16, void* dy, void* dweights, cudaStream_t stream,
                                   bool pdl) {
  auto kern = w_bf16 ? k_moe_combine_bwd<true> : k_moe_combine_bwd<false>;
  return launch_tok(kern, T + (dy ? zero_blocks(L) : 0), stream, pdl, static_cast<const bf*>(dout),
                    static_cast<const bf*>(y), plan + L.pos, plan + L.src, weights,
                    static_cast<bf*>(dy), dweights, L.rows, T, top_k, H,
                    zero_rows(L));
}

}  // namespace mlpk
