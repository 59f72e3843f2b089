// Token rows to their places in the sorted layout and back:
//   k_moe_dispatch     xs[pos[t, j]] = x[t], zeros in the other rows
//   k_moe_combine      out[t] = residual[t] + sum_j w[t, j] y[pos[t, j]]
//                      (without weights: the gradient of the dispatch)
//   k_moe_combine_bwd  dy[pos[t, j]] = w[t, j] dout[t] (zeros in the other
//                      rows), dw[t, j] = sum_h dout[t, h] y[pos[t, j], h]
// All are bound by HBM: every row is read once and written once.  Measured with
// 8192 tokens of 2048 and 8 slots each: dispatch 47 us (6.4 TB/s), combine 46 (6.7),
// its gradients 91 (6.3); with 2 slots 6.1, 6.1 and 5.7 TB/s.  The work
// goes by token, not by sorted row, so that a token's row (or its gradient)
// is read once for all its slots and the sum over its slots needs no atomic
// (the same bits on every run).  Sums are fp32 and rounded once.
#include <type_traits>

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

// Blocks [0, T segs): one segment of CH x TOK_COLS columns of one token each
// (CH pieces of 16 bytes a thread, all loaded before any is stored); the blocks
// after them clear the empty rows (TOK_THREADS / 32 groups of `per` rows a
// block).
template <int CH>
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
  const int t = blockIdx.x / segs, c0 = (blockIdx.x % segs) * (CH * TOK_COLS) + 8 * threadIdx.x;
  uint4 v[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i)
    if (c0 + i * TOK_COLS < H) v[i] = ld_global_v4(x + static_cast<size_t>(t) * H + c0 + i * TOK_COLS);
  const int* p = pos + static_cast<size_t>(t) * top_k;
  for (int j = 0; j < top_k; ++j) {
    const int r = p[j];
    if (r < 0) continue;
    __nv_bfloat16* o = xs + static_cast<size_t>(r) * H + c0;
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (c0 + i * TOK_COLS < H) st_global_v4(o + i * TOK_COLS, v[i]);
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

// Eight values of a row of y, bf16 or fp32.
template <bool Y32>
struct Piece {
  uint4 v;
  __device__ __forceinline__ void load(const void* y, size_t at) {
    v = ld_global_v4(static_cast<const __nv_bfloat16*>(y) + at);
  }
  __device__ __forceinline__ void add(float (&a)[8], float w) const { fma8(a, w, v); }
};
template <>
struct Piece<true> {
  float4 v[2];
  __device__ __forceinline__ void load(const void* y, size_t at) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(y) + at);
    v[0] = p[0];
    v[1] = p[1];
  }
  __device__ __forceinline__ void add(float (&a)[8], float w) const {
    const float f[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = fmaf(w, f[i], a[i]);
  }
};

template <bool HAS_W, bool W_BF16, int CH, bool Y32>
__global__ void __launch_bounds__(TOK_THREADS)
    k_moe_combine(const void* __restrict__ y, const int* __restrict__ pos,
                  const void* __restrict__ weights, const __nv_bfloat16* residual,
                  __nv_bfloat16* out, int top_k, int H, int segs) {
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x / segs, c0 = (blockIdx.x % segs) * (CH * TOK_COLS) + 8 * threadIdx.x;
  const size_t s0 = static_cast<size_t>(t) * top_k, o = static_cast<size_t>(t) * H + c0;
  float a[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) a[i][e] = 0.f;
    if (residual && c0 + i * TOK_COLS < H) fma8(a[i], 1.f, ld_global_v4(residual + o + i * TOK_COLS));
  }
  // SL slots' rows in flight at a time
  constexpr int SL = CH == 1 ? 4 : 2;
  for (int j0 = 0; j0 < top_k; j0 += SL) {
    Piece<Y32> v[SL][CH];
    float w[SL];
    int r[SL];
#pragma unroll
    for (int j = 0; j < SL; ++j) r[j] = j0 + j < top_k ? pos[s0 + j0 + j] : -1;
#pragma unroll
    for (int j = 0; j < SL; ++j) {
      w[j] = 1.f;
      if (r[j] < 0) continue;
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (c0 + i * TOK_COLS < H)
          v[j][i].load(y, static_cast<size_t>(r[j]) * H + c0 + i * TOK_COLS);
      if constexpr (HAS_W) w[j] = ld_weight<W_BF16>(weights, s0 + j0 + j);
    }
#pragma unroll
    for (int j = 0; j < SL; ++j) {
      if (r[j] < 0) continue;
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (c0 + i * TOK_COLS < H) v[j][i].add(a[i], w[j]);
    }
  }
#pragma unroll
  for (int i = 0; i < CH; ++i)
    if (c0 + i * TOK_COLS < H)
      st_global_v4(out + o + i * TOK_COLS,
                   make_uint4(pack_bf16x2(a[i][0], a[i][1]), pack_bf16x2(a[i][2], a[i][3]),
                              pack_bf16x2(a[i][4], a[i][5]), pack_bf16x2(a[i][6], a[i][7])));
}

// y's fp32 rows (in the plan, from the down projection) to the bf16 rows that the
// caller gets; they stay in the plan for the routing weights' gradient.  A block a
// row; a few MB at most (up to MOE_FINE_SLOTS slots).
__global__ void __launch_bounds__(TOK_THREADS)
    k_moe_fine_rows(int* plan, const MoePlan L, int E, int H, __nv_bfloat16* __restrict__ y) {
  pdl_wait();
  pdl_launch_dependents();
  const int r = blockIdx.x;
  if (r == 0 && threadIdx.x == 0) plan[L.fine_flag] = 1;
  if (r >= plan[L.offsets + E]) return;
  const float* f = reinterpret_cast<const float*>(plan + L.fine) + static_cast<size_t>(r) * H;
  for (int c = 8 * threadIdx.x; c < H; c += TOK_COLS) {
    const float4 a = *reinterpret_cast<const float4*>(f + c);
    const float4 b = *reinterpret_cast<const float4*>(f + c + 4);
    st_global_v4(y + static_cast<size_t>(r) * H + c,
                 make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y),
                            pack_bf16x2(b.z, b.w)));
  }
}

constexpr int BWD_SLOTS = 4;   // slots of a token in one walk over its columns
constexpr int BWD_PIECES = 2;  // 16-byte pieces of each row a thread has in flight

// TPT threads per token (and the blocks that clear dy's empty rows): the token's
// gradient row against the rows of up to BWD_SLOTS slots at a time.  A warp per
// token needs no block-wide sum; a block per token serves few tokens.
// FINE: dweights is a sum of random signs, which cancels, and over a handful of
// slots y's rounding to bf16 does not average out of it (a median of 0.0028 of
// dweights' norm, 0.0016 of it the result's own rounding, but in 14 % of the steps of
// up to eight slots over 0.005 and at worst 0.08).  The plan then has y in fp32
// (fine, once *have is set): an fp32 value is taken where it rounds to the y given, so
// that the sum is of that y whatever the plan holds.
template <bool W_BF16, int TPT, bool FINE>
__global__ void __launch_bounds__(TOK_THREADS)
    k_moe_combine_bwd(const __nv_bfloat16* __restrict__ dout, const __nv_bfloat16* __restrict__ y,
                      const int* __restrict__ pos, const int* __restrict__ src,
                      const void* __restrict__ weights, __nv_bfloat16* __restrict__ dy,
                      void* __restrict__ dweights, const float* __restrict__ fine,
                      const int* have, long long rows, int T, int top_k, int H, int per,
                      int token_blocks) {
  __shared__ float part[TOK_THREADS / 32][BWD_SLOTS];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x >= token_blocks) {
    const long long group = (blockIdx.x - token_blocks) * (TOK_THREADS / 32) + warp;
    zero_empty_rows(src, rows, group, per, dy, H);
    return;
  }
  constexpr int STEP = 8 * TPT;  // columns of one piece of all the token's threads
  const int tid = threadIdx.x % TPT;
  const size_t t = static_cast<size_t>(blockIdx.x) * (TOK_THREADS / TPT) + threadIdx.x / TPT;
  if (t >= T) return;  // warp-uniform (TPT = 32) or never
  const __nv_bfloat16* d = dout + t * H;
  const bool use_fine = FINE && *have != 0;
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
    for (int c0 = 8 * tid; c0 < H; c0 += BWD_PIECES * STEP) {
      uint4 dv[BWD_PIECES], v[BWD_PIECES][BWD_SLOTS];
#pragma unroll
      for (int i = 0; i < BWD_PIECES; ++i) {
        const int c = c0 + i * STEP;
        if (c >= H) continue;
        dv[i] = ld_global_v4(d + c);
        if (dweights) {
#pragma unroll
          for (int j = 0; j < BWD_SLOTS; ++j)
            if (r[j] >= 0) v[i][j] = ld_global_v4(y + static_cast<size_t>(r[j]) * H + c);
        }
      }
#pragma unroll
      for (int i = 0; i < BWD_PIECES; ++i) {
        const int c = c0 + i * STEP;
        if (c >= H) continue;
        const uint32_t dq[4] = {dv[i].x, dv[i].y, dv[i].z, dv[i].w};
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 u = unpack_bf16x2(dq[k]);
          f[2 * k] = u.x;
          f[2 * k + 1] = u.y;
        }
#pragma unroll
        for (int j = 0; j < BWD_SLOTS; ++j) {
          if (r[j] < 0) continue;
          if (dweights) {
            const uint32_t q[4] = {v[i][j].x, v[i][j].y, v[i][j].z, v[i][j].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float2 u = unpack_bf16x2(q[k]);
              if constexpr (FINE) {
                if (use_fine) {
                  const float2 z = *reinterpret_cast<const float2*>(
                      fine + static_cast<size_t>(r[j]) * H + c + 2 * k);
                  const uint32_t off = pack_bf16x2(z.x, z.y) ^ q[k];
                  if ((off & 0xffffu) == 0) u.x = z.x;
                  if ((off >> 16) == 0) u.y = z.y;
                }
              }
              acc[j] = fmaf(f[2 * k], u.x, acc[j]);
              acc[j] = fmaf(f[2 * k + 1], u.y, acc[j]);
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
    }
    if (!dweights) continue;
#pragma unroll
    for (int j = 0; j < BWD_SLOTS; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
      if (TPT > 32 && lane == 0) part[warp][j] = acc[j];
    }
    if (TPT > 32) __syncthreads();
    if (tid < BWD_SLOTS && j0 + tid < top_k) {
      float sum = 0.f;
      if constexpr (TPT > 32) {
#pragma unroll
        for (int k = 0; k < TOK_THREADS / 32; ++k) sum += part[k][tid];
      } else {
#pragma unroll
        for (int j = 0; j < BWD_SLOTS; ++j)
          if (tid == j) sum = acc[j];
      }
      const size_t s = t * top_k + j0 + tid;
      if constexpr (W_BF16) static_cast<__nv_bfloat16*>(dweights)[s] = __float2bfloat16_rn(sum);
      else static_cast<float*>(dweights)[s] = sum;
    }
    if (TPT > 32) __syncthreads();
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

// 16-byte pieces of a row that a thread holds: with many slots a token their
// rows are in flight together; with few, more pieces of each row are, once
// there are enough blocks for all SMs without.
int pieces(int T, int top_k, int H) {
  const long long blocks = static_cast<long long>(T) * ((H + TOK_COLS - 1) / TOK_COLS);
  if (blocks < 16 * 152 || H <= TOK_COLS) return 1;
  return top_k >= 4 || H <= 2 * TOK_COLS ? 2 : 4;
}

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
  const int ch = pieces(T, top_k, H), segs = (H + ch * TOK_COLS - 1) / (ch * TOK_COLS);
  const long long tokens = static_cast<long long>(T) * segs;
  return launch_tok(ch == 1 ? k_moe_dispatch<1> : ch == 2 ? k_moe_dispatch<2> : k_moe_dispatch<4>,
                    tokens + zero_blocks(L), stream, pdl,
                    static_cast<const bf*>(x), plan + L.pos, plan + L.src, static_cast<bf*>(xs),
                    L.rows, top_k, H, segs, tokens, zero_rows(L));
}

cudaError_t launch_moe_combine(const void* y, bool y32, const int* plan, const MoePlan& L, int T,
                               int top_k, int H, const void* weights, bool w_bf16,
                               const void* residual, void* out, cudaStream_t stream, bool pdl) {
  const int ch = pieces(T, top_k, H), segs = (H + ch * TOK_COLS - 1) / (ch * TOK_COLS);
  auto pick = [&](auto c) {
    constexpr int CH = decltype(c)::value;
    if (y32) return w_bf16 ? k_moe_combine<true, true, CH, true> : k_moe_combine<true, false, CH, true>;
    return weights == nullptr ? k_moe_combine<false, false, CH, false>
           : w_bf16           ? k_moe_combine<true, true, CH, false>
                              : k_moe_combine<true, false, CH, false>;
  };
  auto kern = ch == 1   ? pick(std::integral_constant<int, 1>{})
              : ch == 2 ? pick(std::integral_constant<int, 2>{})
                        : pick(std::integral_constant<int, 4>{});
  if (y32 && weights == nullptr) return cudaErrorInvalidValue;
  return launch_tok(kern, static_cast<long long>(T) * segs, stream, pdl, y, plan + L.pos, weights,
                    static_cast<const bf*>(residual), static_cast<bf*>(out), top_k, H, segs);
}

cudaError_t launch_moe_combine_bwd(const void* dout, const void* y, const int* plan,
                                   const MoePlan& L, int T, int top_k, int H, const void* weights,
                                   bool w_bf16, void* dy, void* dweights, cudaStream_t stream,
                                   bool pdl) {
  // a warp per token once that gives every SM eight of them
  const bool warps = T >= 8 * 152;
  const bool fine = dweights && L.fine >= 0;  // (then few tokens)
  auto pick = [&](auto w) {
    constexpr bool W = decltype(w)::value;
    return fine    ? k_moe_combine_bwd<W, TOK_THREADS, true>
           : warps ? k_moe_combine_bwd<W, 32, false>
                   : k_moe_combine_bwd<W, TOK_THREADS, false>;
  };
  auto kern = w_bf16 ? pick(std::true_type{}) : pick(std::false_type{});
  const int tokens = warps ? (T + TOK_THREADS / 32 - 1) / (TOK_THREADS / 32) : T;
  return launch_tok(kern, tokens + (dy ? zero_blocks(L) : 0), stream, pdl,
                    static_cast<const bf*>(dout), static_cast<const bf*>(y), plan + L.pos,
                    plan + L.src, weights, static_cast<bf*>(dy), dweights,
                    fine ? reinterpret_cast<const float*>(plan + L.fine) : nullptr,
                    fine ? plan + L.fine_flag : nullptr, L.rows, T, top_k, H, zero_rows(L), tokens);
}

cudaError_t launch_moe_fine_rows(int* plan, const MoePlan& L, int E, int H, void* y,
                                 cudaStream_t stream, bool pdl) {
  return launch_tok(k_moe_fine_rows, L.rows, stream, pdl, plan, L, E, H, static_cast<bf*>(y));
}

}  // namespace mlpk
