// The layer norm with the residual sum in front of it (mlp_norm.h), forward and backward.
//
// A row belongs to G threads, each with NV vectors of 8 of its values, so that it is read once:
// the mean first, then the squares of what is left of it (no cancellation), then the outputs.
// HBM's bandwidth bounds both passes, and what reaches it is bytes in flight: a block walks over
// rows and copies the next ones' values to shared memory (cp.async) while it works on one.  A
// thread copies exactly what it will read, so that the copies need no barrier.  The backward's
// threads hold their columns' sums for the weight's and the bias's gradients in registers from
// row to row; a block leaves one partial sum a column, and a second kernel adds the blocks up in
// their order.
#include <cuda_bf16.h>

#include "gemm_params.h"
#include "ptx.cuh"
#include "step.h"

namespace mlpk {

namespace {

// Eight values of a row, 16 bytes (bf16) or 32 (fp32), and as four pairs of fp32 for the
// two-wide instructions.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = ld_global_v4(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { st_global_v4(p, a); }
  __device__ __forceinline__ void get(uint64_t (&f)[4]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack_bf16x2(w[i]);
      f[i] = f2_pack(v.x, v.y);
    }
  }
  __device__ __forceinline__ void set(const uint64_t (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = f2_unpack(f[i]);
      w[i] = pack_bf16x2(v.x, v.y);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec8<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = ld_global_v4(p);
    b = ld_global_v4(p + 4);
  }
  __device__ __forceinline__ void store(float* p) const {
    st_global_v4(p, a);
    st_global_v4(p + 4, b);
  }
  __device__ __forceinline__ void get(uint64_t (&f)[4]) const {
    f[0] = f2_pack(__uint_as_float(a.x), __uint_as_float(a.y));
    f[1] = f2_pack(__uint_as_float(a.z), __uint_as_float(a.w));
    f[2] = f2_pack(__uint_as_float(b.x), __uint_as_float(b.y));
    f[3] = f2_pack(__uint_as_float(b.z), __uint_as_float(b.w));
  }
  __device__ __forceinline__ void set(const uint64_t (&f)[4]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = f2_unpack(f[i]);
      w[2 * i] = __float_as_uint(v.x);
      w[2 * i + 1] = __float_as_uint(v.y);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
  }
};
__device__ __forceinline__ uint64_t f2_both(float v) { return f2_pack(v, v); }
__device__ __forceinline__ float f2_sum(uint64_t v) {
  const float2 f = f2_unpack(v);
  return f.x + f.y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits until all but the newest DEPTH - 1 groups have landed.
template <int DEPTH>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
}

// A thread's vectors of the next rows in shared memory: some rows of ARRAYS arrays of NV
// vectors, in planes of 16 bytes a thread.
template <typename T, int NV, int ARRAYS>
struct Ahead {
  static constexpr int PLANES = sizeof(T) == 2 ? 1 : 2;  // 16-byte parts of a vector
  uint32_t mine;   // this thread's first plane
  uint32_t plane;  // bytes of a plane
  __device__ __forceinline__ uint32_t at(int stage, int array, int i) const {
    return mine + plane * static_cast<uint32_t>(((stage * ARRAYS + array) * NV + i) * PLANES);
  }
  __device__ __forceinline__ void copy(int stage, int array, int i, const T* src) const {
    const uint32_t to = at(stage, array, i);
    cp_async16(to, src);
    if constexpr (PLANES == 2) cp_async16(to + plane, src + 4);
  }
  __device__ __forceinline__ void get(int stage, int array, int i, uint64_t (&f)[4]) const {
    Vec8<T> q;
    q.a = ld_shared_v4(at(stage, array, i));
    if constexpr (PLANES == 2) q.b = ld_shared_v4(at(stage, array, i) + plane);
    q.get(f);
  }
};

// Eight of the weight's or bias's values (null: `none`).
__device__ __forceinline__ void load_param(const void* p, bool bf16, int at, float none,
                                           uint64_t (&f)[4]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2_both(none);
  } else if (bf16) {
    Vec8<__nv_bfloat16> v;
    v.load(static_cast<const __nv_bfloat16*>(p) + at);
    v.get(f);
  } else {
    Vec8<float> v;
    v.load(static_cast<const float*>(p) + at);
    v.get(f);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

constexpr int MAX_THREADS = 512;

// Sums over the row's threads (a warp's, or the block's), in every one of them.  `turn`
// alternates between calls, so that one barrier a call is enough.
template <bool WARP>
struct RowSum {
  float2 (*s)[MAX_THREADS / 32];
  int turn = 0;
  __device__ __forceinline__ float2 operator()(float a, float b) {
    a = warp_sum(a);
    b = warp_sum(b);
    if constexpr (WARP) {
      return make_float2(a, b);
    } else {
      if (threadIdx.x % 32 == 0) s[turn][threadIdx.x / 32] = make_float2(a, b);
      __syncthreads();
      float2 t = make_float2(0.f, 0.f);
      const int warps = blockDim.x / 32;
#pragma unroll 8
      for (int i = 0; i < warps; ++i) {
        const float2 v = s[turn][i];
        t.x += v.x;
        t.y += v.y;
      }
      turn ^= 1;
      return t;
    }
  }
};

// How a row is laid out.  Up to 1024 values it is a warp's, and a block of 256 threads has eight
// rows at a time; wider ones are a block's, of just the warps that they need.
struct Shape {
  int nv, threads, depth;
  bool warp;
};
// Rows under way: three, fewer where three arrays of the widest would not fit (192 KB).
template <typename T, bool WARP, int NV>
constexpr int DEPTH = (WARP ? 256 : NV == 1 ? 256 : 512) * NV * sizeof(T) * 8 <= 16384   ? 3
                      : (WARP ? 256 : NV == 1 ? 256 : 512) * NV * sizeof(T) * 8 <= 32768 ? 2
                                                                                         : 1;

template <typename T, bool WARP, int NV, bool RESIDUAL>
__global__ void __launch_bounds__(WARP || NV == 1 ? 256 : MAX_THREADS, WARP || NV == 1 ? 3 : 1)
    k_layernorm_fwd(const NormArgs a, const T* x, const T* residual, const void* __restrict__ weight,
                    const void* __restrict__ bias, T* y, T* h, float* __restrict__ mean,
                    float* __restrict__ rstd) {
  constexpr int D = DEPTH<T, WARP, NV>;
  extern __shared__ uint4 norm_smem[];
  __shared__ float2 sums_s[2][MAX_THREADS / 32];
  RowSum<WARP> sum{sums_s};
  const int G = WARP ? 32 : static_cast<int>(blockDim.x);  // threads of a row
  constexpr int AT_ONCE = WARP ? 8 : 1;                    // rows of a block at a time
  const Ahead<T, NV, RESIDUAL ? 2 : 1> ahead{smem_u32(norm_smem) + threadIdx.x * 16,
                                             blockDim.x * 16};
  const int first = threadIdx.x % G * 8;  // this thread's first column; the next G * 8 on
  const int step = gridDim.x * AT_ONCE;
  const int row0 = blockIdx.x * AT_ONCE + threadIdx.x / G;
  pdl_wait();
  pdl_launch_dependents();
  const long long x_step = step * a.ldx, r_step = step * a.ldr;
  const T* next_x = x + row0 * a.ldx + first;
  const T* next_r = RESIDUAL ? residual + row0 * a.ldr + first : nullptr;
  int left = row0 < a.M ? (a.M - 1 - row0) / step + 1 : 0;  // rows to work on
  int to_fetch = left;
  auto fetch = [&](int stage) {
    if (to_fetch > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (first + i * G * 8 < a.H) {
          ahead.copy(stage, 0, i, next_x + i * G * 8);
          if constexpr (RESIDUAL) ahead.copy(stage, 1, i, next_r + i * G * 8);
        }
      --to_fetch;
      next_x += x_step;
      if constexpr (RESIDUAL) next_r += r_step;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(d);
  // the thread's weights and biases, kept from row to row where the registers are there
  constexpr bool KEEP = NV <= 2;
  uint64_t kept_w[KEEP ? NV : 1][4], kept_b[KEEP ? NV : 1][4];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (first + i * G * 8 < a.H) {
        load_param(weight, a.w_bf16, first + i * G * 8, 1.f, kept_w[i]);
        load_param(bias, a.w_bf16, first + i * G * 8, 0.f, kept_b[i]);
      }
  }
  const float inv = 1.f / static_cast<float>(a.H);
  size_t at = static_cast<size_t>(row0) * a.H + first;
  int stage = 0, row = row0;
  for (; left > 0; --left, row += step, at += static_cast<size_t>(step) * a.H) {
    cp_async_wait<D>();
    uint64_t v[NV][4];
    uint64_t s = 0;  // two zeros
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (first + i * G * 8 < a.H) {
        ahead.get(stage, 0, i, v[i]);
        if constexpr (RESIDUAL) {
          uint64_t r[4];
          ahead.get(stage, 1, i, r);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = f2_add(v[i][j], r[j]);
        }
        if (h) {
          Vec8<T> q;
          q.set(v[i]);
          q.store(h + at + i * G * 8);
        }
        if constexpr (RESIDUAL) {  // what is normed is the sum as it is stored
          Vec8<T> q;
          q.set(v[i]);
          q.get(v[i]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) s = f2_add(s, v[i][j]);
      }
    fetch(stage);
    stage = stage + 1 == D ? 0 : stage + 1;
    const float mu = sum(f2_sum(s), 0.f).x * inv;
    const uint64_t minus = f2_both(-mu);
    s = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (first + i * G * 8 < a.H) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[i][j] = f2_add(v[i][j], minus);
          s = f2_fma(v[i][j], v[i][j], s);
        }
      }
    const float rs = 1.f / sqrtf(sum(f2_sum(s), 0.f).x * inv + a.eps);
    if (first == 0) {
      if (mean) mean[row] = mu;
      if (rstd) rstd[row] = rs;
    }
    const uint64_t rs2 = f2_both(rs);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (first + i * G * 8 < a.H) {
        if constexpr (KEEP) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[i][j] = f2_fma(f2_mul(v[i][j], rs2), kept_w[i][j], kept_b[i][j]);
        } else {
          uint64_t w[4], b[4];
          load_param(weight, a.w_bf16, first + i * G * 8, 1.f, w);
          load_param(bias, a.w_bf16, first + i * G * 8, 0.f, b);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = f2_fma(f2_mul(v[i][j], rs2), w[j], b[j]);
        }
        Vec8<T> q;
        q.set(v[i]);
        q.store(y + at + i * G * 8);
      }
  }
}

template <typename T, bool WARP, int NV, bool SUMS, bool DH>
__global__ void __launch_bounds__(WARP || NV == 1 ? 256 : MAX_THREADS)
    k_layernorm_bwd(const NormArgs a, const T* dy, const T* __restrict__ h,
                    const void* __restrict__ weight, const float* __restrict__ mean,
                    const float* __restrict__ rstd, const T* dh, T* dx, float* __restrict__ part,
                    int* status) {
  constexpr int D = DEPTH<T, WARP, NV>;
  extern __shared__ uint4 norm_smem[];
  __shared__ float2 sums_s[2][MAX_THREADS / 32];
  RowSum<WARP> sum{sums_s};
  const int G = WARP ? 32 : static_cast<int>(blockDim.x);  // threads of a row
  constexpr int AT_ONCE = WARP ? 8 : 1;                    // rows of a block at a time
  const Ahead<T, NV, DH ? 3 : 2> ahead{smem_u32(norm_smem) + threadIdx.x * 16, blockDim.x * 16};
  const int lane = threadIdx.x % G;
  const int first = lane * 8;  // this thread's first column; the next G * 8 on
  const int step = gridDim.x * AT_ONCE;
  const int row0 = blockIdx.x * AT_ONCE + threadIdx.x / G;
  pdl_wait();
  pdl_launch_dependents();
  if (SUMS && status && blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  uint64_t dw[SUMS ? NV : 1][4], db[SUMS ? NV : 1][4];
  if constexpr (SUMS) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) dw[i][j] = db[i][j] = 0;
  }
  size_t at = static_cast<size_t>(row0) * a.H + first;
  const size_t at_step = static_cast<size_t>(step) * a.H;
  int left = row0 < a.M ? (a.M - 1 - row0) / step + 1 : 0;  // rows to work on
  int to_fetch = left;
  size_t next = at;
  auto fetch = [&](int stage) {
    if (to_fetch > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (first + i * G * 8 < a.H) {
          ahead.copy(stage, 0, i, dy + next + i * G * 8);
          ahead.copy(stage, 1, i, h + next + i * G * 8);
          if constexpr (DH) ahead.copy(stage, 2, i, dh + next + i * G * 8);
        }
      --to_fetch;
      next += at_step;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(d);
  // the thread's weights, kept from row to row where the registers are there
  constexpr bool KEEP = NV <= 2;
  uint64_t kept[KEEP ? NV : 1][4];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (first + i * G * 8 < a.H) load_param(weight, a.w_bf16, first + i * G * 8, 1.f, kept[i]);
  }
  auto weights = [&](int i, uint64_t (&w)[4]) {
    if constexpr (KEEP) {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = kept[i][j];
    } else {
      load_param(weight, a.w_bf16, first + i * G * 8, 1.f, w);
    }
  };
  const float inv = 1.f / static_cast<float>(a.H);
  int stage = 0, row = row0;
  float mu = 0.f, rs = 0.f;
  if (left > 0) mu = mean[row], rs = rstd[row];
  for (; left > 0; --left, at += at_step) {
    if (left > 1) row += step;
    const float next_mu = mean[row], next_rs = rstd[row];
    cp_async_wait<D>();
    const uint64_t minus = f2_both(-mu), rs2 = f2_both(rs);
    uint64_t s1 = 0, s2 = 0;  // two zeros each
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (first + i * G * 8 < a.H) {
        uint64_t d[4], x[4], w[4];
        ahead.get(stage, 0, i, d);
        ahead.get(stage, 1, i, x);
        weights(i, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t xh = f2_mul(f2_add(x[j], minus), rs2), g = f2_mul(d[j], w[j]);
          s1 = f2_add(s1, g);
          s2 = f2_fma(g, xh, s2);
          if constexpr (SUMS) {
            dw[i][j] = f2_fma(d[j], xh, dw[i][j]);
            db[i][j] = f2_add(db[i][j], d[j]);
          }
        }
      }
    if (dx) {
      const float2 t = sum(f2_sum(s1), f2_sum(s2));
      const uint64_t m1 = f2_both(-t.x * inv), m2 = f2_both(-t.y * inv);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (first + i * G * 8 < a.H) {
          uint64_t d[4], x[4], w[4];
          ahead.get(stage, 0, i, d);
          ahead.get(stage, 1, i, x);
          weights(i, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t xh = f2_mul(f2_add(x[j], minus), rs2);
            d[j] = f2_mul(f2_fma(xh, m2, f2_fma(d[j], w[j], m1)), rs2);
          }
          if constexpr (DH) {
            uint64_t e[4];
            ahead.get(stage, 2, i, e);
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] = f2_add(d[j], e[j]);
          }
          Vec8<T> q;
          q.set(d);
          q.store(dx + at + i * G * 8);
        }
    }
    fetch(stage);
    stage = stage + 1 == D ? 0 : stage + 1;
    mu = next_mu;
    rs = next_rs;
  }
  if constexpr (SUMS) {
    float* out = part + static_cast<size_t>(blockIdx.x) * 2 * a.H;
    if constexpr (!WARP) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (first + i * G * 8 < a.H) {
          Vec8<float> q;
          q.set(dw[i]);
          q.store(out + first + i * G * 8);
          q.set(db[i]);
          q.store(out + a.H + first + i * G * 8);
        }
    } else {  // the block's warps in their order
      __shared__ float cols_s[2][32 * NV * 8];
      for (int w = 0; w < AT_ONCE; ++w) {
        if (threadIdx.x / 32 == w) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 p = f2_unpack(dw[i][j]), q = f2_unpack(db[i][j]);
              const int c = (i * 8 + 2 * j) * 32 + lane;
              cols_s[0][c] = w ? cols_s[0][c] + p.x : p.x;
              cols_s[0][c + 32] = w ? cols_s[0][c + 32] + p.y : p.y;
              cols_s[1][c] = w ? cols_s[1][c] + q.x : q.x;
              cols_s[1][c + 32] = w ? cols_s[1][c + 32] + q.y : q.y;
            }
        }
        __syncthreads();
      }
      for (int c = threadIdx.x; c < a.H; c += static_cast<int>(blockDim.x)) {
        const int from = (c / 256 * 8 + c % 8) * 32 + c / 8 % 32;
        out[c] = cols_s[0][from];
        out[a.H + c] = cols_s[1][from];
      }
    }
  }
}

// The blocks' sums of a column: 32 threads a column, then their sums.
constexpr int SUM_ROWS = 32;
__global__ void __launch_bounds__(32 * SUM_ROWS)
    k_layernorm_sums(const int H, const int blocks, const float* __restrict__ part, void* dweight,
                     void* dbias, const bool bf16, const bool accum) {
  __shared__ float s[SUM_ROWS][33];
  const int lane = threadIdx.x % 32, r = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  void* out = blockIdx.y == 0 ? dweight : dbias;
  pdl_wait();
  pdl_launch_dependents();
  if (!out) return;
  float t = 0.f;
  if (c < H) {
    const float* p = part + static_cast<size_t>(blockIdx.y) * H + c;
#pragma unroll 10
    for (int b = r; b < blocks; b += SUM_ROWS) t += p[static_cast<size_t>(b) * 2 * H];
  }
  s[r][lane] = t;
  __syncthreads();
  // (column r of the block's 32, its sums one a lane)
  t = s[lane][r];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const int mine = blockIdx.x * 32 + r;
  if (lane || mine >= H) return;
  if (accum) static_cast<float*>(out)[mine] += t;
  else if (bf16) static_cast<__nv_bfloat16*>(out)[mine] = __float2bfloat16_rn(t);
  else static_cast<float*>(out)[mine] = t;
}

template <class F>
auto by_width(int H, F&& f) {
  const int vecs = H / 8;
#define MLP_NORM_SHAPE(WARP, NV) \
  return f(std::integral_constant<bool, WARP>{}, std::integral_constant<int, NV>{})
  if (vecs <= 32) MLP_NORM_SHAPE(true, 1);
  if (vecs <= 64) MLP_NORM_SHAPE(true, 2);
  if (vecs <= 128) MLP_NORM_SHAPE(true, 4);
  if (vecs <= 256) MLP_NORM_SHAPE(false, 1);
  if (vecs <= 1024) MLP_NORM_SHAPE(false, 2);
  MLP_NORM_SHAPE(false, 4);
#undef MLP_NORM_SHAPE
}
Shape shape(int H, bool bf16) {
  return by_width(H, [&](auto w, auto v) {
    constexpr bool WARP = decltype(w)::value;
    constexpr int NV = decltype(v)::value;
    const int threads = WARP ? 256 : ((H / 8 + NV - 1) / NV + 31) / 32 * 32;
    return Shape{NV, threads,
                 bf16 ? DEPTH<__nv_bfloat16, WARP, NV> : DEPTH<float, WARP, NV>, WARP};
  });
}
// Bytes of the rows under way in a block.
size_t ahead_bytes(const Shape& p, int arrays, bool bf16) {
  return (size_t)arrays * p.depth * p.threads * p.nv * (bf16 ? 16 : 32);
}
int block_rows(const Shape& p) { return p.warp ? 8 : 1; }
// Blocks of an SM, by the shared memory that they take (a KB of each is the driver's, 8 KB the
// columns' sums) and `most` threads, which the registers allow.
int sm_blocks(const Shape& p, int arrays, bool bf16, int most) {
  const int fit = static_cast<int>(228 * 1024 / (ahead_bytes(p, arrays, bf16) +
                                                 (p.warp ? 9 * 1024 : 1280)));
  const int n = fit < most / p.threads ? fit : most / p.threads;
  return n < 1 ? 1 : n;
}

cudaLaunchConfig_t config(dim3 blocks, int threads, cudaStream_t stream,
                          cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = blocks;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

constexpr int NORM_SMEM = 192 * 1024;  // the most that a row's depth takes

template <typename T>
cudaError_t fwd_of(const NormArgs& a, const void* x, const void* residual, const void* weight,
                   const void* bias, void* y, void* h, float* mean, float* rstd,
                   cudaStream_t stream) {
  const Shape p = shape(a.H, a.bf16);
  const int arrays = residual ? 2 : 1;
  const int all = (a.M - 1) / block_rows(p) + 1;
  const int most = 152 * sm_blocks(p, arrays, a.bf16, p.nv == 1 ? 768 : 640);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config(dim3(all < most ? all : most), p.threads, stream, attr);
  cfg.dynamicSmemBytes = ahead_bytes(p, arrays, a.bf16);
  return by_width(a.H, [&](auto w, auto nv) {
    constexpr bool WARP = decltype(w)::value;
    constexpr int NV = decltype(nv)::value;
    auto go = [&](auto kern) {
      const cudaError_t e = kern.allow_smem(NORM_SMEM);
      if (e != cudaSuccess) return e;
      return cudaLaunchKernelEx(&cfg, kern.kernel, a, static_cast<const T*>(x),
                                static_cast<const T*>(residual), weight, bias, static_cast<T*>(y),
                                static_cast<T*>(h), mean, rstd);
    };
    return residual ? go(KernelOf<k_layernorm_fwd<T, WARP, NV, true>>{})
                    : go(KernelOf<k_layernorm_fwd<T, WARP, NV, false>>{});
  });
}

template <typename T>
cudaError_t bwd_of(const NormArgs& a, const void* dy, const void* h, const void* weight,
                   const float* mean, const float* rstd, const void* dh, void* dx, float* part,
                   int* status, cudaStream_t stream) {
  const Shape p = shape(a.H, a.bf16);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg =
      config(dim3(layernorm_blocks(a.M, a.H, a.bf16)), p.threads, stream, attr);
  cfg.dynamicSmemBytes = ahead_bytes(p, dh ? 3 : 2, a.bf16);
  return by_width(a.H, [&](auto w, auto nv) {
    constexpr bool WARP = decltype(w)::value;
    constexpr int NV = decltype(nv)::value;
    auto go = [&](auto kern) {
      const cudaError_t e = kern.allow_smem(NORM_SMEM);
      if (e != cudaSuccess) return e;
      return cudaLaunchKernelEx(&cfg, kern.kernel, a, static_cast<const T*>(dy),
                                static_cast<const T*>(h), weight, mean, rstd,
                                static_cast<const T*>(dh), static_cast<T*>(dx), part, status);
    };
    if (part) return dh ? go(KernelOf<k_layernorm_bwd<T, WARP, NV, true, true>>{})
                        : go(KernelOf<k_layernorm_bwd<T, WARP, NV, true, false>>{});
    return dh ? go(KernelOf<k_layernorm_bwd<T, WARP, NV, false, true>>{})
              : go(KernelOf<k_layernorm_bwd<T, WARP, NV, false, false>>{});
  });
}

}  // namespace

// (a function of the sizes and the type alone: the workspace is, too)
int layernorm_blocks(int M, int H, bool bf16) {
  const Shape p = shape(H, bf16);
  const int all = (M - 1) / block_rows(p) + 1;
  const int most = 152 * sm_blocks(p, 3, bf16, p.warp || p.nv == 4 ? 512 : p.nv == 1 ? 768 : 640);
  return all < most ? all : most;
}

cudaError_t launch_layernorm_fwd(const NormArgs& a, const void* x, const void* residual,
                                 const void* weight, const void* bias, void* y, void* h,
                                 float* mean, float* rstd, cudaStream_t stream) {
  return a.bf16 ? fwd_of<__nv_bfloat16>(a, x, residual, weight, bias, y, h, mean, rstd, stream)
                : fwd_of<float>(a, x, residual, weight, bias, y, h, mean, rstd, stream);
}

cudaError_t launch_layernorm_bwd(const NormArgs& a, const void* dy, const void* h,
                                 const void* weight, const float* mean, const float* rstd,
                                 const void* dh, void* dx, float* part, int* status,
                                 cudaStream_t stream) {
  return a.bf16 ? bwd_of<__nv_bfloat16>(a, dy, h, weight, mean, rstd, dh, dx, part, status, stream)
                : bwd_of<float>(a, dy, h, weight, mean, rstd, dh, dx, part, status, stream);
}

cudaError_t launch_layernorm_sums(int H, int blocks, const float* part, void* dweight, void* dbias,
                                  bool w_bf16, bool accum, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config(dim3((H + 31) / 32, 2), 32 * SUM_ROWS, stream, attr);
  return cudaLaunchKernelEx(&cfg, k_layernorm_sums, H, blocks, part, dweight, dbias, w_bf16, accum);
}

}  // namespace mlpk
