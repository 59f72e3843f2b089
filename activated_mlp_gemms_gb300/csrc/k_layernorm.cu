// The layer norm with the residual sum in front of it (mlp_norm.h), forward and backward.
//
// A row belongs to G threads, each with NP pieces of 16 bytes of it, so that it is read once:
// the mean first, then the squares of what is left of it (no cancellation), then the outputs.
// HBM's bandwidth bounds both passes, and what reaches it is bytes in flight: a block walks over
// rows and copies the next ones' values to shared memory (cp.async) while it works on one.  A
// thread copies exactly what it will read, so that the copies need no barrier.  The backward's
// threads hold their columns' sums for the weight's and the bias's gradients in registers from
// row to row; a block leaves one partial sum a column, and a second kernel adds the blocks up in
// their order.
// Measured (us; TB/s of what the pass reads and writes), a launch by itself, when half of what it
// wrote is still in L2: 8192 x 4096 bf16 with the residual sum 40.6 (6.6), its backward with dh and
// the weight's and bias's gradients 49 (5.5) and their sums 3 (9 alone); 4097 x 4872 fp32 34 (4.7:
// two reductions a row, in one block an SM) and 44 (5.4).  Back to back: 8192 x 4096 48 (5.6) and 53
// with the sums; 4097 x 4872 33 and 48; 16384 x 2048 fp32 46 (5.8) and 66 (6.1); 20000 x 768 bf16
// 16 (3.9) and 38, 16384 x 2560 bf16 32 (5.3) and 79.
#include <cuda_bf16.h>

#include <type_traits>

#include "gemm_params.h"
#include "ptx.cuh"
#include "step.h"

namespace mlpk {

namespace {

// A piece of a row: 16 bytes, and as pairs of fp32 for the two-wide instructions.
template <typename T>
struct Piece {
  static constexpr int C = 16 / sizeof(T);  // its columns
  uint4 a;
  __device__ __forceinline__ void store(T* p) const { st_global_v4(p, a); }
  __device__ __forceinline__ void get(uint64_t (&f)[C / 2]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    if constexpr (C == 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = unpack_bf16x2(w[i]);
        f[i] = f2_pack(v.x, v.y);
      }
    } else {
      f[0] = f2_pack(__uint_as_float(w[0]), __uint_as_float(w[1]));
      f[1] = f2_pack(__uint_as_float(w[2]), __uint_as_float(w[3]));
    }
  }
  __device__ __forceinline__ void set(const uint64_t (&f)[C / 2]) {
    uint32_t w[4];
    if constexpr (C == 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = f2_unpack(f[i]);
        w[i] = pack_bf16x2(v.x, v.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 v = f2_unpack(f[i]);
        w[2 * i] = __float_as_uint(v.x);
        w[2 * i + 1] = __float_as_uint(v.y);
      }
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
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

// A thread's pieces of the next rows in shared memory: some rows of ARRAYS arrays of NP pieces,
// in planes of 16 bytes a thread.
template <typename T, int NP, int ARRAYS>
struct Ahead {
  uint32_t mine;   // this thread's first plane
  uint32_t plane;  // bytes of a plane
  __device__ __forceinline__ uint32_t at(int stage, int array, int i) const {
    return mine + plane * static_cast<uint32_t>((stage * ARRAYS + array) * NP + i);
  }
  __device__ __forceinline__ void copy(int stage, int array, int i, const T* src) const {
    cp_async16(at(stage, array, i), src);
  }
  __device__ __forceinline__ void get(int stage, int array, int i,
                                      uint64_t (&f)[Piece<T>::C / 2]) const {
    Piece<T> q;
    q.a = ld_shared_v4(at(stage, array, i));
    q.get(f);
  }
};

// 2 N of the weight's or bias's values (null: `none`).
template <int N>
__device__ __forceinline__ void load_param(const void* p, bool bf16, int at, float none,
                                           uint64_t (&f)[N]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = f2_both(none);
  } else if (bf16) {
    const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(p) + at;
    uint32_t w[N];
    if constexpr (N == 4) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(from));
      w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(from));
      w[0] = q.x, w[1] = q.y;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 v = unpack_bf16x2(w[i]);
      f[i] = f2_pack(v.x, v.y);
    }
  } else {
    const float4* w = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float4 v = __ldg(w + i);
      f[2 * i] = f2_pack(v.x, v.y);
      f[2 * i + 1] = f2_pack(v.z, v.w);
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of N values over the row's threads (a warp's, or the block's), in every one of them.
// `turn` alternates between calls, so that one barrier a call is enough.
template <bool WARP, int N>
struct RowSum {
  float (*s)[N][32];  // [2]: a warp's sums each
  int warps;          // the block's; groups of 8, 16 or 32 lanes add them up
  int turn = 0;
  __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    if constexpr (!WARP) {
      const int lane = threadIdx.x % 32, group = warps > 16 ? 32 : warps > 8 ? 16 : 8;
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[turn][i][threadIdx.x / 32] = v[i];
      }
      __syncthreads();
      const int from = lane & (group - 1);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = from < warps ? s[turn][i][from] : 0.f;
      if (group == 32) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
      }
      if (group >= 16) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 8);
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
      }
      turn ^= 1;
    }
  }
};

// How a row is laid out.  Up to 16 columns a lane it is a warp's, and a block of 256 threads has
// eight rows at a time; a wider one is a block's, of just the warps that it needs: NP pieces a
// thread, so that a thread holds 8, 16 or (the widest) 32 columns.
template <typename T, bool WARP, int NP>
struct Layout {
  static constexpr int COLUMNS = NP * Piece<T>::C;  // a thread
  // (85 registers a thread of 768 are enough for 8 columns)
  static constexpr int THREADS = WARP || NP == 1 ? 256 : NP == 2 && COLUMNS == 8 ? 768 : 512;
  // rows under way: three, fewer where three arrays of the widest would not fit (216 KB)
  static constexpr int DEPTH = THREADS * NP <= 1536 ? 3 : THREADS * NP <= 2048 ? 2 : 1;
  static constexpr bool KEEP = COLUMNS <= 16;  // weights stay in registers
};
constexpr int NORM_SMEM = 216 * 1024;

template <typename T, bool WARP, int NP, bool RESIDUAL>
__global__ void __launch_bounds__(Layout<T, WARP, NP>::THREADS,
                                  Layout<T, WARP, NP>::THREADS == 256 ? 3 : 1)
    k_layernorm_fwd(const NormArgs a, const T* x, const T* residual, const void* __restrict__ weight,
                    const void* __restrict__ bias, T* y, T* h, float* __restrict__ mean,
                    float* __restrict__ rstd) {
  using Lay = Layout<T, WARP, NP>;
  constexpr int D = Lay::DEPTH, C = Piece<T>::C, N2 = C / 2;  // columns, pairs of a piece
  constexpr bool KEEP = Lay::KEEP;
  extern __shared__ uint4 norm_smem[];
  __shared__ float sums_s[2][1][32];
  RowSum<WARP, 1> sum{sums_s, static_cast<int>(blockDim.x) / 32};
  const int G = WARP ? 32 : static_cast<int>(blockDim.x);  // threads of a row
  constexpr int AT_ONCE = WARP ? 8 : 1;                    // rows of a block at a time
  const Ahead<T, NP, RESIDUAL ? 2 : 1> ahead{smem_u32(norm_smem) + threadIdx.x * 16,
                                             blockDim.x * 16};
  const int first = threadIdx.x % G * C;  // this thread's first column; its next piece G C on
  bool has[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) has[i] = first + i * G * C < a.H;
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
      for (int i = 0; i < NP; ++i)
        if (has[i]) {
          ahead.copy(stage, 0, i, next_x + i * G * C);
          if constexpr (RESIDUAL) ahead.copy(stage, 1, i, next_r + i * G * C);
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
  uint64_t kept_w[KEEP ? NP : 1][N2], kept_b[KEEP ? NP : 1][N2];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (has[i]) {
        load_param(weight, a.w_bf16, first + i * G * C, 1.f, kept_w[i]);
        load_param(bias, a.w_bf16, first + i * G * C, 0.f, kept_b[i]);
      }
  }
  const float inv = 1.f / static_cast<float>(a.H);
  size_t at = static_cast<size_t>(row0) * a.H + first;
  int stage = 0, row = row0;
  for (; left > 0; --left, row += step, at += static_cast<size_t>(step) * a.H) {
    cp_async_wait<D>();
    uint64_t v[NP][N2];
    uint64_t s = 0;  // two zeros
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (has[i]) {
        ahead.get(stage, 0, i, v[i]);
        if constexpr (RESIDUAL) {
          uint64_t r[N2];
          ahead.get(stage, 1, i, r);
#pragma unroll
          for (int j = 0; j < N2; ++j) v[i][j] = f2_add(v[i][j], r[j]);
        }
        if (h) {
          Piece<T> q;
          q.set(v[i]);
          q.store(h + at + i * G * C);
        }
        if constexpr (RESIDUAL) {  // what is normed is the sum as it is stored
          Piece<T> q;
          q.set(v[i]);
          q.get(v[i]);
        }
#pragma unroll
        for (int j = 0; j < N2; ++j) s = f2_add(s, v[i][j]);
      }
    fetch(stage);
    stage = stage + 1 == D ? 0 : stage + 1;
    float total[1] = {f2_sum(s)};
    sum(total);
    const float mu = total[0] * inv;
    const uint64_t minus = f2_both(-mu);
    s = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (has[i]) {
#pragma unroll
        for (int j = 0; j < N2; ++j) {
          v[i][j] = f2_add(v[i][j], minus);
          s = f2_fma(v[i][j], v[i][j], s);
        }
      }
    total[0] = f2_sum(s);
    sum(total);
    const float rs = 1.f / sqrtf(total[0] * inv + a.eps);
    if (first == 0) {
      if (mean) mean[row] = mu;
      if (rstd) rstd[row] = rs;
    }
    const uint64_t rs2 = f2_both(rs);
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (has[i]) {
        if constexpr (KEEP) {
#pragma unroll
          for (int j = 0; j < N2; ++j)
            v[i][j] = f2_fma(f2_mul(v[i][j], rs2), kept_w[i][j], kept_b[i][j]);
        } else {
          uint64_t w[N2], b[N2];
          load_param(weight, a.w_bf16, first + i * G * C, 1.f, w);
          load_param(bias, a.w_bf16, first + i * G * C, 0.f, b);
#pragma unroll
          for (int j = 0; j < N2; ++j) v[i][j] = f2_fma(f2_mul(v[i][j], rs2), w[j], b[j]);
        }
        Piece<T> q;
        q.set(v[i]);
        q.store(y + at + i * G * C);
      }
  }
}

template <typename T, bool WARP, int NP, bool SUMS, bool DH>
__global__ void __launch_bounds__(Layout<T, WARP, NP>::THREADS)
    k_layernorm_bwd(const NormArgs a, const T* dy, const T* __restrict__ h,
                    const void* __restrict__ weight, const float* __restrict__ mean,
                    const float* __restrict__ rstd, const T* dh, T* dx, float* __restrict__ part,
                    int* status) {
  using Lay = Layout<T, WARP, NP>;
  constexpr int D = Lay::DEPTH, C = Piece<T>::C, N2 = C / 2;  // columns, pairs of a piece
  constexpr bool KEEP = Lay::KEEP;
  extern __shared__ uint4 norm_smem[];
  __shared__ float sums_s[2][2][32];
  RowSum<WARP, 2> sum{sums_s, static_cast<int>(blockDim.x) / 32};
  const int G = WARP ? 32 : static_cast<int>(blockDim.x);  // threads of a row
  constexpr int AT_ONCE = WARP ? 8 : 1;                    // rows of a block at a time
  const Ahead<T, NP, DH ? 3 : 2> ahead{smem_u32(norm_smem) + threadIdx.x * 16, blockDim.x * 16};
  const int lane = threadIdx.x % G;
  const int first = lane * C;  // this thread's first column; its next piece G C on
  bool has[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) has[i] = first + i * G * C < a.H;
  const int step = gridDim.x * AT_ONCE;
  const int row0 = blockIdx.x * AT_ONCE + threadIdx.x / G;
  pdl_wait();
  pdl_launch_dependents();
  if (SUMS && status && blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  uint64_t dw[SUMS ? NP : 1][N2], db[SUMS ? NP : 1][N2];
  if constexpr (SUMS) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int j = 0; j < N2; ++j) dw[i][j] = db[i][j] = 0;
  }
  size_t at = static_cast<size_t>(row0) * a.H + first;
  const size_t at_step = static_cast<size_t>(step) * a.H;
  int left = row0 < a.M ? (a.M - 1 - row0) / step + 1 : 0;  // rows to work on
  int to_fetch = left;
  size_t next = at;
  auto fetch = [&](int stage) {
    if (to_fetch > 0) {
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (has[i]) {
          ahead.copy(stage, 0, i, dy + next + i * G * C);
          ahead.copy(stage, 1, i, h + next + i * G * C);
          if constexpr (DH) ahead.copy(stage, 2, i, dh + next + i * G * C);
        }
      --to_fetch;
      next += at_step;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(d);
  // the thread's weights, kept from row to row where the registers are there
  uint64_t kept[KEEP ? NP : 1][N2];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (has[i]) load_param(weight, a.w_bf16, first + i * G * C, 1.f, kept[i]);
  }
  auto weights = [&](int i, uint64_t (&w)[N2]) {
    if constexpr (KEEP) {
#pragma unroll
      for (int j = 0; j < N2; ++j) w[j] = kept[i][j];
    } else {
      load_param(weight, a.w_bf16, first + i * G * C, 1.f, w);
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
    for (int i = 0; i < NP; ++i)
      if (has[i]) {
        uint64_t d[N2], x[N2], w[N2];
        ahead.get(stage, 0, i, d);
        ahead.get(stage, 1, i, x);
        weights(i, w);
#pragma unroll
        for (int j = 0; j < N2; ++j) {
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
      float t[2] = {f2_sum(s1), f2_sum(s2)};
      sum(t);
      const uint64_t m1 = f2_both(-t[0] * inv), m2 = f2_both(-t[1] * inv);
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (has[i]) {
          uint64_t d[N2], x[N2], w[N2];
          ahead.get(stage, 0, i, d);
          ahead.get(stage, 1, i, x);
          weights(i, w);
#pragma unroll
          for (int j = 0; j < N2; ++j) {
            const uint64_t xh = f2_mul(f2_add(x[j], minus), rs2);
            d[j] = f2_mul(f2_fma(xh, m2, f2_fma(d[j], w[j], m1)), rs2);
          }
          if constexpr (DH) {
            uint64_t e[N2];
            ahead.get(stage, 2, i, e);
#pragma unroll
            for (int j = 0; j < N2; ++j) d[j] = f2_add(d[j], e[j]);
          }
          Piece<T> q;
          q.set(d);
          q.store(dx + at + i * G * C);
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
      for (int i = 0; i < NP; ++i)
        if (has[i]) {
#pragma unroll
          for (int j = 0; j < N2; ++j) {
            float2* to = reinterpret_cast<float2*>(out + first + i * G * C) + j;
            to[0] = f2_unpack(dw[i][j]);
            to[a.H / 2] = f2_unpack(db[i][j]);
          }
        }
    } else {  // the block's warps in their order
      __shared__ float2 cols_s[2][NP * N2][32];
      for (int w = 0; w < AT_ONCE; ++w) {
        if (threadIdx.x / 32 == w) {
#pragma unroll
          for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < N2; ++j) {
              float2 p = f2_unpack(dw[i][j]), q = f2_unpack(db[i][j]);
              float2 &to_p = cols_s[0][i * N2 + j][lane], &to_q = cols_s[1][i * N2 + j][lane];
              if (w) {
                p.x += to_p.x, p.y += to_p.y;
                q.x += to_q.x, q.y += to_q.y;
              }
              to_p = p;
              to_q = q;
            }
        }
        __syncthreads();
      }
      for (int c = threadIdx.x; c < a.H; c += static_cast<int>(blockDim.x)) {
        const int i = c / (32 * C), l = c / C % 32, j = c % C;  // piece, lane, column of it
        const float2 p = cols_s[0][i * N2 + j / 2][l], q = cols_s[1][i * N2 + j / 2][l];
        out[c] = j % 2 ? p.y : p.x;
        out[a.H + c] = j % 2 ? q.y : q.x;
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

// A row of 129 to 256 pieces has 128 threads of two, so that an SM has five or six rows under way;
// ONE a thread is faster for bf16 with a residual in the forward alone (16384 x 2048 bf16, one /
// two pieces: 45 / 52 us; without a residual 32 / 26, the backward 59 / 50, with dh 63 / 62; 32768
// x 1024 fp32 54 / 49, with a residual 93 / 88, the backward 89 / 68).  Of bf16 also a row of 65 to
// 128 pieces, where a warp's four a lane, 32 columns, would leave no registers for the weights
// (32768 x 1024: a warp a row 44, two warps 26; with a residual 54 / 49, the backward 70 / 51).
template <typename T, bool ONE, class F>
auto by_width(int H, F&& f) {
  const int pieces = H / Piece<T>::C;
#define MLP_NORM_LAYOUT(WARP, NP) return f(Layout<T, WARP, NP>{}, std::integral_constant<bool, WARP>{}, std::integral_constant<int, NP>{})
  if (pieces <= 32) MLP_NORM_LAYOUT(true, 1);
  if (pieces <= 64) MLP_NORM_LAYOUT(true, 2);
  if constexpr (sizeof(T) == 4) {
    if (pieces <= 128) MLP_NORM_LAYOUT(true, 4);
  }
  if constexpr (ONE) {
    if (pieces <= 256) MLP_NORM_LAYOUT(false, 1);
  }
  if (pieces <= 2 * Layout<T, false, 2>::THREADS) MLP_NORM_LAYOUT(false, 2);
  if constexpr (sizeof(T) == 4) {
    if (pieces > 2048) MLP_NORM_LAYOUT(false, 8);
  }
  MLP_NORM_LAYOUT(false, 4);
#undef MLP_NORM_LAYOUT
}
struct Shape {
  int rows, threads, columns;  // of a block; of a thread
  size_t ahead;                // bytes of one array's rows under way in a block
};
template <typename T, bool ONE = false>
Shape shape_of(int H) {
  return by_width<T, ONE>(H, [&](auto lay, auto warp, auto np) {
    constexpr int NP = decltype(np)::value;
    const int threads =
        decltype(warp)::value ? 256 : ((H / Piece<T>::C + NP - 1) / NP + 31) / 32 * 32;
    return Shape{decltype(warp)::value ? 8 : 1, threads, decltype(lay)::COLUMNS,
                 (size_t)decltype(lay)::DEPTH * threads * NP * 16};
  });
}
Shape shape(int H, bool bf16) { return bf16 ? shape_of<__nv_bfloat16>(H) : shape_of<float>(H); }
// Blocks of an SM, by the shared memory that they take (a KB of each is the driver's; 4 KB the
// columns' sums of a warp a row) and by `most` threads: 768 with 8 columns a thread, whose kernels
// use up to 80 registers, 640 with 16, the backward 512 with 32.  With 16 columns of bf16 the
// forward with a residual (101 registers) and the backward with dh and sums (112) fit 512 threads
// alone, and some of the blocks planned come as a second wave: planned / resident an SM 10 / 8
// of 64 threads (the backward of 520 to 1024 columns), 5 / 4 of 128 (2048), both passes 2 / 1 of
// 320 (5120), but 2 / 2 of 256 (4096).  A plan by each kernel's own registers has not been tried.
int sm_blocks(const Shape& p, int arrays, int most) {
  const int fit =
      static_cast<int>(228 * 1024 / (arrays * p.ahead + (p.rows > 1 ? 6 * 1024 : 1536)));
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

template <typename T, bool RESIDUAL>
cudaError_t fwd_of(const NormArgs& a, const void* x, const void* residual, const void* weight,
                   const void* bias, void* y, void* h, float* mean, float* rstd,
                   cudaStream_t stream) {
  constexpr bool ONE = RESIDUAL && sizeof(T) == 2;
  const Shape p = shape_of<T, ONE>(a.H);
  const int arrays = RESIDUAL ? 2 : 1;
  const int all = (a.M - 1) / p.rows + 1;
  const int most = 152 * sm_blocks(p, arrays, p.columns <= 8 ? 768 : 640);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = config(dim3(all < most ? all : most), p.threads, stream, attr);
  cfg.dynamicSmemBytes = arrays * p.ahead;
  return by_width<T, ONE>(a.H, [&](auto, auto warp, auto np) {
    constexpr bool WARP = decltype(warp)::value;
    constexpr int NP = decltype(np)::value;
    using Kernel = KernelOf<k_layernorm_fwd<T, WARP, NP, RESIDUAL>>;
    const cudaError_t e = Kernel::allow_smem(NORM_SMEM);
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, Kernel::kernel, a, static_cast<const T*>(x),
                              static_cast<const T*>(residual), weight, bias, static_cast<T*>(y),
                              static_cast<T*>(h), mean, rstd);
  });
}

template <typename T>
cudaError_t bwd_of(const NormArgs& a, const void* dy, const void* h, const void* weight,
                   const float* mean, const float* rstd, const void* dh, void* dx, float* part,
                   int* status, cudaStream_t stream) {
  const Shape p = shape_of<T>(a.H);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg =
      config(dim3(layernorm_blocks(a.M, a.H, a.bf16)), p.threads, stream, attr);
  cfg.dynamicSmemBytes = (dh ? 3 : 2) * p.ahead;
  return by_width<T, false>(a.H, [&](auto, auto warp, auto np) {
    constexpr bool WARP = decltype(warp)::value;
    constexpr int NP = decltype(np)::value;
    auto go = [&](auto kern) {
      const cudaError_t e = kern.allow_smem(NORM_SMEM);
      if (e != cudaSuccess) return e;
      return cudaLaunchKernelEx(&cfg, kern.kernel, a, static_cast<const T*>(dy),
                                static_cast<const T*>(h), weight, mean, rstd,
                                static_cast<const T*>(dh), static_cast<T*>(dx), part, status);
    };
    if (part) return dh ? go(KernelOf<k_layernorm_bwd<T, WARP, NP, true, true>>{})
                        : go(KernelOf<k_layernorm_bwd<T, WARP, NP, true, false>>{});
    return dh ? go(KernelOf<k_layernorm_bwd<T, WARP, NP, false, true>>{})
              : go(KernelOf<k_layernorm_bwd<T, WARP, NP, false, false>>{});
  });
}

}  // namespace

// (a function of the sizes and the type alone: the workspace is, too)
int layernorm_blocks(int M, int H, bool bf16) {
  const Shape p = shape(H, bf16);
  const int all = (M - 1) / p.rows + 1;
  const int most = 152 * sm_blocks(p, 3, p.columns <= 8 ? 768 : p.columns <= 16 ? 640 : 512);
  return all < most ? all : most;
}

cudaError_t launch_layernorm_fwd(const NormArgs& a, const void* x, const void* residual,
                                 const void* weight, const void* bias, void* y, void* h,
                                 float* mean, float* rstd, cudaStream_t stream) {
  auto go = [&](auto type, auto has) {
    return fwd_of<decltype(type), decltype(has)::value>(a, x, residual, weight, bias, y, h, mean,
                                                        rstd, stream);
  };
  if (residual) return a.bf16 ? go(__nv_bfloat16{}, std::true_type{}) : go(0.f, std::true_type{});
  return a.bf16 ? go(__nv_bfloat16{}, std::false_type{}) : go(0.f, std::false_type{});
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
