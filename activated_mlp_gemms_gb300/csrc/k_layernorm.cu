// The layer norm with the residual sum in front of it (mlp_norm.h), forward and backward.
//
// A row belongs to G threads, each with NV vectors of 8 of its values in registers, so that
// it is read once: the mean first, then the squares of what is left of it (no cancellation),
// then the outputs.  The backward's blocks walk over rows with the same columns in each
// thread, which holds its columns' sums for the weight's and the bias's gradients in
// registers; a block leaves one partial sum a column, and a second kernel adds the blocks up
// in their order.
#include <cuda_bf16.h>

#include "gemm_params.h"
#include "ptx.cuh"
#include "step.h"

namespace mlpk {

namespace {

// Eight values of a row, 16 bytes (bf16) or 32 (fp32).
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = ld_global_v4(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { st_global_v4(p, a); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack_bf16x2(w[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    a = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
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
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                   __float_as_uint(f[3]));
    b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                   __float_as_uint(f[7]));
  }
};

// Eight of the weight's or bias's values (null: `none`).
__device__ __forceinline__ void load_param(const void* p, bool bf16, int at, float none,
                                           float (&f)[8]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = none;
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

// Sums over the row's G threads (G > 32: all of the block's), in every one of them.
// `turn` alternates between calls, so that one barrier a call is enough.
template <int G>
struct RowSum {
  float2 (*s)[G / 32];
  int turn = 0;
  __device__ __forceinline__ float2 operator()(float a, float b) {
    a = warp_sum(a);
    b = warp_sum(b);
    if constexpr (G == 32) {
      return make_float2(a, b);
    } else {
      if (threadIdx.x % 32 == 0) s[turn][threadIdx.x / 32] = make_float2(a, b);
      __syncthreads();
      float2 t = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < G / 32; ++i) {
        const float2 v = s[turn][i];
        t.x += v.x;
        t.y += v.y;
      }
      turn ^= 1;
      return t;
    }
  }
};

// Rows a block has in hand at a time.
template <int G>
constexpr int AT_ONCE = G == 32 ? 8 : 1;
template <int G>
constexpr int THREADS = G * AT_ONCE<G>;

template <typename T, int G, int NV>
__global__ void __launch_bounds__(THREADS<G>)
    k_layernorm_fwd(const NormArgs a, const T* x, const T* residual, const void* __restrict__ weight,
                    const void* __restrict__ bias, T* y, T* h, float* __restrict__ mean,
                    float* __restrict__ rstd) {
  __shared__ float2 sums_s[2][G / 32];
  RowSum<G> sum{sums_s};
  const int lane = threadIdx.x % G;
  const long long row = static_cast<long long>(blockIdx.x) * AT_ONCE<G> + threadIdx.x / G;
  pdl_wait();
  pdl_launch_dependents();
  if (row >= a.M) return;  // (whole warps; G > 32: whole blocks)
  float v[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * G + lane) * 8;
    if (at < a.H) {
      Vec8<T> q;
      q.load(x + row * a.ldx + at);
      q.get(v[i]);
    }
  }
  if (residual) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = (i * G + lane) * 8;
      if (at < a.H) {
        Vec8<T> q;
        float r[8];
        q.load(residual + row * a.ldr + at);
        q.get(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += r[j];
        q.set(v[i]);  // what is normed is what is stored
        q.get(v[i]);
        if (h) q.store(h + row * a.H + at);
      }
    }
  } else if (h) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = (i * G + lane) * 8;
      if (at < a.H) {
        Vec8<T> q;
        q.set(v[i]);
        q.store(h + row * a.H + at);
      }
    }
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if ((i * G + lane) * 8 < a.H) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[i][j];
    }
  const float mu = sum(s, 0.f).x / static_cast<float>(a.H);
  s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if ((i * G + lane) * 8 < a.H) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] -= mu;
        s += v[i][j] * v[i][j];
      }
    }
  const float rs = 1.f / sqrtf(sum(s, 0.f).x / static_cast<float>(a.H) + a.eps);
  if (lane == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = rs;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * G + lane) * 8;
    if (at < a.H) {
      float w[8], b[8];
      load_param(weight, a.w_bf16, at, 1.f, w);
      load_param(bias, a.w_bf16, at, 0.f, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rs * w[j] + b[j];
      Vec8<T> q;
      q.set(v[i]);
      q.store(y + row * a.H + at);
    }
  }
}

template <typename T, int G, int NV, bool SUMS>
__global__ void __launch_bounds__(THREADS<G>)
    k_layernorm_bwd(const NormArgs a, const T* dy, const T* __restrict__ h,
                    const void* __restrict__ weight, const float* __restrict__ mean,
                    const float* __restrict__ rstd, const T* dh, T* dx, float* __restrict__ part,
                    int* status) {
  __shared__ float2 sums_s[2][G / 32];
  RowSum<G> sum{sums_s};
  const int lane = threadIdx.x % G;
  pdl_wait();
  pdl_launch_dependents();
  if (SUMS && status && blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  float dw[SUMS ? NV : 1][8], db[SUMS ? NV : 1][8];
  if constexpr (SUMS) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.f;
  }
  const float inv = 1.f / static_cast<float>(a.H);
  for (long long row = static_cast<long long>(blockIdx.x) * AT_ONCE<G> + threadIdx.x / G;
       row < a.M; row += static_cast<long long>(gridDim.x) * AT_ONCE<G>) {
    const size_t off = static_cast<size_t>(row) * a.H;
    Vec8<T> qy[NV], qh[NV], qd[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = (i * G + lane) * 8;
      if (at < a.H) {
        qy[i].load(dy + off + at);
        qh[i].load(h + off + at);
        if (dh) qd[i].load(dh + off + at);
      }
    }
    const float mu = mean[row], rs = rstd[row];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = (i * G + lane) * 8;
      if (at < a.H) {
        float d[8], x[8], w[8];
        qy[i].get(d);
        qh[i].get(x);
        load_param(weight, a.w_bf16, at, 1.f, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = (x[j] - mu) * rs, g = d[j] * w[j];
          s1 += g;
          s2 += g * xh;
          if constexpr (SUMS) {
            dw[i][j] += d[j] * xh;
            db[i][j] += d[j];
          }
        }
      }
    }
    if (dx) {
      const float2 t = sum(s1, s2);
      const float m1 = t.x * inv, m2 = t.y * inv;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int at = (i * G + lane) * 8;
        if (at < a.H) {
          float d[8], x[8], w[8], e[8];
          qy[i].get(d);
          qh[i].get(x);
          load_param(weight, a.w_bf16, at, 1.f, w);
          if (dh) qd[i].get(e);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float xh = (x[j] - mu) * rs;
            d[j] = rs * (d[j] * w[j] - m1 - xh * m2) + (dh ? e[j] : 0.f);
          }
          Vec8<T> q;
          q.set(d);
          q.store(dx + off + at);
        }
      }
    }
  }
  if constexpr (SUMS) {
    float* out = part + static_cast<size_t>(blockIdx.x) * 2 * a.H;
    if constexpr (G > 32) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int at = (i * G + lane) * 8;
        if (at < a.H) {
          Vec8<float> q;
          q.set(dw[i]);
          q.store(out + at);
          q.set(db[i]);
          q.store(out + a.H + at);
        }
      }
    } else {  // the block's warps in their order
      __shared__ float cols_s[2][32 * NV * 8];
      for (int w = 0; w < AT_ONCE<G>; ++w) {
        if (threadIdx.x / 32 == w) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int at = (i * 8 + j) * 32 + lane;
              cols_s[0][at] = w ? cols_s[0][at] + dw[i][j] : dw[i][j];
              cols_s[1][at] = w ? cols_s[1][at] + db[i][j] : db[i][j];
            }
        }
        __syncthreads();
      }
      for (int c = threadIdx.x; c < a.H; c += THREADS<G>) {
        const int at = (c / 256 * 8 + c % 8) * 32 + c / 8 % 32;
        out[c] = cols_s[0][at];
        out[a.H + c] = cols_s[1][at];
      }
    }
  }
}

// The blocks' sums of a column: 8 threads a column, then their sums.
__global__ void __launch_bounds__(256)
    k_layernorm_sums(const int H, const int blocks, const float* __restrict__ part, void* dweight,
                     void* dbias, const bool bf16, const bool accum) {
  __shared__ float s[8][33];
  const int lane = threadIdx.x % 32, r = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  void* out = blockIdx.y == 0 ? dweight : dbias;
  pdl_wait();
  pdl_launch_dependents();
  if (!out) return;
  float t = 0.f;
  if (c < H) {
    const float* p = part + static_cast<size_t>(blockIdx.y) * H + c;
#pragma unroll 8
    for (int b = r; b < blocks; b += 8) t += p[static_cast<size_t>(b) * 2 * H];
  }
  s[r][lane] = t;
  __syncthreads();
  if (r || c >= H) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) t += s[i][lane];
  if (accum) static_cast<float*>(out)[c] += t;
  else if (bf16) static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(t);
  else static_cast<float*>(out)[c] = t;
}

// Threads a row and vectors a thread, by the row's length.
template <class F>
cudaError_t by_width(int H, F&& f) {
  const int vecs = H / 8;
#define MLP_NORM_SHAPE(G, NV) \
  return f(std::integral_constant<int, G>{}, std::integral_constant<int, NV>{})
  if (vecs <= 32) MLP_NORM_SHAPE(32, 1);
  if (vecs <= 64) MLP_NORM_SHAPE(32, 2);
  if (vecs <= 128) MLP_NORM_SHAPE(32, 4);
  if (vecs <= 256) MLP_NORM_SHAPE(128, 2);
  if (vecs <= 512) MLP_NORM_SHAPE(256, 2);
  if (vecs <= 1024) MLP_NORM_SHAPE(512, 2);
  MLP_NORM_SHAPE(512, 4);
#undef MLP_NORM_SHAPE
}
int rows_of(int H) { return H <= 1024 ? 8 : 1; }

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

template <typename T>
cudaError_t fwd_of(const NormArgs& a, const void* x, const void* residual, const void* weight,
                   const void* bias, void* y, void* h, float* mean, float* rstd,
                   cudaStream_t stream) {
  return by_width(a.H, [&](auto g, auto nv) {
    constexpr int G = decltype(g)::value, NV = decltype(nv)::value;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg =
        config(dim3((a.M - 1) / AT_ONCE<G> + 1), THREADS<G>, stream, attr);
    return cudaLaunchKernelEx(&cfg, k_layernorm_fwd<T, G, NV>, a, static_cast<const T*>(x),
                              static_cast<const T*>(residual), weight, bias, static_cast<T*>(y),
                              static_cast<T*>(h), mean, rstd);
  });
}

template <typename T>
cudaError_t bwd_of(const NormArgs& a, const void* dy, const void* h, const void* weight,
                   const float* mean, const float* rstd, const void* dh, void* dx, float* part,
                   int* status, cudaStream_t stream) {
  return by_width(a.H, [&](auto g, auto nv) {
    constexpr int G = decltype(g)::value, NV = decltype(nv)::value;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg =
        config(dim3(layernorm_blocks(a.M, a.H)), THREADS<G>, stream, attr);
    auto go = [&](auto kern) {
      return cudaLaunchKernelEx(&cfg, kern, a, static_cast<const T*>(dy),
                                static_cast<const T*>(h), weight, mean, rstd,
                                static_cast<const T*>(dh), static_cast<T*>(dx), part, status);
    };
    return part ? go(k_layernorm_bwd<T, G, NV, true>) : go(k_layernorm_bwd<T, G, NV, false>);
  });
}

}  // namespace

// (a function of the sizes alone: the workspace is, too)
int layernorm_blocks(int M, int H) {
  const int all = (M - 1) / rows_of(H) + 1;
  const int most = H <= 2048 ? 4 * 152 : H <= 4096 ? 2 * 152 : 152;
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
  cudaLaunchConfig_t cfg = config(dim3((H + 31) / 32, 2), 256, stream, attr);
  return cudaLaunchKernelEx(&cfg, k_layernorm_sums, H, blocks, part, dweight, dbias, w_bf16, accum);
}

}  // namespace mlpk
