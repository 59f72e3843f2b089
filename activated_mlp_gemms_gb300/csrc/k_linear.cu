// The linear layer's kernels beside its GEMM:
//   k_linear_stream  a few rows: the weights stream once (HBM-bound), dot
//                    products on the warp-level MMA as in k_decode_mma.cu,
//                    bias, activation and residual in the epilogue (one row of
//                    14336 x 4096: 20.4 us, 5.8 TB/s)
//   k_linear_dact    dz = dout act'(z), and the bias gradient's partial sums
//                    in the same pass over dout (HBM-bound: 3 M N bf16 values;
//                    8192 x 4864 with the GELU's derivative and db 38 us, 6.2 TB/s)
//   k_linear_db      the sum of those partial sums, in a fixed order
// All epilogue arithmetic is fp32 and rounds once, to the bf16 it stores.
#include <atomic>
#include <type_traits>

#include "act.cuh"
#include "linear.h"
#include "stream.cuh"

namespace mlpk {

namespace {

using bf = __nv_bfloat16;

template <class... Args, class... Given>
cudaError_t launch(void (*kern)(Args...), dim3 grid, int threads, cudaStream_t stream, bool pdl,
                   Given... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Args>(args)...);
}

// Calls f with the activation as a compile-time constant.
template <class F>
cudaError_t with_act(int act, F&& f) {
  switch (act) {
    case ACT_SILU_EXP: return f(std::integral_constant<int, ACT_SILU_EXP>{});
    case ACT_RELU_SQ: return f(std::integral_constant<int, ACT_RELU_SQ>{});
    case ACT_GELU_EXP: return f(std::integral_constant<int, ACT_GELU_EXP>{});
    case ACT_RELU: return f(std::integral_constant<int, ACT_RELU>{});
    case ACT_SIGMOID_EXP: return f(std::integral_constant<int, ACT_SIGMOID_EXP>{});
    default: return f(std::integral_constant<int, ACT_NONE>{});
  }
}

constexpr int LS_MAX_WARPS = 16;
constexpr int LS_ROWS = 16;  // weight rows of a CTA (the MMA's M)

// A CTA owns 16 weight rows and all of K; its warps take the 64-wide k groups
// round-robin with two in flight each, and their sums meet in shared memory.
template <int ACT>
__global__ void __launch_bounds__(32 * LS_MAX_WARPS)
    k_linear_stream(const bf* __restrict__ x, int ldx, const bf* __restrict__ Wt,
                    const bf* __restrict__ bias, const bf* resid, int ldr, float rs, bf* out,
                    int ldo, bf* __restrict__ pre, int M, int N, int K, int* status) {
  using G = MdGroup<1, 8, 1>;
  __shared__ float4 part[LS_MAX_WARPS][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nwarps = blockDim.x >> 5;
  const int row0 = blockIdx.x * LS_ROWS;
  const bf* const W[2] = {Wt, nullptr};
  const int ngroups = (K + MD_KG - 1) / MD_KG;
  const int m = lane >> 2;
  const bf* const tok[1] = {m < M ? x + static_cast<size_t>(m) * ldx : nullptr};
  float acc[1][1][1][4] = {};
  G buf[2];
  pdl_wait();  // before the weights too: the kernel before may have written them
  if (warp < ngroups) buf[0].load_w(W, row0, N, K, warp * MD_KG, lane);
  if (status != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  if (warp < ngroups) buf[0].load_t_rows(tok, K, warp * MD_KG, lane);
  if (warp + nwarps < ngroups) {
    buf[1].load_w(W, row0, N, K, (warp + nwarps) * MD_KG, lane);
    buf[1].load_t_rows(tok, K, (warp + nwarps) * MD_KG, lane);
  }
  pdl_launch_dependents();
  for (int gi = warp; gi < ngroups;) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (gi < ngroups) {
        buf[j].mma(acc);
        const int nx = gi + 2 * nwarps;
        if (nx < ngroups) {
          buf[j].load_w(W, row0, N, K, nx * MD_KG, lane);
          buf[j].load_t_rows(tok, K, nx * MD_KG, lane);
        }
      }
      gi += nwarps;
    }
  }
  part[warp][lane] = make_float4(acc[0][0][0][0], acc[0][0][0][1], acc[0][0][0][2],
                                 acc[0][0][0][3]);
  __syncthreads();
  if (warp != 0) return;
  float4 v = part[0][lane];
  for (int w = 1; w < nwarps; ++w) {
    const float4 u = part[w][lane];
    v.x += u.x;
    v.y += u.y;
    v.z += u.z;
    v.w += u.w;
  }
  const float y[4] = {v.x, v.y, v.z, v.w};
  // element (h, e) of lane (g, q): weight row g + 8h, token 2q + e
  const int g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = row0 + g + 8 * h;
    if (n >= N) continue;
    const float b = bias ? __bfloat162float(bias[n]) : 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = 2 * q + e;
      if (t >= M) continue;
      const float z = y[2 * h + e] + b;
      float o = act_f<ACT>(z);
      if (resid) o = fmaf(rs, __bfloat162float(resid[static_cast<size_t>(t) * ldr + n]), o);
      if (pre) pre[static_cast<size_t>(t) * N + n] = __float2bfloat16_rn(z);
      out[static_cast<size_t>(t) * ldo + n] = __float2bfloat16_rn(o);
    }
  }
}

// Warps per CTA: the most with which the whole grid is resident at once (every
// CTA then streams its share of HBM evenly, with no partial last wave).
template <int ACT>
int stream_warps(int blocks, int ngroups) {
  static std::atomic<int> occ_cache[LS_MAX_WARPS + 1];  // CTAs per SM by warps, + 1 (0: unknown)
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 2;
  int best = 2;
  for (int w = 2; w <= LS_MAX_WARPS && w <= ngroups; ++w) {
    int occ = occ_cache[w].load() - 1;
    if (occ < 0) {
      if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, k_linear_stream<ACT>, 32 * w, 0) !=
          cudaSuccess)
        return best;
      occ_cache[w].store(occ + 1);
    }
    if (static_cast<long long>(occ) * sms >= blocks) best = w;
  }
  return best;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = unpack_bf16x2(q[i]);
    f[2 * i] = u.x;
    f[2 * i + 1] = u.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

constexpr int DACT_WARPS = 8;
constexpr int DACT_BLOCKS = 6;  // resident on an SM: 48 warps, two rows in flight each
constexpr int DACT_COLS = 256;  // columns of a block: 8 (16 bytes) per lane

// Block (cx, cy): 256 columns, a chunk of rows; warp w takes rows w, w + 8, ...
// of the chunk, two at a time.  Where dz is stored, dout and pre are read for the
// last time and leave L2 first, so that dz is still there for the GEMMs (4 blocks of
// four rows in flight a warp, without that hint: 45 us for the 38 above).
template <int ACT>
__global__ void __launch_bounds__(32 * DACT_WARPS, DACT_BLOCKS)
    k_linear_dact(const bf* __restrict__ dout, int ldd, const bf* __restrict__ pre,
                  bf* __restrict__ dz, float* __restrict__ part, void* __restrict__ db, int accum,
                  int M, int N, int chunk, int* status) {
  __shared__ float sums[DACT_WARPS][DACT_COLS];
  pdl_wait();
  pdl_launch_dependents();
  if (status != nullptr && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * DACT_COLS + 8 * lane;
  const int r0 = blockIdx.y * chunk, r1 = min(M, r0 + chunk);
  const uint64_t pol = dz ? policy_evict_first() : policy_evict_normal();
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < N) {
#pragma unroll 2
    for (int r = r0 + warp; r < r1; r += DACT_WARPS) {
      float d[8];
      unpack8(ld_global_v4(dout + static_cast<size_t>(r) * ldd + c, pol), d);
      if constexpr (ACT != ACT_NONE) {
        float z[8];
        unpack8(ld_global_v4(pre + static_cast<size_t>(r) * N + c, pol), z);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float a, da;
          act_and_grad<ACT>(z[k], a, da);
          d[k] *= da;
        }
      }
      if (dz) st_global_v4(dz + static_cast<size_t>(r) * N + c, pack8(d));
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] += d[k];
    }
  }
  if (!part) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) sums[warp][8 * lane + k] = s[k];
  __syncthreads();
  const int n = blockIdx.x * DACT_COLS + threadIdx.x;
  if (n < N) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < DACT_WARPS; ++w) t += sums[w][threadIdx.x];
    if (gridDim.y > 1) part[static_cast<size_t>(blockIdx.y) * N + n] = t;
    else if (accum) static_cast<float*>(db)[n] += t;
    else static_cast<bf*>(db)[n] = __float2bfloat16_rn(t);
  }
}

// A block sums 32 columns; warp w takes chunks w, w + 16, ... (one thread a column,
// over all chunks, was a chain of loads: 9 us longer for 1024 columns of 152 chunks).
constexpr int DB_WARPS = 16;
__global__ void __launch_bounds__(32 * DB_WARPS)
    k_linear_db(const float* __restrict__ part, int chunks, void* __restrict__ db, int N,
                int accum) {
  __shared__ float sums[DB_WARPS][32];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = blockIdx.x * 32 + lane;
  float t = 0.f;
  if (n < N) {
#pragma unroll 8
    for (int k = warp; k < chunks; k += DB_WARPS) t += part[static_cast<size_t>(k) * N + n];
  }
  sums[warp][lane] = t;
  __syncthreads();
  if (warp != 0 || n >= N) return;
#pragma unroll
  for (int w = 1; w < DB_WARPS; ++w) t += sums[w][lane];
  if (accum) static_cast<float*>(db)[n] += t;
  else static_cast<bf*>(db)[n] = __float2bfloat16_rn(t);
}

}  // namespace

cudaError_t launch_linear_stream(const void* x, int ldx, const void* W, const void* bias,
                                 const void* resid, int ldr, float rs, void* out, int ldo,
                                 void* pre, int M, int N, int K, int act, cudaStream_t stream,
                                 bool pdl, int* status) {
  if (M < 1 || M > LINEAR_STREAM_MAX_M) return cudaErrorInvalidValue;
  const int blocks = (N + LS_ROWS - 1) / LS_ROWS;
  return with_act(act, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    const int warps = stream_warps<ACT>(blocks, (K + MD_KG - 1) / MD_KG);
    return launch(k_linear_stream<ACT>, dim3(blocks), 32 * warps, stream, pdl,
                  static_cast<const bf*>(x), ldx, static_cast<const bf*>(W),
                  static_cast<const bf*>(bias), static_cast<const bf*>(resid), ldr, rs,
                  static_cast<bf*>(out), ldo, static_cast<bf*>(pre), M, N, K, status);
  });
}

// Row chunks of the derivative pass: the blocks that fit on 152 SMs, each
// with at least 16 rows; up to 128 rows are one chunk, which needs no second
// kernel for db.
static int dact_chunk(int M, int N) {
  if (M <= 128) return M;
  const int cols = (N + DACT_COLS - 1) / DACT_COLS;
  int chunks = (DACT_BLOCKS * 152 + cols - 1) / cols;
  const int most = (M + 15) / 16;
  if (chunks > most) chunks = most;
  return (M + chunks - 1) / chunks;
}

int linear_db_chunks(int M, int N) {
  const int chunk = dact_chunk(M, N);
  return (M + chunk - 1) / chunk;
}

cudaError_t launch_linear_dact(const void* dout, int ldd, const void* pre, void* dz, float* part,
                               void* db, bool accum, int M, int N, int act, int* status,
                               cudaStream_t stream, bool pdl) {
  const dim3 grid((N + DACT_COLS - 1) / DACT_COLS, linear_db_chunks(M, N));
  return with_act(act, [&](auto a) {
    return launch(k_linear_dact<decltype(a)::value>, grid, 32 * DACT_WARPS, stream, pdl,
                  static_cast<const bf*>(dout), ldd, static_cast<const bf*>(pre),
                  static_cast<bf*>(dz), part, db, accum ? 1 : 0, M, N, dact_chunk(M, N), status);
  });
}

cudaError_t launch_linear_db(const float* part, int chunks, void* db, int N, bool accum,
                             cudaStream_t stream, bool pdl) {
  return launch(k_linear_db, dim3((N + 31) / 32), 32 * DB_WARPS, stream, pdl, part, chunks, db,
                N, accum ? 1 : 0);
}

}  // namespace mlpk
