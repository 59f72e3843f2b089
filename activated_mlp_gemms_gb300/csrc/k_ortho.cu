// The orthogonalised update (mlp_ortho.h): the norm of G, X = G / (|G| + eps), and the
// products of a Newton-Schulz step,
//   A = X X^T,  P = b A + c A A,  X <- a X + P X,
// on the tensor cores.
//
// Arithmetic.  The iteration stretches small singular values by up to a = 3.4 a step, and
// with them the rounding of X: in bf16 terms alone five steps leave 1-30 % of error.  Here X is
// the sum of two fp16 terms (22 bits), so that a X carries no rounding; the products take the
// leading terms (11 bits, the same speed as bf16), whose errors the contraction of the other
// singular values damps: 0.2-1.7e-3 of the result over spectra from flat to 1e-4, at or below
// the rounding of a bf16 result.  An fp32 result takes hi lo + lo hi + hi hi, as an fp32
// product would have it (1e-5 and below).
//
// The GEMM: one CTA of 320 threads an SM; CTA pairs with 256 x 256 tiles (tcgen05
// cta_group::2), or single CTAs with 128 x 128 tiles where those are too few.
//   warp 0     TMA loads of both operands' 64-wide k-blocks into a ring of six 32 KB stages
//   warp 1     issues tcgen05.mma into one of two accumulators; in a pair's other CTA it
//              tells the leader that the accumulator has been read
//   warps 2-9  read the accumulator (a row a thread), add `in`, round and store
// The units are dealt in turn (unit u to cluster u mod clusters): all cost the same.  Of a
// symmetric product only the tiles on and below the diagonal are formed, and stored twice.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "gemm_params.h"
#include "ortho.h"
#include "ptx.cuh"

namespace mlpk {

namespace {

constexpr int OSTAGES = 6;
constexpr int OPERAND = 128 * 64 * 2;  // bytes of an operand's k-block in one CTA
constexpr int OSTAGE = 2 * OPERAND;
constexpr int OTHREADS = 320;
constexpr int OSMEM = OSTAGES * OSTAGE + 1024 + 256;  // ring, alignment, control block
constexpr int O_TIMEOUT = -6;                         // MLP_ERR_TIMEOUT

// kind::f16 with fp16 operands (format 0), fp32 accumulators, M = N = TILE.
template <int TILE, bool Q_MN>
constexpr uint32_t IDESC_FP16 = (1u << 4) | ((Q_MN ? 1u : 0u) << 16) |
                                (static_cast<uint32_t>(TILE >> 3) << 17) |
                                (static_cast<uint32_t>(TILE >> 4) << 24);

struct Tile {
  int b, tm, tn;
};
__device__ __forceinline__ Tile tile_of(const OrthoGemm& g, int unit) {
  Tile t;
  const int per = g.units / g.batch;
  t.b = unit / per;
  const int u = unit - t.b * per;
  if (g.sym) {  // row tm of the triangle begins at tm (tm + 1) / 2
    t.tm = static_cast<int>((sqrtf(8.f * static_cast<float>(u) + 1.f) - 1.f) * 0.5f);
    while (t.tm * (t.tm + 1) / 2 > u) --t.tm;
    while ((t.tm + 1) * (t.tm + 2) / 2 <= u) ++t.tm;
    t.tn = u - t.tm * (t.tm + 1) / 2;
  } else {  // down the rows of P, then the next columns: Q's panel is read by all at once
    t.tn = u / g.tiles_m;
    t.tm = u - t.tn * g.tiles_m;
  }
  return t;
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// A thread's 32 columns [col, col + 32) of row `row` of matrix b of the stack.
__device__ __forceinline__ void store_chunk(const OrthoGemm& g, int b, int row, int col,
                                            bool mirror, const uint32_t (&acc)[32]) {
  const bool row_ok = row < g.M;
  const size_t mn = static_cast<size_t>(g.M) * g.N;
  const size_t at = b * mn + static_cast<size_t>(row) * g.N + col;
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = g.beta * __uint_as_float(acc[i]);
  if (g.in_hi && row_ok) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (col + 8 * i >= g.N) break;
      const uint4 h = ld_global_v4(static_cast<const __half*>(g.in_hi) + at + 8 * i);
      const uint32_t hw[4] = {h.x, h.y, h.z, h.w};
      uint32_t lw[4] = {};
      if (g.in_lo) {
        const uint4 l = ld_global_v4(static_cast<const __half*>(g.in_lo) + at + 8 * i);
        lw[0] = l.x, lw[1] = l.y, lw[2] = l.z, lw[3] = l.w;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = unpack_half2(hw[j]), y = unpack_half2(lw[j]);
        v[8 * i + 2 * j] += g.alpha * (x.x + y.x);
        v[8 * i + 2 * j + 1] += g.alpha * (x.y + y.y);
      }
    }
  }
  if (g.out) {
    if (g.transposed) {  // the warp's 32 rows are contiguous
      if (row_ok) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (col + i >= g.N) break;
          const size_t o = b * mn + static_cast<size_t>(col + i) * g.M + row;
          if (g.out_bf16) static_cast<__nv_bfloat16*>(g.out)[o] = __float2bfloat16_rn(v[i]);
          else static_cast<float*>(g.out)[o] = v[i];
        }
      }
    } else if (row_ok) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (col + 8 * i >= g.N) break;
        const float* f = v + 8 * i;
        if (g.out_bf16) {
          st_global_v4(static_cast<__nv_bfloat16*>(g.out) + at + 8 * i,
                       make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                  pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])));
        } else {
          float* o = static_cast<float*>(g.out) + at + 8 * i;
          *reinterpret_cast<float4*>(o) = make_float4(f[0], f[1], f[2], f[3]);
          *reinterpret_cast<float4*>(o + 4) = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
    }
    return;
  }
#pragma unroll
  for (int term = 0; term < 2; ++term) {
    __half* to = static_cast<__half*>(term ? g.lo : g.hi);
    if (!to) break;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      w[i] = pack_half2(v[2 * i], v[2 * i + 1]);
      const float2 x = unpack_half2(w[i]);  // the second term: what the first leaves
      v[2 * i] -= x.x;
      v[2 * i + 1] -= x.y;
    }
    if (!row_ok) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + 8 * i < g.N)
        st_global_v4(to + at + 8 * i, make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
    if (mirror) {  // (symmetric: M is N)
      uint16_t* m = reinterpret_cast<uint16_t*>(to) + b * mn + row;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (col + i >= g.N) break;
        m[static_cast<size_t>(col + i) * g.N] =
            static_cast<uint16_t>(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
      }
    }
  }
}

template <int CG, bool Q_MN>
__global__ void __launch_bounds__(OTHREADS, 1) k_ortho_gemm(const __grid_constant__ OrthoGemm g) {
  extern __shared__ uint8_t ortho_smem[];
  constexpr bool PAIR = CG == 2;
  constexpr int TILE = 128 * CG;  // rows and columns of a tile
  constexpr uint32_t IDESC = IDESC_FP16<TILE, Q_MN>;
  constexpr uint32_t COLS = 2 * TILE;  // two accumulators
  const uint32_t base = (smem_u32(ortho_smem) + 1023u) & ~1023u;
  uint8_t* ctrl = ortho_smem + (base - smem_u32(ortho_smem)) + OSTAGES * OSTAGE;
  uint64_t* bar = reinterpret_cast<uint64_t*>(ctrl);
  constexpr int FULL = 0, EMPTY = OSTAGES, TFULL = 2 * OSTAGES, TEMPTY = TFULL + 2,
                DRAIN = TEMPTY + 2, NBAR = DRAIN + 1;
  static_assert(8 * NBAR + 8 <= 256, "control block");
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(ctrl + 8 * NBAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_s + 1);
  auto bar_s = [&](int i) { return smem_u32(bar + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  auto lead = [&](uint32_t local) { return PAIR ? mapa_shared(local, 0) : local; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < OSTAGES; ++i) {
      mbar_init(bar_s(FULL + i), 1);
      mbar_init(bar_s(EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_s(TFULL + i), 1);
      // the eight epilogue warps; the leader's also: the other CTA's
      mbar_init(bar_s(TEMPTY + i), 8 + (PAIR && leader ? 1 : 0));
    }
    mbar_init(bar_s(DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&g.p);
    prefetch_tmap(&g.q);
  }
  if (warp == 1) {
    tmem_alloc<CG>(smem_u32(tmem_s), COLS);
    tmem_relinquish<CG>();
  }
  tc_fence_before();
  if constexpr (PAIR) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_s;
  pdl_wait();
  pdl_launch_dependents();

  const uint64_t lim = g.timeout_ns;
  const int first = static_cast<int>(blockIdx.x) / CG, step = static_cast<int>(gridDim.x) / CG;
  const int segs = g.terms == 2 ? 3 : 1;
  const int kb_all = g.kblocks * segs;
  auto failed = [&] {
    *abort_flag = 1;
    atomicExch(g.status, O_TIMEOUT);
  };

  if (warp == 0) {
    if (lane == 0 && !(g.debug_flags & 1)) {  // (testing: without loads the waits run out)
      fence_proxy_async_global();  // the previous kernel's plain stores, before TMA's reads
      const uint64_t pol = policy_evict_normal();
      const uint32_t full0 = lead(bar_s(FULL));
      auto load = [&](uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, uint32_t full) {
        if constexpr (PAIR) tma_load_3d_pair(dst, m, c0, c1, c2, full, pol);
        else tma_load_3d(dst, m, c0, c1, c2, full, pol);
      };
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int unit = first; ok && unit < g.units; unit += step) {
        const Tile t = tile_of(g, unit);
        const int m0 = t.tm * TILE + static_cast<int>(rank) * 128;
        const int n0 = t.tn * TILE + static_cast<int>(rank) * 128;
        int seg = 0, kb = 0;
        for (int i = 0; i < kb_all; ++i) {
          if (!mbar_wait<PAIR>(bar_s(EMPTY + stage), phase ^ 1u, lim, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t full = full0 + 8u * stage, s = base + stage * OSTAGE;
          if (leader) mbar_expect_tx(bar_s(FULL + stage), CG * OSTAGE);
          const int k0 = kb * 64;
          // the terms' depths: hi lo, lo hi, hi hi.  (The accumulator truncates at every
          // instruction, by more the larger its sum: the small products come first.)
          const int zp = t.b + (segs == 3 && seg == 1 ? g.batch : 0);
          const int zq = t.b + (segs == 3 && seg == 0 ? g.batch : 0);
          load(s, &g.p, k0, m0, zp, full);
          if constexpr (Q_MN) {
            load(s + OPERAND, &g.q, n0, k0, zq, full);
            load(s + OPERAND + OPERAND / 2, &g.q, n0 + 64, k0, zq, full);
          } else {
            load(s + OPERAND, &g.q, k0, n0, zq, full);
          }
          ++issued;
          if (++kb == g.kblocks) { kb = 0; ++seg; }
          if (++stage == OSTAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {
        failed();
        if (leader) {  // copies in flight land before shared memory is released
          for (int i = 0; i < OSTAGES && i < issued; ++i) {
            if (--stage < 0) { stage = OSTAGES - 1; phase ^= 1u; }
            volatile int never = 0;
            mbar_wait<PAIR>(bar_s(FULL + stage), phase, 10000000ull, &never);
          }
        } else {
          __nanosleep(100000);  // its copies signal the leader's barriers
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, aphase = 0;
      bool ok = true, any = false;
      for (int unit = first; ok && unit < g.units; unit += step) {
        if (!mbar_wait<PAIR>(bar_s(TEMPTY + acc), aphase ^ 1u, lim, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + acc * TILE;
        for (int i = 0; i < kb_all; ++i) {
          if (!mbar_wait<PAIR>(bar_s(FULL + stage), phase, lim, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sp = base + stage * OSTAGE, sq = sp + OPERAND;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t pd = sdesc_sw128(sp + k * 32, 16, 1024);
            const uint64_t qd = Q_MN ? sdesc_sw128(sq + k * 2048, 8192, 1024)
                                     : sdesc_sw128(sq + k * 32, 16, 1024);
            if constexpr (PAIR) tc_mma_bf16_pair(d, pd, qd, IDESC, i > 0 || k > 0);
            else tc_mma_bf16(d, pd, qd, IDESC, i > 0 || k > 0);
          }
          any = true;
          if constexpr (PAIR) tc_commit_pair(bar_s(EMPTY + stage), 3);
          else tc_commit(bar_s(EMPTY + stage));
          if (++stage == OSTAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if constexpr (PAIR) tc_commit_pair(bar_s(TFULL + acc), 3);
        else tc_commit(bar_s(TFULL + acc));
        acc ^= 1;
        if (acc == 0) aphase ^= 1u;
      }
      if (!ok) {
        failed();
        if (any) {  // the MMAs already issued end before TMEM is freed
          if constexpr (PAIR) tc_commit_pair(bar_s(DRAIN), 1);
          else tc_commit(bar_s(DRAIN));
          volatile int never = 0;
          mbar_wait<PAIR>(bar_s(DRAIN), 0, 10000000ull, &never);
        }
      }
    } else if (PAIR && lane == 0) {
      // tells the leader that this CTA's warps have read an accumulator: one release at
      // cluster scope, from a thread that has no stores of its own to wait for
      int acc = 0;
      uint32_t aphase = 0;
      for (int unit = first; unit < g.units; unit += step) {
        if (!mbar_wait(bar_s(TEMPTY + acc), aphase, lim, abort_flag)) {
          failed();
          break;
        }
        tc_fence_after();
        tc_fence_before();
        mbar_arrive_cluster(lead(bar_s(TEMPTY + acc)));
        acc ^= 1;
        if (acc == 0) aphase ^= 1u;
      }
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;  // TMEM lanes, half of the columns
    int acc = 0;
    uint32_t aphase = 0;
    for (int unit = first; unit < g.units; unit += step) {
      const Tile t = tile_of(g, unit);
      if (!mbar_wait<PAIR>(bar_s(TFULL + acc), aphase, lim, abort_flag)) {
        failed();
        break;
      }
      tc_fence_after();
      const int row0 = t.tm * TILE + static_cast<int>(rank) * 128 + q * 32;
      const uint32_t tb = tmem + acc * TILE + (static_cast<uint32_t>(q * 32) << 16);
      if (row0 < g.M) {
#pragma unroll 1
        for (int c = half * (TILE / 2); c < (half + 1) * (TILE / 2); c += 32) {
          const int col = t.tn * TILE + c;
          if (col >= g.N) break;
          uint32_t a[32];
          __syncwarp();
          tmem_ld32(tb + c, a);
          tmem_wait_ld();
          store_chunk(g, t.b, row0 + lane, col, g.sym && t.tm != t.tn, a);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_s(TEMPTY + acc));
      acc ^= 1;
      if (acc == 0) aphase ^= 1u;
    }
  }

  tc_fence_before();
  if constexpr (PAIR) cluster_sync();  // no remote arrival or copy may target an exited CTA
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<CG>(tmem, COLS);
  }
}

template <int CG, bool Q_MN>
cudaError_t prepare() {
  auto kern = k_ortho_gemm<CG, Q_MN>;
  static std::atomic<unsigned long long> done{0};  // devices that have the attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load() >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, OSMEM);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev);
  return e;
}

cudaLaunchConfig_t ortho_config(int cg, int grid, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(OTHREADS, 1, 1);
  cfg.dynamicSmemBytes = OSMEM;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cg);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

template <int CG, bool Q_MN>
int clusters() {
  if (prepare<CG, Q_MN>() != cudaSuccess) return 0;
  int dev = 0, sms = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  static std::atomic<int> cache[64];
  if (dev < 64 && cache[dev].load() > 0) return cache[dev].load();
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = ortho_config(CG, sms / CG * CG, nullptr, attr);
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, k_ortho_gemm<CG, Q_MN>, &cfg) != cudaSuccess) return 0;
  if (dev < 64) cache[dev].store(n);
  return n;
}

template <int CG, bool Q_MN>
cudaError_t launch_of(const OrthoGemm& g, cudaStream_t stream) {
  const int n = clusters<CG, Q_MN>();
  if (n <= 0) return cudaErrorUnknown;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = ortho_config(CG, CG * (g.units < n ? g.units : n), stream, attr);
  return cudaLaunchKernelEx(&cfg, k_ortho_gemm<CG, Q_MN>, g);
}

// ------------------------------------------------------------- norm and scale
constexpr int NORM_THREADS = 512;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 v = ld_global_v4(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack_bf16x2(w[i]);
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  } else {
    const uint4 a = ld_global_v4(p), b = ld_global_v4(p + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  }
}

template <typename T>
__global__ void __launch_bounds__(NORM_THREADS)
    k_ortho_norm(const T* __restrict__ G, long long size, float* __restrict__ part, int* status) {
  __shared__ float warps_s[NORM_THREADS / 32];
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = 0;
  const T* M = G + blockIdx.y * size;
  float s = 0.f;
#pragma unroll 4
  for (long long i = (static_cast<long long>(blockIdx.x) * NORM_THREADS + threadIdx.x) * 8;
       i < size; i += static_cast<long long>(ORTHO_PARTS) * NORM_THREADS * 8) {
    float f[8];
    load8(M + i, f);
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) t += f[j] * f[j];
    s += t;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (threadIdx.x % 32 == 0) warps_s[threadIdx.x / 32] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < NORM_THREADS / 32; ++i) s += warps_s[i];
    part[blockIdx.y * ORTHO_PARTS + blockIdx.x] = s;
  }
}

// 64 x 64 values a block: straight, or through shared memory with rows and columns changed.
template <typename T>
__global__ void __launch_bounds__(256)
    k_ortho_scale(const T* __restrict__ G, int rows, int cols, int batch,
                  const float* __restrict__ part, float eps, __half* __restrict__ X) {
  __shared__ float tile[64][65];
  __shared__ float factor_s;
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.z;
  if (threadIdx.x < 32) {
    const float* p = part + b * ORTHO_PARTS;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < ORTHO_PARTS / 32; ++i) s += p[threadIdx.x + 32 * i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x == 0) factor_s = ORTHO_X / (sqrtf(s) + eps);
  }
  const size_t size = static_cast<size_t>(rows) * cols;
  const T* M = G + b * size;
  __half* hi = X + b * size;
  __half* lo = hi + static_cast<size_t>(batch) * size;
  const int r0 = static_cast<int>(blockIdx.y) * 64, c0 = static_cast<int>(blockIdx.x) * 64;
  const bool transposed = rows > cols;
  __syncthreads();
  const float factor = factor_s;
  auto put = [&](size_t at, const float (&f)[8]) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = f[2 * j] * factor, c = f[2 * j + 1] * factor;
      h[j] = pack_half2(a, c);
      const float2 x = unpack_half2(h[j]);
      l[j] = pack_half2(a - x.x, c - x.y);
    }
    st_global_v4(hi + at, make_uint4(h[0], h[1], h[2], h[3]));
    st_global_v4(lo + at, make_uint4(l[0], l[1], l[2], l[3]));
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int v = static_cast<int>(threadIdx.x) + 256 * i, r = v / 8, c = v % 8 * 8;
    if (r0 + r < rows && c0 + c < cols) {
      float f[8];
      load8(M + static_cast<size_t>(r0 + r) * cols + c0 + c, f);
      if (!transposed) {
        put(static_cast<size_t>(r0 + r) * cols + c0 + c, f);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) tile[r][c + j] = f[j];
      }
    }
  }
  if (!transposed) return;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int v = static_cast<int>(threadIdx.x) + 256 * i, c = v / 8, r = v % 8 * 8;
    if (c0 + c < cols && r0 + r < rows) {  // (rows and cols are multiples of 8)
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = tile[r + j][c];
      put(static_cast<size_t>(c0 + c) * rows + r0 + r, f);
    }
  }
}

cudaLaunchConfig_t plain_config(dim3 grid, int threads, cudaStream_t stream,
                                cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

int ortho_clusters(int cg, bool q_mn) {
  if (cg == 2) return q_mn ? clusters<2, true>() : clusters<2, false>();
  return q_mn ? clusters<1, true>() : clusters<1, false>();
}

cudaError_t launch_ortho_gemm(const OrthoGemm& g, int cg, bool q_mn, cudaStream_t stream) {
  cudaError_t e;
  if (cg == 2) {
    if ((e = q_mn ? prepare<2, true>() : prepare<2, false>()) != cudaSuccess) return e;
    return q_mn ? launch_of<2, true>(g, stream) : launch_of<2, false>(g, stream);
  }
  if ((e = q_mn ? prepare<1, true>() : prepare<1, false>()) != cudaSuccess) return e;
  return q_mn ? launch_of<1, true>(g, stream) : launch_of<1, false>(g, stream);
}

cudaError_t launch_ortho_norm(const void* G, bool bf16, long long size, int batch, float* part,
                              int* status, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = plain_config(dim3(ORTHO_PARTS, batch), NORM_THREADS, stream, attr);
  if (bf16)
    return cudaLaunchKernelEx(&cfg, k_ortho_norm<__nv_bfloat16>,
                              static_cast<const __nv_bfloat16*>(G), size, part, status);
  return cudaLaunchKernelEx(&cfg, k_ortho_norm<float>, static_cast<const float*>(G), size, part,
                            status);
}

cudaError_t launch_ortho_scale(const void* G, bool bf16, int rows, int cols, int batch,
                               const float* part, float eps, void* X, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg =
      plain_config(dim3((cols + 63) / 64, (rows + 63) / 64, batch), 256, stream, attr);
  if (bf16)
    return cudaLaunchKernelEx(&cfg, k_ortho_scale<__nv_bfloat16>,
                              static_cast<const __nv_bfloat16*>(G), rows, cols, batch, part, eps,
                              static_cast<__half*>(X));
  return cudaLaunchKernelEx(&cfg, k_ortho_scale<float>, static_cast<const float*>(G), rows, cols,
                            batch, part, eps, static_cast<__half*>(X));
}

}  // namespace mlpk
