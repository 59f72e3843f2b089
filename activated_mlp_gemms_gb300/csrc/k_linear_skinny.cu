// The linear layer where 256 x 256 output tiles are too few: out = act(x W^T +
// bias) + rs * resid, and dx = dz W, for a few dozen to some hundreds of rows (or
// a narrow N).
//
// With M rows the layer does 2 M flops per weight, below the tensor cores'
// balance against HBM up to M of a few hundred, so the weights' stream is the
// bound, and tiles of 256 output columns are too few to draw it.  The operands
// change places: 128 weight rows are the MMA's M, the rows of x its N (up to 256
// a tile, in equal tiles rounded up to 16), so a CTA streams 128 rows of W (16
// KB a k-block) against all of its rows of x, and the MMA wastes nothing on
// absent rows.  (For dx the 128 are columns of W, read MN-major in two boxes.)
// When the blocks are fewer than the SMs, a cluster of 2, 4 or 8 CTAs shares a
// block's K: the rows of x are dealt out to its CTAs, each writes its fp32 sums of
// a row to the row's owner through distributed shared memory, and the owner adds
// them in rank order.
// (Stores that nothing waits for; owners that read the others' sums instead
// waited for each round: 26 against 15 us for 160 x 1024 x 8192.)  No partial
// sums in global memory, no atomics: the same bits on every run.
//
// Measured: 48 x 14336 x 4096 23.3 us (5.1 TB/s), 16 x 4096 x 4096 10, 300 x 4096 x
// 4096 16 (27 as 256 x 256 tiles), 6740 x 592 x 2016 17.7 (33).
//
// Warp 0 feeds the ring by TMA, warp 1 issues tcgen05.mma, warps 2-9 move the
// accumulator (lane = feature) to shared memory; all ten finish rows, 8 features
// (16 bytes) of two rows a thread at a time.
#include <atomic>

#include "act.cuh"
#include "linear.h"
#include "ptx.cuh"

namespace mlpk {

namespace {

using bf = __nv_bfloat16;

constexpr int SK_THREADS = 320;
constexpr int SK_ROWS = 128;                     // weight rows of a CTA
constexpr int SK_A = SK_ROWS * BK * 2;           // bytes of a k-block of them
// bytes of the ring (2 KB of alignment and control apart): one CTA an SM, or two
constexpr int SK_MAX_SMEM = 232448 - 2048, SK_HALF_SMEM = 114688 - 2048;
constexpr int SK_MAX_STAGES = 10;
constexpr int SK_MAX_SHARE = 8;
constexpr int SK_TIMEOUT = -6;  // MLP_ERR_TIMEOUT

__host__ __device__ constexpr int sk_stage(int mp) { return SK_A + mp * BK * 2; }
__host__ __device__ constexpr int sk_stages(int mp, bool two) {
  const int n = (two ? SK_HALF_SMEM : SK_MAX_SMEM) / sk_stage(mp);
  return n < SK_MAX_STAGES ? n : SK_MAX_STAGES;
}
// the sums' [mp][128] fp32 take the ring's place
__host__ __device__ constexpr bool sk_sums_fit(int mp, bool two) {
  return sk_stages(mp, two) >= 3 && sk_stages(mp, two) * sk_stage(mp) >= mp * SK_ROWS * 4;
}
static_assert(sk_sums_fit(256, false) && sk_sums_fit(16, false) && sk_sums_fit(16, true), "ring");

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  const uint4 v = ld_shared_v4(addr);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                     __uint_as_float(v.w));
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
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

template <int ACT, bool A_MN>
__global__ void __launch_bounds__(SK_THREADS, 2)
    k_linear_skinny(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                    const bf* __restrict__ bias, const bf* resid, int ldr, float rs, bf* out,
                    int ldo, bf* __restrict__ pre, int M, int N, int K, int mp, int stages, int clear,
                    int no_work, int* status, unsigned long long limit_ns) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const int stage_bytes = sk_stage(mp);
  // 1 KB of control after the ring: full[], empty[], done, TMEM base, abort flag
  uint8_t* ctrl = smem_raw + (base - raw) + stages * stage_bytes;
  uint64_t* bar = reinterpret_cast<uint64_t*>(ctrl);
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(bar + 2 * SK_MAX_STAGES + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_s + 1);
  auto full = [&](int i) { return smem_u32(bar + i); };
  auto empty = [&](int i) { return smem_u32(bar + SK_MAX_STAGES + i); };
  const uint32_t done = smem_u32(bar + 2 * SK_MAX_STAGES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int share = gridDim.y, rank = blockIdx.y;  // the cluster that shares this block's K
  // x: the blocks of features, a row tile after the other (y and z end at 65535)
  const int blocks = (N + SK_ROWS - 1) / SK_ROWS, tile = blockIdx.x / blocks;
  const int row0 = (blockIdx.x - tile * blocks) * SK_ROWS;  // the features
  const int m0 = tile * mp, m1 = min(M, m0 + mp);
  const int kbs = (K + BK - 1) / BK;
  const int kb0 = static_cast<int>(static_cast<long long>(kbs) * rank / share);
  const int kb1 = static_cast<int>(static_cast<long long>(kbs) * (rank + 1) / share);
  const uint32_t cols = mp <= 32 ? 32u : mp <= 64 ? 64u : mp <= 128 ? 128u : 256u;

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&map_w);
    prefetch_tmap(&map_x);
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_u32(tmem_s), cols);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_s;
  pdl_wait();
  pdl_launch_dependents();
  if (clear && blockIdx.x == 0 && rank == 0 && threadIdx.x == 0) *status = 0;
  auto give_up = [&] {
    *abort_flag = 1;
    atomicExch(status, SK_TIMEOUT);
  };

  if (warp == 0) {
    if (lane == 0 && !no_work) {
      const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(empty(stage), phase ^ 1u, limit_ns, abort_flag)) {
          ok = false;
          break;
        }
        mbar_expect_tx(full(stage), stage_bytes);
        const uint32_t s = base + stage * stage_bytes;
        if constexpr (A_MN) {
          tma_load_2d(s, &map_w, row0, kb * BK, full(stage), pol_w);
          tma_load_2d(s + SK_A / 2, &map_w, row0 + 64, kb * BK, full(stage), pol_w);
        } else {
          tma_load_2d(s, &map_w, kb * BK, row0, full(stage), pol_w);
        }
        tma_load_2d(s + SK_A, &map_x, kb * BK, m0, full(stage), pol_x);
        ++issued;
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) {
        give_up();
        // the copies in flight land before shared memory is used for the sums
        for (int i = 0; i < stages && i < issued; ++i) {
          if (--stage < 0) {
            stage = stages - 1;
            phase ^= 1u;
          }
          volatile int never = 0;
          mbar_wait(full(stage), phase, 10000000ull, &never);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(SK_ROWS, mp, A_MN, false);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(full(stage), phase, limit_ns, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sA = base + stage * stage_bytes, sB = sA + SK_A;
#pragma unroll
        for (int k = 0; k < BK / 16; ++k)
          tc_mma_bf16(tmem,
                      A_MN ? sdesc_sw128(sA + k * 2048, SK_A / 2, 1024)
                           : sdesc_sw128(sA + k * 32, 16, 1024),
                      sdesc_sw128(sB + k * 32, 16, 1024), idesc, kb > kb0 || k > 0);
        tc_commit(empty(stage));
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) give_up();
      tc_commit(done);  // after the MMAs issued so far, if any
    }
  }
  __syncwarp();
  // every MMA has completed, and with them every copy: the ring is free
  const bool summed = mbar_wait(done, 0, limit_ns + limit_ns / 2, abort_flag);
  if (!summed) {  // (what was issued ends before shared memory and TMEM are used again)
    if (lane == 0) give_up();
    volatile int never = 0;
    mbar_wait(done, 0, 10000000ull, &never);
  }
  __syncwarp();
  if (share > 1) cluster_sync();  // the owners' rings are free too
  // [rank][row of the owner][feature] in every CTA: row j of the tile belongs to
  // CTA j % share, as its row j / share
  const int rows = mp / share;
  if (warp >= 2) {
    tc_fence_after();
    const int q = warp & 3;  // the TMEM lanes this warp may read: features 32 q + lane
    const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t col = base + static_cast<uint32_t>(rank * rows) * (SK_ROWS * 4) +
                         static_cast<uint32_t>(32 * q + lane) * 4u;
    for (int c = 16 * ((warp - 2) >> 2); c < mp; c += 32) {  // two warps a quadrant
      uint32_t v[16];
      tmem_ld16(tb + c, v);
      tmem_wait_ld();
      if (share == 1) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          st_shared_f32(col + static_cast<uint32_t>(c + j) * (SK_ROWS * 4), __uint_as_float(v[j]));
      } else {
        // (16 is a multiple of share)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          st_cluster_f32(mapa_shared(col + static_cast<uint32_t>((c + j) / share) * (SK_ROWS * 4),
                                     (c + j) % share),
                         __uint_as_float(v[j]));
      }
    }
    tc_fence_before();
  }
  if (share > 1) cluster_sync();  // every sum has arrived
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, cols);
  }

  // this CTA's rows of x: 16 threads a row, 8 features each, two rows at a time
  const int seg = threadIdx.x & 15, n = row0 + 8 * seg;
  if (n < N) {
    float b[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (bias) unpack8(ld_global_v4(bias + n), b);
    constexpr int STEP = SK_THREADS / 16;
    for (int la = threadIdx.x >> 4; la < rows; la += 2 * STEP) {
      uint4 rv[2];
      float z[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = m0 + rank + share * (la + h * STEP);
        rv[h] = resid && m < m1 ? ld_global_v4(resid + static_cast<size_t>(m) * ldr + n)
                                : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[h][i] = b[i];
      }
      for (int c = 0; c < share; ++c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int l = la + h * STEP < rows ? la + h * STEP : la;
          const uint32_t at = base + static_cast<uint32_t>(c * rows + l) * (SK_ROWS * 4) + 32u * seg;
          const float4 u = ld_shared_f4(at), v = ld_shared_f4(at + 16);
          z[h][0] += u.x, z[h][1] += u.y, z[h][2] += u.z, z[h][3] += u.w;
          z[h][4] += v.x, z[h][5] += v.y, z[h][6] += v.z, z[h][7] += v.w;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int l = la + h * STEP, m = m0 + rank + share * l;
        if (l >= rows || m >= m1) break;
        float r[8], o[8];
        unpack8(rv[h], r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[i] = act_f<ACT>(z[h][i]);
          if (resid) o[i] = fmaf(rs, r[i], o[i]);
        }
        if (pre)
          st_global_v4(pre + static_cast<size_t>(m) * N + n,
                       make_uint4(pack_bf16x2(z[h][0], z[h][1]), pack_bf16x2(z[h][2], z[h][3]),
                                  pack_bf16x2(z[h][4], z[h][5]), pack_bf16x2(z[h][6], z[h][7])));
        st_global_v4(out + static_cast<size_t>(m) * ldo + n,
                     make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]),
                                pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])));
      }
    }
  }
}

struct Config {
  dim3 grid;
  int mp, stages;
  size_t smem() const { return static_cast<size_t>(stages) * sk_stage(mp) + 2048; }
};

void fill(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], const Config& k,
          cudaStream_t stream, bool pdl) {
  cfg.gridDim = k.grid;
  cfg.blockDim = dim3(SK_THREADS, 1, 1);
  cfg.dynamicSmemBytes = k.smem();
  cfg.stream = stream;
  int na = 0;
  if (pdl) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (k.grid.y > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = 1;
    attr[na].val.clusterDim.y = k.grid.y;
    attr[na++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
}

// Clusters of `share` CTAs (one CTA an SM) that are resident together: fewer
// than SMs / share, as a cluster stays within a group of SMs.  Cached.
template <class Kern>
int resident_clusters(Kern kern, int share) {
  static std::atomic<int> cache[64][SK_MAX_SHARE + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = cache[dev][share].load();
  if (n > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  fill(cfg, attr, Config{dim3(1, share), 16, sk_stages(16, false)}, nullptr, false);
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  cache[dev][share].store(n);
  return n;
}

template <int ACT, bool A_MN>
cudaError_t launch(const CUtensorMap& map_w, const CUtensorMap& map_x, const bf* bias,
                   const bf* resid, int ldr, float rs, bf* out, int ldo, bf* pre, int M, int N,
                   int K, int clear, int no_work, int* status, unsigned long long limit_ns,
                   cudaStream_t stream, bool pdl) {
  auto kern = k_linear_skinny<ACT, A_MN>;
  static std::atomic<unsigned> configured{0};  // devices that got the shared-memory attribute
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (dev >= 31 || !(configured.load() & (1u << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SK_MAX_SMEM + 2048);
    if (e != cudaSuccess) return e;
    if (dev < 31) configured.fetch_or(1u << dev);
  }
  const SkinnyShape sh = linear_skinny_shape(M, N, K);
  const int blocks = sh.blocks * sh.tiles, kbs = (K + BK - 1) / BK;
  // a block's K is shared while the clusters stay resident in one wave and a
  // CTA keeps four k-blocks
  int share = 1;
  while (share < SK_MAX_SHARE && 2 * share * blocks <= sms && kbs >= 8 * share &&
         blocks <= resident_clusters(kern, 2 * share))
    share *= 2;
  Config k;
  k.grid = dim3(blocks, share);
  k.mp = sh.mp;
  // more blocks than SMs: two CTAs an SM, one filling its ring while the other
  // finishes
  k.stages = sk_stages(k.mp, blocks > sms && sk_sums_fit(k.mp, true));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  fill(cfg, attr, k, stream, pdl);
  return cudaLaunchKernelEx(&cfg, kern, map_w, map_x, bias, resid, ldr, rs, out, ldo, pre, M, N, K,
                            k.mp, k.stages, clear, no_work, status, limit_ns);
}

}  // namespace

SkinnyShape linear_skinny_shape(int M, int N, int K) {
  SkinnyShape s;
  s.tiles = (M + 255) / 256;
  s.mp = ((M + s.tiles - 1) / s.tiles + 15) / 16 * 16;
  s.tiles = (M + s.mp - 1) / s.mp;
  s.blocks = (N + SK_ROWS - 1) / SK_ROWS;
  const int units = s.blocks * s.tiles, kbs = (K + BK - 1) / BK;
  s.share = 1;  // (of 152 SMs; the launch asks how many clusters are resident)
  while (s.share < SK_MAX_SHARE && 2 * s.share * units <= 152 && kbs >= 8 * s.share) s.share *= 2;
  return s;
}

cudaError_t launch_linear_skinny(const CUtensorMap& map_w, const CUtensorMap& map_x,
                                 const void* bias, const void* resid, int ldr, float rs, void* out,
                                 int ldo, void* pre, int M, int N, int K, int act, bool w_mn,
                                 bool clear, int no_work, int* status, unsigned long long limit_ns,
                                 cudaStream_t stream, bool pdl) {
  if (M < 1) return cudaErrorInvalidValue;
  const bf *b = static_cast<const bf*>(bias), *r = static_cast<const bf*>(resid);
  bf *o = static_cast<bf*>(out), *z = static_cast<bf*>(pre);
#define MLP_SK(A, MN)                                                                         \
  launch<A, MN>(map_w, map_x, b, r, ldr, rs, o, ldo, z, M, N, K, clear, no_work, status, limit_ns, \
                stream, pdl)
  if (w_mn) return act == ACT_NONE ? MLP_SK(ACT_NONE, true) : cudaErrorInvalidValue;
  switch (act) {
    case ACT_SILU_EXP: return MLP_SK(ACT_SILU_EXP, false);
    case ACT_RELU_SQ: return MLP_SK(ACT_RELU_SQ, false);
    case ACT_GELU_EXP: return MLP_SK(ACT_GELU_EXP, false);
    case ACT_RELU: return MLP_SK(ACT_RELU, false);
    case ACT_SIGMOID_EXP: return MLP_SK(ACT_SIGMOID_EXP, false);
    default: return MLP_SK(ACT_NONE, false);
  }
#undef MLP_SK
}

}  // namespace mlpk
