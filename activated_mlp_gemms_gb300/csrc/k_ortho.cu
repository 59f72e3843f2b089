// The orthogonalised update (mlp_ortho.h): the norm of G, X = G / (|G| + eps), and the
// products of a Newton-Schulz step,
//   A = X X^T,  P = b A + c A A,  X <- a X + P X,
// on the tensor cores.
//
// Arithmetic.  The iteration stretches small singular values by up to a = 3.4 a step, and
// with them the rounding of X: in bf16 terms alone five steps leave 1-30 % of error.  Here X is
// the sum of two fp16 terms (22 bits), so that a X carries no rounding; the products take the
// leading terms (11 bits, the same speed as bf16), whose errors the contraction of the other
// singular values damps: 0.2-2.4e-3 of the result beside the 1.7e-3 of rounding it to bf16, the
// most where the smallest singular values are a tenth of the largest (up to 128 rows P X takes both
// terms: 1.1e-3 at most).  An fp32 result takes hi lo + lo hi + hi hi (1e-5 and below).
//
// The GEMM: one CTA of 320 threads an SM; CTA pairs with 256 x 256 tiles (tcgen05
// cta_group::2), or single CTAs with 128 x 128 tiles where those are too few.
//   warp 0     TMA loads of both operands' 64-wide k-blocks into a ring of five 32 KB stages
//   warp 1     issues tcgen05.mma into one of two accumulators; in a pair's other CTA it
//              tells the leader that the accumulator has been read
//   warps 2-9  read the accumulator (a row a thread) 32 columns at a time, add `in`, round and
//              store; `in` and what is stored pass through 32 x 32 boxes in shared memory, two
//              sets a warp, that TMA fills ahead of the accumulator and empties behind it
//              (sixteen warps with a set each were no faster: 16 x 1408 x 2048 step 122 us, 118
//              so; a unit's k-blocks draw 12 TB/s of L2, and that is what `in` and D wait for)
// The tensor cores truncate their accumulator at every instruction, by about half of its last bit:
// over a long K an fp32 result would lose a digit by it (4864: 3e-5, now 5e-6).  With both
// terms the leading products therefore come in chunks of g.chunk k-blocks, whose sums the
// epilogue's warps add up in fp32, rounded to nearest, in registers.
// With SPLIT a unit of a symmetric product has a cluster of two pairs, each with half of its
// k-blocks: a pair keeps half of the tile's columns, leaves its sums of the others in its shared
// memory over the ring, and adds to its own the other pair's, read from there strip by strip.
// The units are dealt in turn (unit u to cluster u mod clusters): all cost the same.  Of a
// symmetric product only the tiles on and below the diagonal are formed, and stored twice.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "gemm_params.h"
#include "ortho.cuh"
#include "ortho.h"
#include "ptx.cuh"

namespace mlpk {

namespace {

constexpr int OSTAGES = 5;
constexpr int OPERAND = 128 * 64 * 2;  // bytes of an operand's k-block in one CTA
constexpr int OSTAGE = 2 * OPERAND;
constexpr int EPI_WARPS = 8;  // two a TMEM lane quadrant
constexpr int OTHREADS = 64 + 32 * EPI_WARPS;
constexpr int BOX = 2048;                              // 32 x 32 fp16 or bf16
constexpr int SET = 2 * BOX;                           // two terms, or a box and its mirror image
constexpr int OSTAGING = EPI_WARPS * 2 * SET;
constexpr int OSMEM = OSTAGES * OSTAGE + OSTAGING + 1024 + 512;  // ... alignment, control block

// kind::f16 with fp16 operands (format 0), fp32 accumulators, M = N = TILE.
template <int TILE, bool Q_MN>
constexpr uint32_t IDESC_FP16 = (1u << 4) | ((Q_MN ? 1u : 0u) << 16) |
                                (static_cast<uint32_t>(TILE >> 3) << 17) |
                                (static_cast<uint32_t>(TILE >> 4) << 24);

// Chunks of a unit's k-blocks, and where chunk c ends: the small products (hi lo, lo hi) belong
// to the first.
__device__ __forceinline__ int chunks_of(const OrthoGemm& g, int kblocks) {
  return (kblocks + g.chunk - 1) / g.chunk;
}
__device__ __forceinline__ int chunk_end(const OrthoGemm& g, int kblocks, int c) {
  const int end = 2 * kblocks + (c + 1) * g.chunk;
  return end < 3 * kblocks ? end : 3 * kblocks;
}

struct Tile {
  int b, tm, tn;
};
template <int KIND>
__device__ __forceinline__ Tile tile_of(const OrthoGemm& g, int unit) {
  Tile t;
  const int per = g.units / g.batch;
  const int b = unit / per, u = unit - b * per;
  t.b = g.backwards ? g.batch - 1 - b : b;
  if (KIND == ORTHO_SYM) {  // row tm of the triangle begins at tm (tm + 1) / 2
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

// Row r of a 32 x 32 box of 2-byte values: 64 bytes, the 16-byte parts swizzled (64-byte
// swizzle), so that a row a thread passes without bank conflicts.
__device__ __forceinline__ uint32_t part16(uint32_t box, int r, int j) {
  return box + static_cast<uint32_t>(r * 64 + ((j ^ (r >> 1 & 3)) << 4));
}
// The same of a box of 4-byte values: 128 bytes, 128-byte swizzle.
__device__ __forceinline__ uint32_t part32(uint32_t box, int r, int j) {
  return box + static_cast<uint32_t>(r * 128 + ((j ^ (r & 7)) << 4));
}
__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(static_cast<uint16_t>(v)) : "memory");
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// The thread's row of 32 packed values, as it is or as column `lane` of the box.
__device__ __forceinline__ void put16(uint32_t box, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    st_shared_v4(part16(box, lane, j), w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}
__device__ __forceinline__ void put16_across(uint32_t box, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    st_shared_u16(part16(box, i, lane >> 3) + static_cast<uint32_t>((lane & 7) * 2),
                  i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
}
// Adds a row of fp16 values, times alpha.
__device__ __forceinline__ void add16(uint32_t box, int lane, float alpha, float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 q = ld_shared_v4(part16(box, lane, j));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack_half2(w[i]);
      v[8 * j + 2 * i] += alpha * x.x;
      v[8 * j + 2 * i + 1] += alpha * x.y;
    }
  }
}
// v as fp16, and what that leaves of it in v.
__device__ __forceinline__ void take_term(float (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    w[i] = pack_half2(v[2 * i], v[2 * i + 1]);
    const float2 x = unpack_half2(w[i]);
    v[2 * i] -= x.x;
    v[2 * i + 1] -= x.y;
  }
}

template <int CG, int KIND, bool TWO, bool SPLIT>
__global__ void __launch_bounds__(OTHREADS, 1) k_ortho_gemm(const __grid_constant__ OrthoGemm g) {
  extern __shared__ uint8_t ortho_smem[];
  constexpr bool PAIR = CG == 2;
  static_assert(PAIR || !SPLIT, "pairs share K");
  constexpr bool Q_MN = KIND != ORTHO_SYM;
  constexpr int TILE = 128 * CG;  // rows and columns of a tile
  constexpr uint32_t IDESC = IDESC_FP16<TILE, Q_MN>;
  constexpr uint32_t COLS = 2 * TILE;  // two accumulators
  const uint32_t base = (smem_u32(ortho_smem) + 1023u) & ~1023u;
  uint8_t* ctrl = ortho_smem + (base - smem_u32(ortho_smem)) + OSTAGES * OSTAGE + OSTAGING;
  uint64_t* bar = reinterpret_cast<uint64_t*>(ctrl);
  constexpr int FULL = 0, EMPTY = OSTAGES, TFULL = 2 * OSTAGES, TEMPTY = TFULL + 2,
                DRAIN = TEMPTY + 2, IN = DRAIN + 1, NBAR = IN + 2 * EPI_WARPS;
  static_assert(8 * NBAR + 8 <= 512, "control block");
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(ctrl + 8 * NBAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_s + 1);
  auto bar_s = [&](int i) { return smem_u32(bar + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t in_cluster = PAIR ? cluster_ctarank() : 0u;
  // the CTA of its pair, and which pair
  const uint32_t rank = SPLIT ? in_cluster & 1u : in_cluster, pair = SPLIT ? in_cluster >> 1 : 0u;
  const bool leader = rank == 0;
  auto lead = [&](uint32_t local) { return PAIR ? mapa_shared(local, 2 * pair) : local; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < OSTAGES; ++i) {
      mbar_init(bar_s(FULL + i), 1);
      mbar_init(bar_s(EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_s(TFULL + i), 1);
      // the epilogue warps; the leader's also: the other CTA's
      mbar_init(bar_s(TEMPTY + i), EPI_WARPS + (PAIR && leader ? 1 : 0));
    }
    mbar_init(bar_s(DRAIN), 1);
    for (int i = 0; i < 2 * EPI_WARPS; ++i) mbar_init(bar_s(IN + i), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&g.p);
    prefetch_tmap(&g.q);
    prefetch_tmap(&g.in);
    prefetch_tmap(&g.d);
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
  constexpr int CTAS = SPLIT ? 2 * CG : CG;  // of a unit
  const int first = static_cast<int>(blockIdx.x) / CTAS, step = static_cast<int>(gridDim.x) / CTAS;
  constexpr int segs = TWO ? 3 : 1;
  // this pair's k-blocks
  const int half = (g.kblocks + 1) / 2;
  const int kb0 = pair ? half : 0;
  const int kb_len = !SPLIT ? g.kblocks : pair ? g.kblocks - half : half;
  const int kb_all = kb_len * segs;
  const int chunks = TWO ? chunks_of(g, kb_len) : 1;
  int acc = 0;  // of the next chunk (or unit), in its readers and its writer alike
  uint32_t aphase = 0;
  auto next_acc = [&] {
    acc ^= 1;
    if (acc == 0) aphase ^= 1u;
  };
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
        const Tile t = tile_of<KIND>(g, unit);
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
          const int k0 = (kb0 + kb) * 64;
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
          if (++kb == kb_len) { kb = 0; ++seg; }
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
    const uint16_t both = static_cast<uint16_t>(3u << (2 * pair));  // CTAs of the pair
    if (lane == 0 && leader) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true, any = false;
      for (int unit = first; ok && unit < g.units; unit += step) {
        int i = 0;
        for (int c = 0; ok && c < chunks; ++c) {
          ok = mbar_wait<PAIR>(bar_s(TEMPTY + acc), aphase ^ 1u, lim, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + acc * TILE;
          const int begin = i;
          for (const int end = TWO ? chunk_end(g, kb_len, c) : kb_all; i < end; ++i) {
            ok = mbar_wait<PAIR>(bar_s(FULL + stage), phase, lim, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sp = base + stage * OSTAGE, sq = sp + OPERAND;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint64_t pd = sdesc_sw128(sp + k * 32, 16, 1024);
              const uint64_t qd = Q_MN ? sdesc_sw128(sq + k * 2048, 8192, 1024)
                                       : sdesc_sw128(sq + k * 32, 16, 1024);
              if constexpr (PAIR) tc_mma_bf16_pair(d, pd, qd, IDESC, i > begin || k > 0);
              else tc_mma_bf16(d, pd, qd, IDESC, i > begin || k > 0);
            }
            any = true;
            if constexpr (PAIR) tc_commit_pair(bar_s(EMPTY + stage), both);
            else tc_commit(bar_s(EMPTY + stage));
            if (++stage == OSTAGES) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          if constexpr (PAIR) tc_commit_pair(bar_s(TFULL + acc), both);
          else tc_commit(bar_s(TFULL + acc));
          next_acc();
        }
      }
      if (!ok) {
        failed();
        if (any) {  // the MMAs already issued end before TMEM is freed
          if constexpr (PAIR) tc_commit_pair(bar_s(DRAIN), both & 0x5);
          else tc_commit(bar_s(DRAIN));
          volatile int never = 0;
          mbar_wait<PAIR>(bar_s(DRAIN), 0, 10000000ull, &never);
        }
      }
    } else if (PAIR && lane == 0) {
      // tells the leader that this CTA's warps have read an accumulator: one release at
      // cluster scope, from a thread that has no stores of its own to wait for
      bool ok = true;
      for (int unit = first; ok && unit < g.units; unit += step)
        for (int c = 0; ok && c < (SPLIT ? chunks - 1 : chunks); ++c) {  // (no unit follows)
          ok = mbar_wait(bar_s(TEMPTY + acc), aphase, lim, abort_flag);
          if (!ok) break;
          tc_fence_after();
          tc_fence_before();
          mbar_arrive_cluster(lead(bar_s(TEMPTY + acc)));
          next_acc();
        }
      if (!ok) failed();
    }
  } else {
    constexpr int WIDTH = TILE / (EPI_WARPS / 4);  // a warp's columns of the tile
    const int q = warp & 3, part = (warp - 2) >> 2;
    const uint32_t stg = base + OSTAGES * OSTAGE + static_cast<uint32_t>(warp - 2) * 2 * SET;
    const uint32_t in_bar = bar_s(IN + 2 * (warp - 2));
    const uint64_t pol = policy_evict_normal();
    fence_proxy_async_global();
    const bool two_terms = KIND == ORTHO_STEP || (KIND == ORTHO_SYM && g.d_terms == 2);
    constexpr bool two_in = KIND != ORTHO_SYM || TWO;
    const bool has_in = g.alpha != 0.f;
    uint32_t in_phase = 0;  // a bit a set
    uint32_t loading = 0;   // sets with a load in flight
    const uint32_t my_lanes = (static_cast<uint32_t>(q * 32) << 16) +
                              static_cast<uint32_t>(part * WIDTH);
    for (int unit = first; unit < g.units; unit += step) {
      const Tile t = tile_of<KIND>(g, unit);
      const int row0 = t.tm * TILE + static_cast<int>(rank) * 128 + q * 32;
      const int col0 = t.tn * TILE + part * WIDTH;
      const bool mirror = KIND == ORTHO_SYM && t.tm != t.tn;
      // strips of 32 columns inside the output
      int strips = row0 < g.M ? (g.N - col0 + 31) / 32 : 0;
      strips = strips < 0 ? 0 : strips < WIDTH / 32 ? strips : WIDTH / 32;
      if (SPLIT && part != static_cast<int>(pair)) strips = 0;  // the other pair's columns
      // `in` of strip c into set c & 1, once what that held has been stored
      auto load = [&](int c) {
        const int s = c & 1;
        if (lane == 0) {
          const uint32_t bar_in = in_bar + 8 * s, box = stg + s * SET;
          mbar_expect_tx(bar_in, two_in ? 2 * BOX : BOX);
          tma_load_3d(box, &g.in, col0 + 32 * c, row0, t.b, bar_in, pol);
          if (two_in) tma_load_3d(box + BOX, &g.in, col0 + 32 * c, row0, g.batch + t.b, bar_in, pol);
        }
        loading |= 1u << s;
      };
      if (lane == 0) bulk_wait_read_all();
      __syncwarp();
      if (has_in) {
        if (strips > 0) load(0);
        if (strips > 1) load(1);
      }
      bool ok = true;
      uint32_t tb = tmem + my_lanes + acc * TILE;
      if (!TWO || chunks == 1) {
        ok = mbar_wait<PAIR>(bar_s(TFULL + acc), aphase, lim, abort_flag);
        tc_fence_after();
      } else {  // the chunks' sums, in registers; then over the last accumulator
        float sum[WIDTH];
#pragma unroll
        for (int i = 0; i < WIDTH; ++i) sum[i] = 0.f;
        for (int c = 0; c < chunks; ++c) {
          ok = mbar_wait<PAIR>(bar_s(TFULL + acc), aphase, lim, abort_flag);
          if (!ok) break;
          tc_fence_after();
          __syncwarp();
          tb = tmem + my_lanes + acc * TILE;
#pragma unroll
          for (int col = 0; col < WIDTH; col += 32) {
            uint32_t a[32];
            tmem_ld32(tb + col, a);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[col + i] += __uint_as_float(a[i]);
          }
          if (c + 1 < chunks) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_s(TEMPTY + acc));
            next_acc();
          }
        }
        if (ok) {
#pragma unroll
          for (int col = 0; col < WIDTH; col += 32) {
            uint32_t a[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) a[i] = __float_as_uint(sum[col + i]);
            tmem_st32(tb + col, a);
          }
          tmem_wait_st();
        }
      }
      if constexpr (SPLIT) {  // (the ring is free: the pair's last MMA is done)
        if (ok && part != static_cast<int>(pair)) {
#pragma unroll 1
          for (int col = 0; col < WIDTH; col += 32) {
            uint32_t a[32];
            __syncwarp();
            tmem_ld32(tb + col, a);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              st_shared_v4(sum_part(base, q * 32 + lane, col / 4 + j), a[4 * j], a[4 * j + 1],
                           a[4 * j + 2], a[4 * j + 3]);
          }
        }
        __syncwarp();
        cluster_sync();
      }
      if (!ok) {
        failed();
        break;
      }
#pragma unroll 1
      for (int c = 0; c < strips; ++c) {
        const int s = c & 1, col = col0 + 32 * c;
        const uint32_t box = stg + s * SET;
        float v[32];
        {
          uint32_t a[32];
          __syncwarp();
          tmem_ld32(tb + 32 * c, a);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(a[i]);
        }
        if constexpr (SPLIT) {  // the other pair's sums of these columns
          float4 o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            o[j] = ld_cluster_f4(mapa_shared(sum_part(base, q * 32 + lane, 8 * c + j), in_cluster ^ 2u));
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            v[4 * j] += o[j].x, v[4 * j + 1] += o[j].y;
            v[4 * j + 2] += o[j].z, v[4 * j + 3] += o[j].w;
          }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= g.beta;
        if (has_in) {
          if (!mbar_wait(in_bar + 8 * s, in_phase >> s & 1u, lim, abort_flag)) {
            ok = false;
            break;
          }
          in_phase ^= 1u << s;
          loading &= ~(1u << s);
          if (two_in) add16(box + BOX, lane, g.alpha, v);
          add16(box, lane, g.alpha, v);
        } else if (lane == 0) {  // the set's last store has read it
          if (KIND == ORTHO_SYM && two_terms) bulk_wait_read_all();
          else asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        }
        __syncwarp();  // (the rows are read before another thread's column goes over them)
        if constexpr (KIND == ORTHO_LAST) {
          if (g.out_bf16) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            if (g.transposed) put16_across(box, lane, w);
            else put16(box, lane, w);
          } else if (g.transposed) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              st_shared_u32(part32(box, i, lane >> 2) + static_cast<uint32_t>((lane & 3) * 4),
                            __float_as_uint(v[i]));
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              st_shared_v4(part32(box, lane, j), __float_as_uint(v[4 * j]),
                           __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                           __float_as_uint(v[4 * j + 3]));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (g.transposed) tma_store_3d(&g.d, box, row0, col, t.b);
            else tma_store_3d(&g.d, box, col, row0, t.b);
            bulk_commit();
          }
        } else if constexpr (KIND == ORTHO_STEP) {
          uint32_t w[16];
          take_term(v, w);
          put16(box, lane, w);
          take_term(v, w);
          put16(box + BOX, lane, w);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&g.d, box, col, row0, t.b);
            tma_store_3d(&g.d, box + BOX, col, row0, g.batch + t.b);
            bulk_commit();
          }
        } else {
          // a term and its mirror image at a time
#pragma unroll 1
          for (int z = t.b; z < (two_terms ? 2 : 1) * g.batch; z += g.batch) {
            uint32_t w[16];
            take_term(v, w);
            if (z != t.b) {
              if (lane == 0) bulk_wait_read_all();
              __syncwarp();
            }
            put16(box, lane, w);
            if (mirror) put16_across(box + BOX, lane, w);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&g.d, box, col, row0, z);
              if (mirror) tma_store_3d(&g.d, box + BOX, row0, col, z);
              bulk_commit();
            }
          }
        }
        if (has_in && c + 2 < strips) {
          if (lane == 0) bulk_wait_read_all();
          __syncwarp();
          load(c + 2);
        }
      }
      if (!ok) {
        failed();
        break;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_s(TEMPTY + acc));
      next_acc();
    }
    // what is in flight ends before shared memory is released
    for (int s = 0; s < 2; ++s)
      if (loading >> s & 1u) {
        volatile int never = 0;
        mbar_wait(in_bar + 8 * s, in_phase >> s & 1u, 10000000ull, &never);
      }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  if constexpr (SPLIT) {
    if (warp < 2) {  // (the epilogue's barrier)
      __syncwarp();
      cluster_sync();
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

// Few units with a long K: a cluster of CTAs shares a 128 x 128 tile's k-blocks.  Each leaves
// its fp32 sums in its shared memory; then each adds up its share of the rows over the
// cluster's memories, in the CTAs' order, and finishes them.  With both terms the leading
// products come in parts, as the chunks above, each in the next of four accumulators, which the
// epilogue's warps add up in registers.
constexpr int SPLIT_STAGES = 6;
constexpr int SPLIT_SMEM = SPLIT_STAGES * OSTAGE + 1024 + 256;

// Stores the terms of eight consecutive values (of D, or of its mirror image).
__device__ __forceinline__ void store_terms(const OrthoGemm& g, size_t at, size_t term, bool two,
                                            const float (&f)[8]) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack_half2(f[2 * i], f[2 * i + 1]);
    const float2 x = unpack_half2(h[i]);
    l[i] = pack_half2(f[2 * i] - x.x, f[2 * i + 1] - x.y);
  }
  __half* d = static_cast<__half*>(g.d_ptr) + at;
  st_global_v4(d, make_uint4(h[0], h[1], h[2], h[3]));
  if (two) st_global_v4(d + term, make_uint4(l[0], l[1], l[2], l[3]));
}
__device__ __forceinline__ void store_out(const OrthoGemm& g, size_t at, const float (&f)[8]) {
  if (g.out_bf16) {
    st_global_v4(static_cast<__nv_bfloat16*>(g.d_ptr) + at,
                 make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                            pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])));
  } else {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(g.d_ptr) + at);
    o[0] = make_float4(f[0], f[1], f[2], f[3]);
    o[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

template <int KIND>
__global__ void __launch_bounds__(OTHREADS, 1) k_ortho_split(const __grid_constant__ OrthoGemm g) {
  extern __shared__ uint8_t ortho_smem[];
  constexpr bool Q_MN = KIND != ORTHO_SYM;
  constexpr uint32_t IDESC = IDESC_FP16<128, Q_MN>;
  const uint32_t base = (smem_u32(ortho_smem) + 1023u) & ~1023u;
  uint8_t* base_g = ortho_smem + (base - smem_u32(ortho_smem));
  uint8_t* ctrl = base_g + SPLIT_STAGES * OSTAGE;
  uint64_t* bar = reinterpret_cast<uint64_t*>(ctrl);
  constexpr int FULL = 0, EMPTY = SPLIT_STAGES, DONE = 2 * SPLIT_STAGES, FREE = DONE + 4,
                DRAIN = FREE + 4, NBAR = DRAIN + 1;
  static_assert(8 * NBAR + 8 <= 256, "control block");
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(ctrl + 8 * NBAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_s + 1);
  auto bar_s = [&](int i) { return smem_u32(bar + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_ctarank());

  if (threadIdx.x == 0) {
    for (int i = 0; i < SPLIT_STAGES; ++i) {
      mbar_init(bar_s(FULL + i), 1);
      mbar_init(bar_s(EMPTY + i), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar_s(DONE + i), 1);
      mbar_init(bar_s(FREE + i), EPI_WARPS);
    }
    mbar_init(bar_s(DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&g.p);
    prefetch_tmap(&g.q);
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_u32(tmem_s), 512);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_s;
  pdl_wait();
  pdl_launch_dependents();

  const uint64_t lim = g.timeout_ns;
  const Tile t = tile_of<KIND>(g, static_cast<int>(blockIdx.x) / S);
  const int m0 = t.tm * 128, n0 = t.tn * 128;
  const int segs = g.terms == 2 ? 3 : 1;
  // a CTA's slice of K, for all of the products (the last CTAs may have none)
  const int per = (g.kblocks + S - 1) / S;
  const int slice0 = rank * per < g.kblocks ? rank * per : g.kblocks;
  const int slice1 = slice0 + per < g.kblocks ? slice0 + per : g.kblocks;
  const int len = slice1 - slice0, mine = len * segs;
  const int parts = len == 0 ? 0 : segs == 1 ? 1 : chunks_of(g, len);
  auto part_end = [&](int i) { return segs == 1 ? mine : chunk_end(g, len, i); };
  auto failed = [&] {
    *abort_flag = 1;
    atomicExch(g.status, O_TIMEOUT);
  };

  if (warp == 0) {
    if (lane == 0 && !(g.debug_flags & 1)) {
      fence_proxy_async_global();
      const uint64_t pol = policy_evict_normal();
      int seg = 0, kb = slice0;
      for (int n = 0; n < mine; ++n) {
        const int stage = n % SPLIT_STAGES;
        if (!mbar_wait(bar_s(EMPTY + stage), (n / SPLIT_STAGES + 1) & 1, lim, abort_flag)) {
          failed();
          for (int j = n - SPLIT_STAGES; j < n; ++j) {  // copies in flight land first
            volatile int never = 0;
            if (j >= 0)
              mbar_wait(bar_s(FULL + j % SPLIT_STAGES), j / SPLIT_STAGES & 1, 10000000ull, &never);
          }
          break;
        }
        const uint32_t full = bar_s(FULL + stage), s = base + stage * OSTAGE;
        mbar_expect_tx(full, OSTAGE);
        const int k0 = kb * 64;
        const int zp = t.b + (segs == 3 && seg == 1 ? g.batch : 0);
        const int zq = t.b + (segs == 3 && seg == 0 ? g.batch : 0);
        tma_load_3d(s, &g.p, k0, m0, zp, full, pol);
        if constexpr (Q_MN) {
          tma_load_3d(s + OPERAND, &g.q, n0, k0, zq, full, pol);
          tma_load_3d(s + OPERAND + OPERAND / 2, &g.q, n0 + 64, k0, zq, full, pol);
        } else {
          tma_load_3d(s + OPERAND, &g.q, k0, n0, zq, full, pol);
        }
        if (++kb == slice1) { kb = slice0; ++seg; }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      bool ok = true;
      int n = 0;
      for (int i = 0; ok && i < parts; ++i) {
        const int acc = i % 4, begin = n;
        if (i >= 4) ok = mbar_wait(bar_s(FREE + acc), (i / 4 + 1) & 1, lim, abort_flag);
        for (const int end = part_end(i); ok && n < end; ++n) {
          const int stage = n % SPLIT_STAGES;
          ok = mbar_wait(bar_s(FULL + stage), n / SPLIT_STAGES & 1, lim, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sp = base + stage * OSTAGE, sq = sp + OPERAND;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t pd = sdesc_sw128(sp + k * 32, 16, 1024);
            const uint64_t qd =
                Q_MN ? sdesc_sw128(sq + k * 2048, 8192, 1024) : sdesc_sw128(sq + k * 32, 16, 1024);
            tc_mma_bf16(tmem + acc * 128, pd, qd, IDESC, n > begin || k > 0);
          }
          tc_commit(bar_s(EMPTY + stage));
        }
        if (ok) tc_commit(bar_s(DONE + acc));
      }
      if (!ok) {
        failed();
        tc_commit(bar_s(DRAIN));
        volatile int never = 0;  // what was issued ends before TMEM is freed
        mbar_wait(bar_s(DRAIN), 0, 10000000ull, &never);
      }
    }
  }
  __syncwarp();
  // the sums to shared memory, over the ring (every load has been read when the MMAs are done)
  bool ok = true;
  if (warp >= 2 && parts > 0) {
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t from = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * 64;
    float sum[64];
    for (int i = 0; ok && i < parts; ++i) {
      ok = mbar_wait(bar_s(DONE + i % 4), i / 4 & 1, lim, abort_flag);
      if (!ok) break;
      __syncwarp();
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        uint32_t a[32];
        tmem_ld32(from + (i % 4) * 128 + c, a);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j)
          sum[c + j] = i ? sum[c + j] + __uint_as_float(a[j]) : __uint_as_float(a[j]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_s(FREE + i % 4));
    }
    if (!ok) failed();
    if (ok) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        st_shared_v4(sum_part(base, q * 32 + lane, half * 16 + j), __float_as_uint(sum[4 * j]),
                     __float_as_uint(sum[4 * j + 1]), __float_as_uint(sum[4 * j + 2]),
                     __float_as_uint(sum[4 * j + 3]));
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();
  // my rows
  const int R = 128 / S, busy = (g.kblocks + per - 1) / per;  // CTAs that had k-blocks
  const int first_row = m0 + rank * R;
  const size_t in_mat = static_cast<size_t>(g.M) * g.ld_in, d_mat = static_cast<size_t>(g.M) * g.ld_d;
  const size_t term = d_mat * g.batch;  // (of D in terms)
  const bool mirror = KIND == ORTHO_SYM && t.tm != t.tn;
  const bool across = mirror || (KIND == ORTHO_LAST && g.transposed);
  const bool two_terms = KIND == ORTHO_STEP || (KIND == ORTHO_SYM && g.d_terms == 2);
  const bool two_in = KIND != ORTHO_SYM || g.terms == 2;
  const int pitch = R + 4;  // of the rows turned to columns, in floats
  float* turned = reinterpret_cast<float*>(base_g + 65536);
  if (warp >= 2) {
    // half a warp a row: 16 lanes of eight columns
    const int c8 = (lane & 15) * 8, col = n0 + c8;
    for (int i = (warp - 2) * 2 + (lane >> 4); i < R; i += 16) {
      const int row = first_row + i, r = rank * R + i;
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = 0.f;
      const uint32_t x = sum_part(base, r, c8 / 4), y = sum_part(base, r, c8 / 4 + 1);
      switch (busy) {
        case 8: cluster_sums<8>(x, y, f); break;
        case 7: cluster_sums<7>(x, y, f); break;
        case 6: cluster_sums<6>(x, y, f); break;
        case 5: cluster_sums<5>(x, y, f); break;
        case 4: cluster_sums<4>(x, y, f); break;
        case 3: cluster_sums<3>(x, y, f); break;
        case 2: cluster_sums<2>(x, y, f); break;
        default: cluster_sums<1>(x, y, f);
      }
      const bool in_d = row < g.M && col < g.N;
      const size_t at = t.b * d_mat + static_cast<size_t>(row) * g.ld_d + col;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= g.beta;
      if (in_d && g.alpha != 0.f) {
        const __half* x = static_cast<const __half*>(g.in_ptr) + t.b * in_mat +
                          static_cast<size_t>(row) * g.ld_in + col;
        for (int z = two_in ? 1 : 0; z >= 0; --z) {
          const uint4 h = ld_global_v4(x + z * (in_mat * g.batch));
          const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 y = unpack_half2(w[j]);
            f[2 * j] += g.alpha * y.x;
            f[2 * j + 1] += g.alpha * y.y;
          }
        }
      }
      if (across) {
#pragma unroll
        for (int j = 0; j < 8; ++j) turned[(c8 + j) * pitch + i] = f[j];
      }
      if (in_d && ok) {
        if constexpr (KIND == ORTHO_LAST) {
          if (!g.transposed) store_out(g, at, f);
        } else {
          store_terms(g, at, term, two_terms, f);
        }
      }
    }
  }
  if (across) {  // (the same in all of the CTA's threads)
    __syncthreads();
    for (int i = threadIdx.x; i < 128 * (R / 8); i += OTHREADS) {
      const int c = i / (R / 8), r8 = i % (R / 8) * 8;
      if (!ok || n0 + c >= g.N || first_row + r8 >= g.M) continue;
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = turned[c * pitch + r8 + j];
      const size_t at =
          static_cast<size_t>(t.b) * g.N * g.ld_d + static_cast<size_t>(n0 + c) * g.ld_d + first_row + r8;
      if constexpr (KIND == ORTHO_LAST) store_out(g, at, f);
      else store_terms(g, at, term, two_terms, f);
    }
  }
  __syncwarp();
  cluster_sync();  // my sums have been read
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, 512);
  }
}

template <int KIND>
cudaError_t launch_split(const OrthoGemm& g, int share, cudaStream_t stream) {
  auto kern = k_ortho_split<KIND>;
  static std::atomic<unsigned long long> done{0};  // devices that have the attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(done.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SPLIT_SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) done.fetch_or(1ull << dev);
  }
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = ortho_config(share, g.units * share, stream, attr);
  cfg.dynamicSmemBytes = SPLIT_SMEM;
  return cudaLaunchKernelEx(&cfg, kern, g);
}

template <int CG, int KIND, bool TWO, bool SPLIT = false>
cudaError_t prepare() {
  auto kern = k_ortho_gemm<CG, KIND, TWO, SPLIT>;
  static std::atomic<unsigned long long> done{0};  // devices that have the attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load() >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, OSMEM);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev);
  return e;
}

template <int CG, int KIND, bool TWO, bool SPLIT = false>
int clusters() {
  constexpr int CTAS = SPLIT ? 2 * CG : CG;
  int dev = 0, sms = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  static std::atomic<int> cache[64];
  if (dev < 64 && cache[dev].load() > 0) return cache[dev].load();
  if (prepare<CG, KIND, TWO, SPLIT>() != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = ortho_config(CTAS, sms / CTAS * CTAS, nullptr, attr);
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, k_ortho_gemm<CG, KIND, TWO, SPLIT>, &cfg) != cudaSuccess) return 0;
  if (dev < 64) cache[dev].store(n);
  return n;
}

template <int CG, int KIND, bool TWO, bool SPLIT = false>
cudaError_t launch_of(const OrthoGemm& g, cudaStream_t stream) {
  const cudaError_t e = prepare<CG, KIND, TWO, SPLIT>();
  if (e != cudaSuccess) return e;
  const int n = clusters<CG, KIND, TWO, SPLIT>();
  if (n <= 0) return cudaErrorUnknown;
  cudaLaunchAttribute attr[2];
  constexpr int CTAS = SPLIT ? 2 * CG : CG;
  const int grid = SPLIT || g.units < n ? g.units : n;  // (split: a unit a cluster)
  cudaLaunchConfig_t cfg = ortho_config(CTAS, CTAS * grid, stream, attr);
  return cudaLaunchKernelEx(&cfg, k_ortho_gemm<CG, KIND, TWO, SPLIT>, g);
}

// ------------------------------------------------------------- norm and scale
constexpr int NORM_THREADS = 512;

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
    k_ortho_scale(const T* __restrict__ G, int rows, int cols, int batch, int pitch,
                  const float* __restrict__ part, float eps, __half* __restrict__ X) {
  __shared__ float tile[64][65];
  __shared__ float factor_s;
  pdl_wait();
  pdl_launch_dependents();
  // (from the end, which the norm's reads have left in L2)
  const int b = static_cast<int>(gridDim.z - 1 - blockIdx.z);
  if (threadIdx.x < 32) {
    const float* p = part + b * ORTHO_PARTS;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < ORTHO_PARTS / 32; ++i) s += p[threadIdx.x + 32 * i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x == 0) factor_s = ORTHO_X / (sqrtf(s) + eps);
  }
  const T* M = G + b * (static_cast<size_t>(rows) * cols);
  const size_t size = static_cast<size_t>(rows < cols ? rows : cols) * pitch;
  __half* hi = X + b * size;
  __half* lo = hi + static_cast<size_t>(batch) * size;
  const int r0 = static_cast<int>(gridDim.y - 1 - blockIdx.y) * 64, c0 = static_cast<int>(blockIdx.x) * 64;
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
        put(static_cast<size_t>(r0 + r) * pitch + c0 + c, f);
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
      put(static_cast<size_t>(c0 + c) * pitch + r0 + r, f);
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

cudaError_t launch_ortho_gemm(const OrthoGemm& g, int cg, OrthoKind kind, cudaStream_t stream) {
  auto of = [&](auto k) {
    constexpr int KIND = decltype(k)::value;
    if (g.terms == 2)
      return cg == 2 ? launch_of<2, KIND, true>(g, stream) : launch_of<1, KIND, true>(g, stream);
    return cg == 2 ? launch_of<2, KIND, false>(g, stream) : launch_of<1, KIND, false>(g, stream);
  };
  switch (kind) {
    case ORTHO_SYM: return of(std::integral_constant<int, ORTHO_SYM>{});
    case ORTHO_STEP: return of(std::integral_constant<int, ORTHO_STEP>{});
    default: return of(std::integral_constant<int, ORTHO_LAST>{});
  }
}

cudaError_t launch_ortho_pairs(const OrthoGemm& g, cudaStream_t stream) {
  return g.terms == 2 ? launch_of<2, ORTHO_SYM, true, true>(g, stream)
                      : launch_of<2, ORTHO_SYM, false, true>(g, stream);
}
int ortho_pairs_clusters() { return clusters<2, ORTHO_SYM, true, true>(); }

cudaError_t launch_ortho_split(const OrthoGemm& g, int share, OrthoKind kind, cudaStream_t stream) {
  switch (kind) {
    case ORTHO_SYM: return launch_split<ORTHO_SYM>(g, share, stream);
    case ORTHO_STEP: return launch_split<ORTHO_STEP>(g, share, stream);
    default: return launch_split<ORTHO_LAST>(g, share, stream);
  }
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

cudaError_t launch_ortho_scale(const void* G, bool bf16, int rows, int cols, int batch, int pitch,
                               const float* part, float eps, void* X, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg =
      plain_config(dim3((cols + 63) / 64, (rows + 63) / 64, batch), 256, stream, attr);
  if (bf16)
    return cudaLaunchKernelEx(&cfg, k_ortho_scale<__nv_bfloat16>,
                              static_cast<const __nv_bfloat16*>(G), rows, cols, batch, pitch, part,
                              eps, static_cast<__half*>(X));
  return cudaLaunchKernelEx(&cfg, k_ortho_scale<float>, static_cast<const float*>(G), rows, cols,
                            batch, pitch, part, eps, static_cast<__half*>(X));
}

}  // namespace mlpk
