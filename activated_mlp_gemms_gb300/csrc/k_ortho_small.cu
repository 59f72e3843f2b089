// The orthogonalised update (mlp_ortho.h) of matrices whose lesser side m is at most 128, in one
// launch: a cluster of up to eight CTAs a matrix, each with WIDTH columns of X in its shared
// memory, in two fp16 terms, from G to the result.  A step:
//   each CTA's share of A = X X^T over its own columns, in fp32 to its shared memory;
//   each adds up 128 / CTAs of A's rows over the cluster and hands them, as fp16, to all;
//   each forms P = b A + c A A for itself, and a X + P X of its columns.
// X is the K-major operand of the first product and the MN-major one of the last: the same
// 128-byte rows serve both.  (Arithmetic and scales as in k_ortho.cu.  P X takes both terms of
// both for a bf16 result, too: its operands make most of that result's error, 2.6e-3 of 64 x 512
// with the leading terms, now 1.8e-3, of which rounding it is 1.7e-3, for 29 -> 32 us.  An fp32
// result's leading products are summed two instructions at a time: 64 x 1024 1.9e-6 -> 0.9e-6 off,
// 43 -> 45 us, 128 x 1024 3.5e-6 -> 1.5e-6, 73 -> 76; products of fp32 0.9e-6 and 1.7e-6.)
// What bounds it is latency: three rounds of MMA, two cluster barriers and three passes over tensor
// memory a step, and the exchange of A's rows, whose shared-memory traffic between CTAs runs at
// some 10 bytes a cycle (so only the m x m that there are move).
// Measured: 64 x 512 32 us, 64 x 1024 33, 128 x 1024 58; 64 x 2048 (256 columns a CTA) 45, of them
// 8 a step, 39 without the second terms in P X; 128 x 2048 76.
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

constexpr int THREADS = 512;  // four warps a TMEM lane quadrant
constexpr int BLOCK = 128 * 128;       // bytes of 128 rows x 64 fp16 columns
constexpr int SUMS = 128 * 128 * 4;    // of the fp32 share of A; P lies over it

template <int WIDTH>
struct Smem {
  static constexpr int X = 0, TERM = WIDTH / 64 * BLOCK;  // X's first term, then its second
  static constexpr int A = X + 2 * TERM;                  // in one term (256 columns) or two
  static constexpr int A_TERM = 2 * BLOCK;
  static constexpr int P = A + (WIDTH == 128 ? 2 : 1) * A_TERM;
  static constexpr int CTRL = P + SUMS;
  static constexpr int BYTES = CTRL + 256 + 1024;  // control block, alignment
};

template <int N, bool B_MN>
constexpr uint32_t IDESC = (1u << 4) | ((B_MN ? 1u : 0u) << 16) |
                           (static_cast<uint32_t>(N >> 3) << 17) | (128u >> 4 << 24);

// Eight columns (c, a multiple of 8) of row r of an operand of 64-column blocks: 128-byte rows,
// 128-byte swizzle.
__device__ __forceinline__ uint32_t piece(uint32_t at, int r, int c) {
  return at + static_cast<uint32_t>((c >> 6) * BLOCK + r * 128 + (((c >> 3 & 7) ^ (r & 7)) << 4));
}
// Eight values as fp16, and what that leaves of them.
__device__ __forceinline__ uint4 take_term(float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = pack_half2(f[2 * i], f[2 * i + 1]);
    const float2 x = unpack_half2(w[i]);
    f[2 * i] -= x.x;
    f[2 * i + 1] -= x.y;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void add_term(uint4 q, float k, float (&f)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack_half2(w[i]);
    f[2 * i] += k * x.x;
    f[2 * i + 1] += k * x.y;
  }
}
__device__ __forceinline__ void put(uint32_t at, uint4 v) { st_shared_v4(at, v.x, v.y, v.z, v.w); }
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
// Plain stores before MMA reads, wherever in the cluster's shared memory.
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}

// PARTS: an fp32 result (128 columns a CTA).
template <int WIDTH, bool BF16, bool PARTS>
__global__ void __launch_bounds__(THREADS, 1) k_ortho_small(const OrthoSmall g) {
  using S = Smem<WIDTH>;
  using T = std::conditional_t<BF16, __nv_bfloat16, float>;  // of G
  extern __shared__ uint8_t small_smem[];
  const uint32_t base = (smem_u32(small_smem) + 1023u) & ~1023u;
  uint8_t* ctrl = small_smem + (base - smem_u32(small_smem)) + S::CTRL;
  const uint32_t bar = smem_u32(ctrl);
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(ctrl + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + 12);
  float* norm_s = reinterpret_cast<float*>(ctrl + 16);   // a CTA's sum of squares each
  const uint32_t drain = smem_u32(ctrl + 48);
  float* warps_s = reinterpret_cast<float*>(ctrl + 64);  // a warp's (16)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ctas = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_ctarank());
  const int b = static_cast<int>(blockIdx.x) / ctas;
  const int col0 = rank * WIDTH;  // of this CTA's columns
  const size_t first = static_cast<size_t>(b) * g.m * g.n;

  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc<1>(smem_u32(tmem_s), 512);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  cluster_sync();  // (every CTA is there, too)
  tc_fence_after();
  const uint32_t tmem = *tmem_s;
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && tid == 0) *g.status = 0;

  // G's columns, eight values at a time: f(row, column of this CTA's, values) with zeros outside.
  // Along X's rows, or along its columns where G holds X transposed.
  constexpr int EIGHTS = 128 * WIDTH / 8;
  auto eight = [&](int i, int& r, int& c, float (&f)[8]) {
    r = g.transposed ? i % 16 * 8 : i / (WIDTH / 8);
    c = g.transposed ? i / 16 : i % (WIDTH / 8) * 8;
    if (r < g.m && col0 + c < g.n) {
      load8(static_cast<const T*>(g.G) + first +
                (g.transposed ? static_cast<size_t>(col0 + c) * g.m + r
                              : static_cast<size_t>(r) * g.n + col0 + c),
            f);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = 0.f;
    }
  };
  float squares = 0.f;
#pragma unroll 4
  for (int i = tid; i < EIGHTS; i += THREADS) {
    int r, c;
    float f[8], t = 0.f;
    eight(i, r, c, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) t += f[j] * f[j];
    squares += t;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) squares += __shfl_xor_sync(0xffffffffu, squares, o);
  if (lane == 0) warps_s[warp] = squares;
  __syncthreads();
  if (tid < ctas) {
    float t = 0.f;
    for (int i = 0; i < THREADS / 32; ++i) t += warps_s[i];
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(
                     mapa_shared(smem_u32(norm_s + rank), static_cast<uint32_t>(tid))),
                 "f"(t)
                 : "memory");
  }
  __syncwarp();
  cluster_sync();
  float total = 0.f;
  for (int i = 0; i < ctas; ++i) total += norm_s[i];
  const float factor = ORTHO_X / (sqrtf(total) + g.eps);
#pragma unroll 4
  for (int i = tid; i < EIGHTS; i += THREADS) {
    int r, c;
    float f[8];
    eight(i, r, c, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= factor;
    const uint4 hi = take_term(f), lo = take_term(f);
    if (!g.transposed) {
      put(piece(base + S::X, r, c), hi);
      put(piece(base + S::X + S::TERM, r, c), lo);
    } else {  // eight rows of a column
      const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t at = piece(base + S::X, r + j, c & ~7) + (c & 7) * 2;
        const int sh = j & 1 ? 16 : 0;
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(at),
                     "h"(static_cast<uint16_t>(h[j / 2] >> sh)) : "memory");
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + S::TERM),
                     "h"(static_cast<uint16_t>(l[j / 2] >> sh)) : "memory");
      }
    }
  }

  for (int i = tid * 16; i < S::P - S::A; i += THREADS * 16) put(base + S::A + i, uint4{});
  // (the first remote stores to A come after the first barrier of a step)

  // A round of MMA: everyone's stores, then thread 0's instructions, then their end.  Once a
  // thread's wait has run out the CTA issues none any more, and that thread waits for none: the
  // end of a round, should it still come, is not taken for another's.  What is left of the steps
  // are the cluster's barriers (other CTAs' are open), over values that are not stored.
  uint32_t phase = 0;
  bool ok = true;
  auto round = [&](auto&& issue) {
    fence_proxy_async_all();
    __syncthreads();
    // (debug_flags: testing; without MMAs the wait runs out)
    if (tid == 0 && !*abort_flag && !(g.debug_flags & 1)) {
      tc_fence_after();
      issue();
      tc_commit(bar);
    }
    __syncwarp();
    if (ok && !mbar_wait(bar, phase, g.timeout_ns, abort_flag)) {
      ok = false;
      *abort_flag = 1;
      atomicExch(g.status, O_TIMEOUT);
    }
    phase ^= 1u;
    __syncwarp();
    tc_fence_after();
  };
  // D = P Q over 16-element steps of K, step k's operands at p(k), q(k) in their first terms:
  // with two terms hi lo, lo hi, hi hi.  For an fp32 result the leading product comes in four parts
  // of two steps, an accumulator each: the tensor cores truncate what they add to.
  static_assert(!PARTS || WIDTH == 128, "four accumulators");
  auto products = [&](bool two, uint32_t idesc, int ksteps, auto&& p, int p_term, auto&& q,
                      int q_term) {
    uint32_t more = 0;
    for (int seg = two ? 0 : 2; seg < 3; ++seg)
      for (int k = 0; k < ksteps; ++k) {
        const int acc = PARTS && seg == 2 ? k >> 1 : 0;
        if (acc > 0) more = k & 1;
        tc_mma_bf16(tmem + acc * 128, p(k, seg == 1 ? p_term : 0), q(k, seg == 0 ? q_term : 0),
                    idesc, more);
        more = 1;
      }
  };
  auto kmajor = [](uint32_t at) {  // step k of an operand of 64-column blocks
    return [at](int k, int term) {
      return sdesc_sw128(at + term + (k >> 2) * BLOCK + (k & 3) * 32, 16, 1024);
    };
  };
  const int q = warp & 3, part = warp >> 2, row = q * 32 + lane;  // lanes, quarter of columns
  const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
  // 32 columns of D from c, a row a thread.
  auto read = [&](int c, float (&f)[32]) {
    uint32_t a[32];
    tmem_ld32(tmem + lanes + c, a);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(a[i]);
#pragma unroll 1
    for (int acc = 1; PARTS && acc < 4; ++acc) {
      tmem_ld32(tmem + acc * 128 + lanes + c, a);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i) f[i] += __uint_as_float(a[i]);
    }
  };
  const int share = (g.m + ctas - 1) / ctas;  // A's rows of a CTA

  for (int step = 0; step < g.steps; ++step) {
    // this CTA's share of A
    round([&] {
      products(PARTS, IDESC<128, false>, WIDTH / 16, kmajor(base + S::X), S::TERM,
               kmajor(base + S::X), S::TERM);
    });
    if (q * 32 < g.m && part * 32 < g.m) {
      float a[32];
      read(part * 32, a);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        st_shared_v4(sum_part(base + S::P, row, part * 8 + j), __float_as_uint(a[4 * j]),
                     __float_as_uint(a[4 * j + 1]), __float_as_uint(a[4 * j + 2]),
                     __float_as_uint(a[4 * j + 3]));
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    // my rows of A over the cluster, to all of it: half a warp a row, a lane eight columns (what
    // lies outside m x m is zero and stays so: the exchange's bytes are most of a step's time)
    for (int i = warp * 2 + (lane >> 4); i < share; i += THREADS / 16) {
      const int r = rank * share + i, c = (lane & 15) * 8;
      if (r >= g.m || c >= g.m) continue;
      const uint32_t x = sum_part(base + S::P, r, c / 4), y = sum_part(base + S::P, r, c / 4 + 1);
      float f[8] = {};
      if (ctas == 8) cluster_sums<8>(x, y, f);
      else if (ctas == 4) cluster_sums<4>(x, y, f);
      else if (ctas == 2) cluster_sums<2>(x, y, f);
      else cluster_sums<1>(x, y, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= ORTHO_A / (ORTHO_X * ORTHO_X);
      const uint4 hi = take_term(f), lo = take_term(f);
      for (int s = 0; s < ctas; ++s) {
        const uint32_t to = mapa_shared(piece(base + S::A, r, c), static_cast<uint32_t>(s));
        st_cluster_v4(to, hi);
        if (PARTS) st_cluster_v4(to + S::A_TERM, lo);
      }
    }
    fence_proxy_async_all();
    __syncwarp();
    cluster_sync();
    // P = b A + c A A
    round([&] {
      products(PARTS, IDESC<128, false>, 8, kmajor(base + S::A), S::A_TERM,
               kmajor(base + S::A), S::A_TERM);
    });
    {
      float a[32];
      read(part * 32, a);
#pragma unroll
      for (int j = 0; j < 32; j += 8) {
        const int col = part * 32 + j;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = g.c / ORTHO_A * a[j + i];
        if (PARTS) add_term(ld_shared_v4(piece(base + S::A + S::A_TERM, row, col)), g.b, f);
        add_term(ld_shared_v4(piece(base + S::A, row, col)), g.b, f);
        put(piece(base + S::P, row, col), take_term(f));
        put(piece(base + S::P + S::A_TERM, row, col), take_term(f));
      }
    }
    tc_fence_before();
    // a X + P X of my columns
    const bool last = step + 1 == g.steps;
    round([&] {
      products(true, IDESC<WIDTH, true>, 8, kmajor(base + S::P), S::A_TERM,
               [&](int k, int term) {
                 return sdesc_sw128(base + S::X + term + k * 2048, BLOCK, 1024);
               },
               S::TERM);
    });
    const float alpha = last ? g.a * (g.scale / ORTHO_X) : g.a;
    const float beta = last ? g.scale / ORTHO_X / ORTHO_A : 1.f / ORTHO_A;
#pragma unroll 1
    for (int c = part * (WIDTH / 4); c < (part + 1) * (WIDTH / 4); c += 32) {
      float a[32];
      __syncwarp();
      read(c, a);
#pragma unroll
      for (int j = 0; j < 32; j += 8) {
        const uint32_t hi = piece(base + S::X, row, c + j), lo = hi + S::TERM;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = beta * a[j + i];
        add_term(ld_shared_v4(lo), alpha, f);
        add_term(ld_shared_v4(hi), alpha, f);
        if (!last) {
          put(hi, take_term(f));
          put(lo, take_term(f));
        } else if (ok && row < g.m && col0 + c + j < g.n) {
          if (g.transposed) {  // the warp's rows are contiguous
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const size_t at = first + static_cast<size_t>(col0 + c + j + i) * g.m + row;
              if (g.out_bf16) static_cast<__nv_bfloat16*>(g.out)[at] = __float2bfloat16_rn(f[i]);
              else static_cast<float*>(g.out)[at] = f[i];
            }
          } else {
            const size_t at = first + static_cast<size_t>(row) * g.n + col0 + c + j;
            if (g.out_bf16) {
              st_global_v4(static_cast<__nv_bfloat16*>(g.out) + at,
                           make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                      pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])));
            } else {
              float4* o = reinterpret_cast<float4*>(static_cast<float*>(g.out) + at);
              o[0] = make_float4(f[0], f[1], f[2], f[3]);
              o[1] = make_float4(f[4], f[5], f[6], f[7]);
            }
          }
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (tid == 0 && *abort_flag) {  // what was issued ends before TMEM and shared memory are freed
    tc_commit(drain);
    volatile int never = 0;
    mbar_wait(drain, 0, 10000000ull, &never);
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, 512);
  }
}

template <int WIDTH, bool BF16, bool PARTS>
cudaError_t launch_of(const OrthoSmall& g, cudaStream_t stream) {
  auto kern = k_ortho_small<WIDTH, BF16, PARTS>;
  static std::atomic<unsigned long long> done{0};  // devices that have the attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(done.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<WIDTH>::BYTES);
    if (e != cudaSuccess) return e;
    if (dev < 64) done.fetch_or(1ull << dev);
  }
  int ctas = 1;
  while (ctas * WIDTH < g.n) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(g.batch * ctas), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = Smem<WIDTH>::BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, g);
}

}  // namespace

cudaError_t launch_ortho_small(const OrthoSmall& g, int width, cudaStream_t stream) {
  auto of = [&](auto bf16) {
    constexpr bool BF16 = decltype(bf16)::value;
    if (width == 256) return launch_of<256, BF16, false>(g, stream);
    return g.terms == 2 ? launch_of<128, BF16, true>(g, stream)
                        : launch_of<128, BF16, false>(g, stream);
  };
  return g.bf16 ? of(std::true_type{}) : of(std::false_type{});
}

}  // namespace mlpk
