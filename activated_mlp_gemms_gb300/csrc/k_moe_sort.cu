// The stable counting sort of the slots by expert, in one launch.
//
// With c(i) the slots of slot i's expert before i, and off(e) the padded
// prefix sum of the experts' slot counts, slot i goes to row
// off(ids[i]) + c(i): no comparison, no atomic, and the same rows on every
// run.  One cluster of up to eight CTAs takes the slots in contiguous chunks,
// a chunk's 32 warps in contiguous sub-chunks:
//   1. every warp counts its sub-chunk per expert (32 slots at a time; lanes
//      with the same expert find each other by ballots, the first adds),
//   2. the counts become exclusive prefixes over the CTA's warps; the CTAs
//      read each other's totals through distributed shared memory,
//   3. every CTA scans the padded totals over the experts,
//   4. the warps walk their slots again and write pos and src (a slot's rank
//      within its warp, known from 1, waits in pos).
// Bound by the latency of its phases (a few cluster barriers and two passes
// over ids), not by its bytes (12 a slot): 5 us for 8198 slots over 8 experts, 13
// us for 65536 over 64.
#include <atomic>

#include "gemm_params.h"
#include "moe.h"
#include "ptx.cuh"

namespace mlpk {

namespace {

constexpr int SORT_WARPS = 32;
constexpr int SORT_THREADS = 32 * SORT_WARPS;
// Slots up to which one CTA sorts alone: a warp then walks at most two
// groups of 32 per pass, less than a cluster barrier costs.
constexpr int SORT_ONE_CTA = 2 * SORT_THREADS;
constexpr int SORT_CLUSTER = 8;
constexpr int SORT_AHEAD = 8;  // groups of 32 ids in flight per warp

// The lanes whose key is this lane's, for keys of `bits` bits: one ballot a bit
// (a warp match serialises over the distinct keys: 65536 slots over 64 experts
// took 19 us with it).
__device__ __forceinline__ unsigned same_key(int key, int bits) {
  unsigned same = 0xffffffffu;
  for (int b = 0; b < bits; ++b) {
    const bool set = (key >> b) & 1;
    const unsigned v = __ballot_sync(0xffffffffu, set);
    same &= set ? v : ~v;
  }
  return same;
}

__device__ __forceinline__ int ld_cluster_int(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Exclusive prefix sum of v over the block's threads (all of them take part);
// `total` receives the sum.  tmp: 33 ints of shared memory.
__device__ __forceinline__ int block_scan(int v, int* tmp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) tmp[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const int w = tmp[lane];
    int t = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += u;
    }
    tmp[lane] = t - w;
    if (lane == 31) tmp[32] = t;
  }
  __syncthreads();
  const int r = tmp[warp] + s - v;
  total = tmp[32];
  __syncthreads();  // tmp may be reused
  return r;
}

// Row tiles of `h` rows: their number and their list.  off: the experts'
// first rows in shared memory (E + 1); first: E + 1 ints of scratch.
__device__ __forceinline__ void write_tiles(const int* off, int E, int h, int* first, int* tmp,
                                            int* ntiles, MoeTile* list) {
  const int e = threadIdx.x;
  const int len = e < E ? off[e + 1] - off[e] : 0;
  int total;
  const int at = block_scan((len + h - 1) / h, tmp, total);
  if (e < E) first[e] = at;
  if (e == 0) {
    first[E] = total;
    *ntiles = total;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += SORT_THREADS) {
    int lo = 0, hi = E - 1;  // the last expert whose first tile is <= i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    MoeTile t;
    t.expert = lo;
    t.row = off[lo];
    t.end = off[lo + 1];
    t.first = first[lo];
    *reinterpret_cast<int4*>(list + i) = *reinterpret_cast<int4*>(&t);
  }
  __syncthreads();
}

// Shared memory: warp counts [32][E], totals of this CTA [E], base rows [E],
// offsets [E + 1], tile scratch [E + 1], scan scratch [33].
__host__ __device__ constexpr size_t sort_smem(int E) {
  return sizeof(int) * (static_cast<size_t>(SORT_WARPS) * E + 4 * static_cast<size_t>(E) + 2 + 33);
}

__global__ void __launch_bounds__(SORT_THREADS, 1)
    k_moe_sort(const int* __restrict__ ids, int* __restrict__ plan, const MoePlan L, int E, int n,
               int per_warp, int bits) {
  extern __shared__ int sm[];
  int* wcnt = sm;
  int* ctot = wcnt + SORT_WARPS * E;
  int* base = ctot + E;
  int* off = base + E;
  int* first = off + E + 1;
  int* tmp = first + E + 1;
  const int ncta = gridDim.x, cta = blockIdx.x;  // one cluster is the whole grid
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();

  for (int i = tid; i < SORT_WARPS * E; i += SORT_THREADS) wcnt[i] = 0;
  __syncthreads();
  const long long begin = (static_cast<long long>(cta) * SORT_WARPS + warp) * per_warp;
  const int lo = static_cast<int>(begin < n ? begin : n);
  const int hi = static_cast<int>(begin + per_warp < n ? begin + per_warp : n);
  int* mine = wcnt + warp * E;
  int* pos = plan + L.pos;
  int* src = plan + L.src;
  // SORT_AHEAD groups of 32 ids are loaded at a time; pos holds each slot's
  // rank within the warp's sub-chunk until the prefixes are known
  for (int i0 = lo; i0 < hi; i0 += 32 * SORT_AHEAD) {
    int id[SORT_AHEAD];
#pragma unroll
    for (int j = 0; j < SORT_AHEAD; ++j) {
      const int i = i0 + 32 * j + lane;
      id[j] = i < hi ? ids[i] : -1;
    }
#pragma unroll
    for (int j = 0; j < SORT_AHEAD; ++j) {
      if (i0 + 32 * j >= hi) break;
      const int i = i0 + 32 * j + lane;
      const int e = (id[j] >= 0 && id[j] < E) ? id[j] : -1;
      const unsigned same = same_key(e < 0 ? E : e, bits);
      const int at = e >= 0 ? mine[e] : 0;
      __syncwarp();
      if (e >= 0 && lane == __ffs(same) - 1) mine[e] = at + __popc(same);
      if (i < hi) pos[i] = at + __popc(same & ((1u << lane) - 1u));
      __syncwarp();
    }
  }
  __syncthreads();
  for (int e = tid; e < E; e += SORT_THREADS) {
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < SORT_WARPS; ++w) {
      const int c = wcnt[w * E + e];
      wcnt[w * E + e] = run;
      run += c;
    }
    ctot[e] = run;
  }
  if (ncta > 1) cluster_sync();
  else __syncthreads();
  int total = 0, before = 0;
  if (tid < E) {
    if (ncta > 1) {
      const uint32_t a = smem_u32(ctot + tid);
      int v[SORT_CLUSTER];
#pragma unroll
      for (int c = 0; c < SORT_CLUSTER; ++c) v[c] = ld_cluster_int(mapa_shared(a, c));
#pragma unroll
      for (int c = 0; c < SORT_CLUSTER; ++c) {
        if (c < cta) before += v[c];
        total += v[c];
      }
    } else {
      total = ctot[tid];
    }
  }
  const int padded = (total + MOE_ALIGN - 1) / MOE_ALIGN * MOE_ALIGN;
  int used;
  const int o = block_scan(padded, tmp, used);
  if (tid < E) {
    off[tid] = o;
    base[tid] = o + before;
  }
  if (tid == 0) off[E] = used;
  __syncthreads();

  for (int i0 = lo; i0 < hi; i0 += 32 * SORT_AHEAD) {
    int id[SORT_AHEAD], rank[SORT_AHEAD];
#pragma unroll
    for (int j = 0; j < SORT_AHEAD; ++j) {
      const int i = i0 + 32 * j + lane;
      id[j] = i < hi ? ids[i] : -1;
      rank[j] = i < hi ? pos[i] : 0;
    }
#pragma unroll
    for (int j = 0; j < SORT_AHEAD; ++j) {
      const int i = i0 + 32 * j + lane;
      if (i >= hi) continue;
      const bool used = id[j] >= 0 && id[j] < E;
      const int row = used ? base[id[j]] + mine[id[j]] + rank[j] : -1;
      pos[i] = row;
      if (used) src[row] = i;
    }
  }
  // the padding rows, the tables and the rows past the end
  if (cta == 0 && tid < E) {
    for (int r = o + total; r < o + padded; ++r) src[r] = -1;
    plan[L.offsets + tid] = o;
    plan[L.counts + tid] = total;
    if (tid == 0) {
      plan[L.offsets + E] = used;
      if (L.fine >= 0) plan[L.fine_flag] = 0;
    }
  }
  for (long long r = used + static_cast<long long>(cta) * SORT_THREADS + tid; r < L.rows;
       r += static_cast<long long>(ncta) * SORT_THREADS)
    src[r] = -1;
  // the two tile lists, by a CTA each where there are several
  for (int h = 0; h < 2; ++h)
    if (cta == (ncta > 1 ? ncta - 1 - h : 0))
      write_tiles(off, E, h == 0 ? 128 : 256, first, tmp, plan + L.ntiles + h,
                  reinterpret_cast<MoeTile*>(plan + L.tiles[h]));
  if (ncta > 1) cluster_sync();  // no CTA leaves while another reads its totals
}

}  // namespace

cudaError_t launch_moe_sort(const int* ids, int* plan, const MoePlan& L, int E, cudaStream_t stream,
                            bool pdl) {
  const int n = static_cast<int>(L.n);
  const int ctas = n <= SORT_ONE_CTA ? 1 : SORT_CLUSTER;
  const int slots = ctas * SORT_WARPS;
  const int per_warp = (n + slots - 1) / slots;
  const size_t smem = sort_smem(E);
  int bits = 1;  // of the keys 0 .. E (E: dropped)
  while ((E >> bits) != 0) ++bits;
  if (smem > 48 * 1024) {
    // once a device, to the most that any call takes: the attribute is the kernel's, and
    // another thread's call between this and the launch must not lower it
    static std::atomic<unsigned> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 31 || !(configured.load() & (1u << dev))) {
      e = cudaFuncSetAttribute(k_moe_sort, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(sort_smem(MOE_MAX_EXPERTS)));
      if (e != cudaSuccess) return e;
      if (dev < 31) configured.fetch_or(1u << dev);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(SORT_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int na = 0;
  if (pdl) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (ctas > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = ctas;
    attr[na].val.clusterDim.y = 1;
    attr[na++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  return cudaLaunchKernelEx(&cfg, k_moe_sort, ids, plan, L, E, n, per_warp, bits);
}

}  // namespace mlpk
