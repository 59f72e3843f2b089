// The mixture of experts for up to eight tokens: the touched experts' weights
// stream once, with no sort, no sorted rows and no row tiles.
//
// Each touched expert is one group; the MMA's eight columns are the tokens
// themselves (a token that does not use the expert is a column of zeros), so
// the sum over a token's experts stays in a lane's registers.  Every CTA
// finds the groups by itself from the few ids: slot i opens a group when no
// earlier slot names its expert (an atomic minimum per expert in shared
// memory), and the groups are numbered in slot order.  A token that names an
// expert twice uses it once with the sum of the weights.
//
//   k_moe_decode_act   items (group, 16 rows of its Wg and Wu, or W1), all of H;
//                      h[slot] = s act(g) u; asks for the groups' Wd in L2 at
//                      its end
//   k_moe_decode_down  CTA r: 16 output features of every group: its warps
//                      walk (group, 64-wide k group) items round-robin, scale
//                      a group's sums by the routing weights as they leave it,
//                      and meet in shared memory; a cluster of CTAs shares the
//                      items when H alone gives too few CTAs, and its first
//                      CTA adds the others' sums in order, then the residual.
//
// HBM-bound: the weights are read once, everything else is small.  One token
// through 8 of 64 experts of 2048 x 1408 (138 MB): 33 us, of which about 9 are the
// two kernels' starts and ends; from there on 5.8 TB/s.  (Sixteen warps an SM,
// each two load groups ahead, because fewer draw less of HBM: eight took 35 us,
// twelve with the down kernel's warps beside them 36.)
#include <atomic>

#include "act.cuh"
#include "moe.h"
#include "stream.cuh"

namespace mlpk {

namespace {

using bf = __nv_bfloat16;

constexpr int DEC_ROWS = 16;  // weight rows of a CTA (the MMA's M)
constexpr int DEC_WARPS = 16;  // at most

// The groups of a call, in shared memory.
struct Groups {
  int n;
  int expert[MOE_DECODE_MAX_SLOTS];
  int slot[MOE_DECODE_MAX_SLOTS][8];    // the token's slot of the group (-1: none)
  float weight[MOE_DECODE_MAX_SLOTS][8];
};

// Fills `gr` (all threads; scratch: E + n ints).  weights == nullptr: the
// weights are not needed.
template <bool W_BF16>
__device__ __forceinline__ void find_groups(Groups& gr, int* scratch, const int* ids,
                                            const void* weights, int T, int top_k, int E) {
  const int n = T * top_k, tid = threadIdx.x, nt = blockDim.x;
  int* first = scratch;
  int* id = scratch + E;
  for (int e = tid; e < E; e += nt) first[e] = n;
  for (int i = tid; i < n; i += nt) {
    const int v = ids[i];
    id[i] = v >= 0 && v < E ? v : -1;
  }
  __syncthreads();
  for (int i = tid; i < n; i += nt)
    if (id[i] >= 0) atomicMin(first + id[i], i);
  __syncthreads();
  if (tid < 32) {
    int count = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + tid;
      const bool opens = i < n && id[i] >= 0 && first[id[i]] == i;
      const unsigned b = __ballot_sync(0xffffffffu, opens);
      if (opens) gr.expert[count + __popc(b & ((1u << tid) - 1u))] = id[i];
      count += __popc(b);
    }
    if (tid == 0) gr.n = count;
  }
  __syncthreads();
  for (int p = tid; p < gr.n * 8; p += nt) {
    const int g = p >> 3, m = p & 7, e = gr.expert[g];
    int at = -1;
    float w = 0.f;
    if (m < T) {
      for (int j = 0; j < top_k; ++j) {
        const int i = m * top_k + j;
        if (id[i] != e) continue;
        if (at < 0) at = i;
        if (weights)
          w += W_BF16 ? __bfloat162float(static_cast<const bf*>(weights)[i])
                      : static_cast<const float*>(weights)[i];
      }
    }
    gr.slot[g][m] = at;
    gr.weight[g][m] = w;
  }
  __syncthreads();
}

// Asks for the groups' Wd in L2 (at most 32 MB of them, a quarter of it), 2 KB
// a lane: HBM keeps streaming while the act kernel drains and the down kernel
// starts.
constexpr long long DEC_PREFETCH_BYTES = 32ll << 20, DEC_PREFETCH_PIECE = 2048;
__device__ __forceinline__ void prefetch_down(const Groups& gr, const bf* Wd, size_t mat,
                                              long long lane, long long lanes) {
  const long long bytes = static_cast<long long>(mat) * 2;
  const long long pieces = (bytes + DEC_PREFETCH_PIECE - 1) / DEC_PREFETCH_PIECE;  // of one expert
  long long total = pieces * gr.n;
  if (total > DEC_PREFETCH_BYTES / DEC_PREFETCH_PIECE)
    total = DEC_PREFETCH_BYTES / DEC_PREFETCH_PIECE;
  for (long long i = lane; i < total; i += lanes) {
    const long long g = i / pieces, off = (i - g * pieces) * DEC_PREFETCH_PIECE;
    const long long n = bytes - off < DEC_PREFETCH_PIECE ? bytes - off : DEC_PREFETCH_PIECE;
    const char* p = reinterpret_cast<const char*>(Wd) + gr.expert[g] * bytes + off;
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(static_cast<int>(n))
                 : "memory");
  }
}

// Work items (group, 16-row block) go round-robin over the CTAs (one an SM,
// all resident: the groups are found once and the loads never drain between
// items); an item's 64-wide k groups go round-robin over the CTA's warps,
// whose sums meet in shared memory, reduced by another warp for each item.
// The ring of two k groups a warp holds in flight runs across items.
template <int ACT, bool GATED>
__global__ void __launch_bounds__(32 * DEC_WARPS)
    k_moe_decode_act(const bf* __restrict__ x, const int* __restrict__ ids,
                     const bf* __restrict__ Wg, const bf* __restrict__ Wu,
                     const bf* __restrict__ Wd, bf* __restrict__ h, int T, int top_k, int E, int H,
                     int I, float s, int* status) {
  constexpr int NMAT = GATED ? 2 : 1;
  using G = MdGroup<NMAT, 8, 1, true>;
  extern __shared__ int scratch[];
  __shared__ Groups gr;
  __shared__ float4 part[2][DEC_WARPS][NMAT][32];
  pdl_wait();
  pdl_launch_dependents();
  if (status != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  find_groups<false>(gr, scratch, ids, nullptr, T, top_k, E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
  const int blocks = (I + DEC_ROWS - 1) / DEC_ROWS, items = gr.n * blocks;
  const int kgs = (H + MD_KG - 1) / MD_KG;  // at least nwarps
  const int g4 = lane >> 2, q = lane & 3;
  float acc[NMAT][1][1][4] = {};
  G buf[2];
  int item = blockIdx.x, kg = warp;          // the next k group to multiply
  int litem = item, lkg = kg;                // the next to load
  const size_t mat = static_cast<size_t>(I) * H;
  bool prefetched = false;
  auto load = [&](G& b) {
    if (litem >= items) {
      if (!prefetched) {
        prefetched = true;
        prefetch_down(gr, Wd, mat, (static_cast<long long>(blockIdx.x) * nwarps + warp) * 32 + lane,
                      static_cast<long long>(gridDim.x) * nwarps * 32);
      }
      return;
    }
    const int group = litem / blocks, row0 = (litem - group * blocks) * DEC_ROWS;
    const size_t at = static_cast<size_t>(gr.expert[group]) * mat;
    const bf* const W[2] = {Wg + at, GATED ? Wu + at : nullptr};
    const bf* const tok[1] = {gr.slot[group][g4] >= 0 ? x + static_cast<size_t>(g4) * H : nullptr};
    b.load_w(W, row0, I, H, lkg * MD_KG, lane);
    b.load_t_rows(tok, H, lkg * MD_KG, lane);
    lkg += nwarps;
    if (lkg >= kgs) {
      lkg = warp;
      litem += gridDim.x;
    }
  };
#pragma unroll
  for (int j = 0; j < 2; ++j) load(buf[j]);
  int done = 0;  // items finished: which half of `part`, and who reduces
  while (item < items) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (item < items) {
        buf[j].mma(acc);
        load(buf[j]);
        kg += nwarps;
        if (kg >= kgs) {
          float4(&mine)[DEC_WARPS][NMAT][32] = part[done & 1];
#pragma unroll
          for (int a = 0; a < NMAT; ++a) {
            float(&v)[4] = acc[a][0][0];
            mine[warp][a][lane] = make_float4(v[0], v[1], v[2], v[3]);
            v[0] = v[1] = v[2] = v[3] = 0.f;
          }
          // (this half is written again two items on, after its reader has
          // come through the next item's barrier)
          asm volatile("bar.sync 1, %0;" ::"r"(static_cast<int>(blockDim.x)) : "memory");
          if (warp == done % nwarps) {
            const int group = item / blocks, row0 = (item - group * blocks) * DEC_ROWS;
            float y[NMAT][4];
#pragma unroll
            for (int a = 0; a < NMAT; ++a) {
              float4 v = mine[0][a][lane];
              for (int w = 1; w < nwarps; ++w) {
                const float4 u = mine[w][a][lane];
                v.x += u.x;
                v.y += u.y;
                v.z += u.z;
                v.w += u.w;
              }
              y[a][0] = v.x;
              y[a][1] = v.y;
              y[a][2] = v.z;
              y[a][3] = v.w;
            }
            // element (hh, e) of lane (g, q): weight row g + 8 hh, token 2q + e
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int r = row0 + g4 + 8 * hh, slot = gr.slot[group][2 * q + e];
                if (r >= I || slot < 0) continue;
                float v = s * act_f<ACT>(y[0][2 * hh + e]);
                if constexpr (GATED) v *= y[NMAT - 1][2 * hh + e];
                h[static_cast<size_t>(slot) * I + r] = __float2bfloat16_rn(v);
              }
          }
          ++done;
          kg = warp;
          item += gridDim.x;
        }
      }
    }
  }
}

__device__ __forceinline__ float4 ld_cluster_float4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <bool W_BF16>
__global__ void __launch_bounds__(32 * DEC_WARPS)
    k_moe_decode_down(const bf* __restrict__ h, const int* __restrict__ ids,
                      const void* __restrict__ weights, const bf* __restrict__ Wd,
                      const bf* residual, bf* out, int T, int top_k, int E, int H, int I) {
  using G = MdGroup<1, 8, 1, true>;
  extern __shared__ int scratch[];
  __shared__ Groups gr;
  __shared__ float4 part[DEC_WARPS][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
  const int share = gridDim.y, rank = blockIdx.y;  // the cluster of one 16-row block
  const int row0 = blockIdx.x * DEC_ROWS;
  // ids, weights and Wd do not depend on the kernel before this one
  find_groups<W_BF16>(gr, scratch, ids, weights, T, top_k, E);
  const int kgs = (I + MD_KG - 1) / MD_KG;
  const int items = gr.n * kgs, step = nwarps * share;
  constexpr int DEPTH = 3;  // k groups in flight per warp
  float acc[1][1][1][4] = {}, sum[4] = {0.f, 0.f, 0.f, 0.f};
  G buf[DEPTH];
  auto load_w = [&](G& b, int it) {
    const int g = it / kgs;
    const bf* const W[2] = {Wd + static_cast<size_t>(gr.expert[g]) * H * I, nullptr};
    b.load_w(W, row0, H, I, (it - g * kgs) * MD_KG, lane);
  };
  auto load_t = [&](G& b, int it) {
    const int g = it / kgs, slot = gr.slot[g][lane >> 2];
    const bf* const tok[1] = {slot >= 0 ? h + static_cast<size_t>(slot) * I : nullptr};
    b.load_t_rows(tok, I, (it - g * kgs) * MD_KG, lane);
  };
  // the sums of a group's columns, times its weights
  auto leave = [&](int g) {
    const float w0 = gr.weight[g][2 * (lane & 3)], w1 = gr.weight[g][2 * (lane & 3) + 1];
    const bool u0 = gr.slot[g][2 * (lane & 3)] >= 0, u1 = gr.slot[g][2 * (lane & 3) + 1] >= 0;
    float(&a)[4] = acc[0][0][0];
    // (a column that is not used adds nothing, whatever the weights hold)
    if (u0) sum[0] = fmaf(w0, a[0], sum[0]), sum[2] = fmaf(w0, a[2], sum[2]);
    if (u1) sum[1] = fmaf(w1, a[1], sum[1]), sum[3] = fmaf(w1, a[3], sum[3]);
    a[0] = a[1] = a[2] = a[3] = 0.f;
  };
  const int it0 = warp * share + rank;
#pragma unroll
  for (int j = 0; j < DEPTH; ++j)
    if (it0 + j * step < items) load_w(buf[j], it0 + j * step);
  pdl_wait();
  pdl_launch_dependents();
#pragma unroll
  for (int j = 0; j < DEPTH; ++j)
    if (it0 + j * step < items) load_t(buf[j], it0 + j * step);
  int group = it0 / kgs;
  for (int it = it0; it < items;) {
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) {
      if (it < items) {
        const int g = it / kgs;
        if (g != group) {
          leave(group);
          group = g;
        }
        buf[j].mma(acc);
        const int nx = it + DEPTH * step;
        if (nx < items) {
          load_w(buf[j], nx);
          load_t(buf[j], nx);
        }
      }
      it += step;
    }
  }
  if (it0 < items) leave(group);
  part[warp][lane] = make_float4(sum[0], sum[1], sum[2], sum[3]);
  __syncthreads();
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (warp == 0) {
    for (int w = 0; w < nwarps; ++w) {
      const float4 u = part[w][lane];
      v.x += u.x;
      v.y += u.y;
      v.z += u.z;
      v.w += u.w;
    }
    part[0][lane] = v;
  }
  if (share > 1) {
    cluster_sync();
    if (rank == 0 && warp == 0) {
      for (int c = 1; c < share; ++c) {
        const float4 u = ld_cluster_float4(mapa_shared(smem_u32(&part[0][lane]), c));
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
      }
    }
    cluster_sync();  // no CTA leaves while its sums are read
  }
  if (rank != 0 || warp != 0) return;
  const float y[4] = {v.x, v.y, v.z, v.w};
  const int g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int hh = 0; hh < 2; ++hh)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = row0 + g + 8 * hh, t = 2 * q + e;
      if (r >= H || t >= T) continue;
      const size_t o = static_cast<size_t>(t) * H + r;
      const float res = residual ? __bfloat162float(residual[o]) : 0.f;
      out[o] = __float2bfloat16_rn(res + y[2 * hh + e]);
    }
}

template <class K>
cudaError_t launch_dec(K kern, dim3 grid, int threads, size_t smem, int cluster_y,
                       cudaStream_t stream, bool pdl, void** args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int na = 0;
  if (pdl) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster_y > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = 1;
    attr[na].val.clusterDim.y = cluster_y;
    attr[na++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kern), args);
}

// Most warps (up to DEC_WARPS and `most`) with which `ctas` CTAs are resident
// at once.
template <class K>
int resident_warps(K kern, std::atomic<int> (&cache)[DEC_WARPS + 1], int sms, int ctas, int most,
                   size_t smem) {
  int best = 1;
  for (int w = 1; w <= DEC_WARPS && w <= most; ++w) {
    int occ = cache[w].load() - 1;
    if (occ < 0) {
      if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, 32 * w, smem) != cudaSuccess)
        return best;
      cache[w].store(occ + 1);
    }
    if (static_cast<long long>(occ) * sms >= ctas) best = w;
  }
  return best;
}

int device_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

template <int ACT, bool GATED>
cudaError_t launch_act(const bf* x, const int* ids, const bf* Wg, const bf* Wu, const bf* Wd, bf* h,
                       int T, int top_k, int E, int H, int I, float s, cudaStream_t stream,
                       bool pdl, int* status) {
  const int n = T * top_k, sms = device_sms();
  if (sms == 0) return cudaErrorInvalidDevice;
  const long long items = static_cast<long long>(n < E ? n : E) * ((I + DEC_ROWS - 1) / DEC_ROWS);
  const int kgs = (H + MD_KG - 1) / MD_KG;
  const int warps = kgs < DEC_WARPS ? kgs : DEC_WARPS;
  void* args[] = {&x, &ids, &Wg, &Wu, &Wd, &h, &T, &top_k, &E, &H, &I, &s, &status};
  return launch_dec(k_moe_decode_act<ACT, GATED>,
                    dim3(static_cast<unsigned>(items < sms ? items : sms)), 32 * warps,
                    sizeof(int) * (E + n), 1, stream, pdl, args);
}

}  // namespace

cudaError_t launch_moe_decode_act(const void* x, const int* ids, const void* Wg, const void* Wu,
                                  const void* Wd, void* h, int T, int top_k, int E, int H, int I,
                                  int act, bool gated, float s, cudaStream_t stream, bool pdl,
                                  int* status) {
  if (T < 1 || T > MOE_DECODE_MAX_T || T * top_k > MOE_DECODE_MAX_SLOTS) return cudaErrorInvalidValue;
  const bf *xb = static_cast<const bf*>(x), *g = static_cast<const bf*>(Wg),
           *u = static_cast<const bf*>(Wu), *d = static_cast<const bf*>(Wd);
  bf* hb = static_cast<bf*>(h);
#define MLP_DEC(A, GT) \
  launch_act<A, GT>(xb, ids, g, u, d, hb, T, top_k, E, H, I, s, stream, pdl, status)
  if (gated) {
    switch (act) {
      case ACT_RELU: return MLP_DEC(ACT_RELU, true);
      case ACT_GELU_TANH: return MLP_DEC(ACT_GELU_EXP, true);
      case ACT_SIGMOID: return MLP_DEC(ACT_SIGMOID, true);
      default: return MLP_DEC(ACT_SILU, true);
    }
  }
  switch (act) {
    case ACT_RELU: return MLP_DEC(ACT_RELU, false);
    case ACT_GELU_TANH: return MLP_DEC(ACT_GELU_EXP, false);
    default: return MLP_DEC(ACT_RELU_SQ, false);
  }
#undef MLP_DEC
}

cudaError_t launch_moe_decode_down(const void* h, const int* ids, const void* weights, bool w_bf16,
                                   const void* Wd, const void* residual, void* out, int T,
                                   int top_k, int E, int H, int I, cudaStream_t stream, bool pdl) {
  if (T < 1 || T > MOE_DECODE_MAX_T || T * top_k > MOE_DECODE_MAX_SLOTS) return cudaErrorInvalidValue;
  static std::atomic<int> occ[2][DEC_WARPS + 1];
  const int n = T * top_k, blocks = (H + DEC_ROWS - 1) / DEC_ROWS, sms = device_sms();
  if (sms == 0) return cudaErrorInvalidDevice;
  const int items = (n < E ? n : E) * ((I + MD_KG - 1) / MD_KG);
  // CTAs sharing a 16-row block: as many as leave at most one CTA an SM, while
  // each has work for eight warps; then the most warps with which all CTAs
  // are resident
  int share = 1;
  while (share < 8 && 2 * share * blocks <= sms && items >= 2 * share * 8) share *= 2;
  auto kern = w_bf16 ? k_moe_decode_down<true> : k_moe_decode_down<false>;
  const size_t smem = sizeof(int) * (E + n);
  const int warps = resident_warps(kern, occ[w_bf16], sms, blocks * share,
                                   (items + share - 1) / share, sizeof(int) * 2048);
  const bf *hb = static_cast<const bf*>(h), *d = static_cast<const bf*>(Wd),
           *r = static_cast<const bf*>(residual);
  bf* o = static_cast<bf*>(out);
  void* args[] = {&hb, &ids, &weights, &d, &r, &o, &T, &top_k, &E, &H, &I};
  return launch_dec(kern, dim3(blocks, share), 32 * warps, smem, share, stream, pdl, args);
}

}  // namespace mlpk
