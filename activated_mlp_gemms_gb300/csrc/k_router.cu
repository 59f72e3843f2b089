// The router of a mixture of experts (mlp_router.h): softmax over a token's logits,
// its top_k experts, their weights, the experts' counts and the balance loss; and the
// logits' gradient.
//
// G lanes take a token, each V of its logits (E <= G V) in registers; a warp holds 32 / G
// tokens, which share its instructions.  Those bound the forward, most of them the choice
// (131072 x 256 fp32, 8 of them, with counts and loss: 57 us, 2.4 TB/s; some 220 instructions a
// token at half an instruction a cycle, by the latencies of its chains; 47 without the sums).  The
// choice goes by a bound from below and a ranking of the few values that reach it; by rounds of a
// largest value over the lanes where equal values are too many, or top_k.  The backward has two
// tokens' worth of memory traffic to one of the forward's: 48 us, 5.6 TB/s, 85 % of a copy.
// What a row needs of the others (counts, the probabilities' sums) stays in registers and
// shared memory until the block's tokens are done, goes out as one partial sum a block, and a
// second kernel (4-5 us) adds the blocks in their order.
#include <cuda_bf16.h>

#include <cfloat>

#include "gemm_params.h"
#include "ptx.cuh"
#include "step.h"

namespace mlpk {

namespace {

constexpr int ROUTER_THREADS = 256;
constexpr int FINISH_CTAS = 8;  // one cluster
constexpr int FINISH_THREADS = 256;
constexpr uint32_t KEY_NEG_INF = 0x007fffffu;

// A float as an unsigned integer of the same order: -0 is 0, a NaN above all.  (Adding zero
// makes -0 zero, and any NaN the canonical one, 0x7fffffff.)
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t b = __float_as_uint(f + 0.f);
  return b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The warp's largest, a NaN if there is one.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// (zero below 2^-126)
__device__ __forceinline__ float exp2_of(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float exp_of(float v) { return exp2_of(v * 1.44269504f); }
// x = e^(x - m), and their sum.
template <int V>
__device__ __forceinline__ float exps(float (&x)[V], float m) {
  const uint64_t minus = f2_pack(-m, -m), log2e = f2_pack(1.44269504f, 1.44269504f);
  uint64_t sum = 0;  // two zeros
#pragma unroll
  for (int v = 0; v < V; v += 2) {
    const float2 t = f2_unpack(f2_mul(f2_add(f2_pack(x[v], x[v + 1]), minus), log2e));
    x[v] = exp2_of(t.x);
    x[v + 1] = exp2_of(t.y);
    sum = f2_add(sum, f2_pack(x[v], x[v + 1]));
  }
  const float2 s = f2_unpack(sum);
  return s.x + s.y;
}
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// The largest of the group's, a NaN if there is one.  (As every collective here: all groups of
// a warp call it together, routed or not.)
template <int G>
__device__ __forceinline__ float group_max(float v) {
  if constexpr (G == 32) {
    return warp_max(v);
  } else {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}

// A lane's V values of a row come in chunks of one load: chunk i at i G C + lane C.
template <typename L, int G, int V>
struct Row {
  static constexpr int MOST = 16 / static_cast<int>(sizeof(L));
  static constexpr int C = V < MOST ? V : MOST;
  static __device__ __forceinline__ int at(int lane, int v) {
    return (v / C) * (G * C) + lane * C + v % C;
  }
  // vec: the row's chunks are aligned
  static __device__ __forceinline__ void load(const L* row, int lane, int E, bool vec,
                                              float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += C) {
      const int e = at(lane, i);
      if (vec && e + C <= E) {
        alignas(16) L raw[C];
        if constexpr (sizeof(raw) == 16)
          *reinterpret_cast<uint4*>(raw) = __ldg(reinterpret_cast<const uint4*>(row + e));
        else
          *reinterpret_cast<uint2*>(raw) = __ldg(reinterpret_cast<const uint2*>(row + e));
#pragma unroll
        for (int j = 0; j < C; ++j) x[i + j] = static_cast<float>(raw[j]);
      } else {
#pragma unroll
        for (int j = 0; j < C; ++j)
          x[i + j] = e + j < E ? static_cast<float>(row[e + j]) : -INFINITY;
      }
    }
  }
  static __device__ __forceinline__ void store(L* row, int lane, int E, bool vec,
                                               const float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += C) {
      const int e = at(lane, i);
      alignas(16) L raw[C];
#pragma unroll
      for (int j = 0; j < C; ++j) raw[j] = static_cast<L>(x[i + j]);
      if (vec && e + C <= E) {
        if constexpr (sizeof(raw) == 16)
          *reinterpret_cast<uint4*>(row + e) = *reinterpret_cast<const uint4*>(raw);
        else
          *reinterpret_cast<uint2*>(row + e) = *reinterpret_cast<const uint2*>(raw);
      } else {
#pragma unroll
        for (int j = 0; j < C; ++j)
          if (e + j < E) row[e + j] = raw[j];
      }
    }
  }
};

// d loss / d p of an expert with c slots, of N routed tokens: six roundings of fp32 (a double's
// division took 2 us of these kernels' last 5).
__device__ __forceinline__ float balance_coef(float E_k, int c, int N) {
  const float n = static_cast<float>(N);
  return N > 0 ? E_k * (static_cast<float>(c) / n) / n : 0.f;
}

// The sum of the block's threads (in a fixed order), in thread 0.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float warps_s[THREADS / 32];
  v = group_sum<32>(v);
  if (threadIdx.x % 32 == 0) warps_s[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < THREADS / 32; ++i) v += warps_s[i];
  return v;
}

struct FwdOut {
  int* ids;
  void* weights;
  int* counts;
  float* balance;
  RouterParts parts;
  int* status;
};

// The top_k largest of the group's values, largest first, by rounds: into sel_id and sel_x.
// Returns the largest, and -inf in all of x.
template <class R, int G, int V>
__device__ __forceinline__ float choose_by_rounds(float (&x)[V], int lane, int k,
                                                  int* sel_id, float* sel_x) {
  uint32_t key[V], top = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    key[v] = order_key(x[v]);
    x[v] = -INFINITY;
  }
  for (int j = 0; j < k; ++j) {
    uint32_t bk = 0;
    int be = 0;
#pragma unroll
    for (int v = V - 1; v >= 0; --v) {
      const bool better = key[v] >= bk;
      bk = better ? key[v] : bk;
      be = better ? R::at(lane, v) : be;
    }
    if constexpr (G == 32) {
      const uint32_t most = __reduce_max_sync(0xffffffffu, bk);
      be = __reduce_min_sync(0xffffffffu, bk == most ? be : 0x7fffffff);
      bk = most;
    } else {
#pragma unroll
      for (int s = G / 2; s > 0; s >>= 1) {
        const uint32_t ok = __shfl_xor_sync(0xffffffffu, bk, s);
        const int oe = __shfl_xor_sync(0xffffffffu, be, s);
        const bool better = ok > bk || (ok == bk && oe < be);
        bk = better ? ok : bk;
        be = better ? oe : be;
      }
    }
    if (j == 0) top = bk;
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = R::at(lane, v) == be ? 0u : key[v];
    if (lane == 0) {
      sel_id[j] = bk > KEY_NEG_INF ? be : -1;
      sel_x[j] = key_value(bk);
    }
  }
  return key_value(top);
}

// The same by a bound from below: the top_k-th largest of four partial largest values a lane.
// What reaches it (top_k values and a few more) goes to `some`, SOME pairs of value and expert,
// and each of those counts how many are before it.  (More than SOME of them, from equal values,
// or a NaN: the rounds, which all groups of a warp take together.)
template <int G>
constexpr int SOME = 4 * G < ROUTER_MAX_TOP_K ? 4 * G : ROUTER_MAX_TOP_K;
template <typename L, class R, int G, int V>
__device__ __forceinline__ float choose_by_bound(const float (&x)[V], const L* row, int lane,
                                                 int k, int* sel_id, float* sel_x, float2* some) {
  constexpr uint32_t ALL = 0xffffffffu;
  float m[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    m[s] = x[s * (V / 4)];
#pragma unroll
    for (int v = 1; v < V / 4; ++v) m[s] = max_nan(m[s], x[s * (V / 4) + v]);
  }
  const float top = group_max<G>(max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3])));
  auto order = [&](int i, int j) {
    const float a = m[i];
    m[i] = fmaxf(a, m[j]);
    m[j] = fminf(a, m[j]);
  };
  order(0, 1), order(2, 3), order(0, 2), order(1, 3), order(1, 2);
  float bound = top;
#pragma unroll 4
  for (int j = 1; j < k; ++j) {  // (equal ones leave together: the bound only gets lower)
    const bool gone = m[0] == bound;
    m[0] = gone ? m[1] : m[0];
    m[1] = gone ? m[2] : m[1];
    m[2] = gone ? m[3] : m[2];
    m[3] = gone ? -INFINITY : m[3];
    bound = m[0];
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) bound = fmaxf(bound, __shfl_xor_sync(ALL, bound, o));
  }
  bound = fmaxf(bound, -FLT_MAX);  // -inf is never chosen
  // by the difference's sign (inf - inf has none, and no zero has one with +0 added)
  uint32_t below_it = 0;  // x[0] the top bit
  const uint64_t minus = f2_pack(0.f - bound, 0.f - bound);
#pragma unroll
  for (int v = 0; v < V; v += 2) {
    const float2 d = f2_unpack(f2_add(f2_pack(x[v], x[v + 1]), minus));
    below_it = __funnelshift_l(__float_as_uint(d.x), below_it, 1);
    below_it = __funnelshift_l(__float_as_uint(d.y), below_it, 1);
  }
  uint32_t mine_in = ~below_it & (0xffffffffu >> (32 - V));
  int n = __popc(mine_in);  // then: those up to this lane's
#pragma unroll
  for (int o = 1; o < G; o <<= 1) {
    const int below = __shfl_up_sync(ALL, n, o, G);
    n += lane >= o ? below : 0;
  }
  int at = n - __popc(mine_in);
  n = __shfl_sync(ALL, n, G - 1, G);
  if (__any_sync(ALL, n > SOME<G> || top != top)) return NAN;
  for (; mine_in; mine_in &= mine_in - 1)  // (a lane has one or two)
    some[at++].y = __int_as_float(R::at(lane, V - __ffs(mine_in)));
  __syncwarp();
  for (int i = lane; i < n; i += G) some[i].x = static_cast<float>(row[__float_as_int(some[i].y)]);
  __syncwarp();
  for (int i = lane; i < n; i += 2 * G) {  // two a lane
    const int i2 = i + G < n ? i + G : i;
    const float2 p = some[i], q = some[i2];
    const int pe = __float_as_int(p.y), qe = __float_as_int(q.y);
    int before_p = 0, before_q = 0;
#pragma unroll 2
    for (int j = 0; j < n; ++j) {
      const float2 o = some[j];
      const int e = __float_as_int(o.y);
      before_p += o.x > p.x || (o.x == p.x && e < pe);
      before_q += o.x > q.x || (o.x == q.x && e < qe);
    }
    if (before_p < k) {
      sel_id[before_p] = pe;
      sel_x[before_p] = p.x;
    }
    if (before_q < k) {
      sel_id[before_q] = qe;
      sel_x[before_q] = q.x;
    }
  }
  for (int j = n + lane; j < k; j += G) {
    sel_id[j] = -1;
    sel_x[j] = 0.f;
  }
  return top;
}

template <typename L, int G, int V, bool SUMS, int THREADS>
__global__ void __launch_bounds__(THREADS)
    k_router_fwd(const RouterArgs a, const FwdOut o, const bool vec) {
  constexpr int NG = THREADS / G;
  using R = Row<L, G, V>;
  extern __shared__ __align__(16) float router_smem[];
  const int tid = threadIdx.x, lane = tid % G, g = tid / G, E = a.E, k = a.top_k;
  float2* some = reinterpret_cast<float2*>(router_smem) + g * SOME<G>;
  float* sels = router_smem + 2 * NG * SOME<G>;
  int* sel_id = reinterpret_cast<int*>(sels) + g * k;
  float* sel_x = sels + (NG + g) * k;
  int* cnt = reinterpret_cast<int*>(sels + 2 * NG * k);  // [E], SUMS
  float* psum = sels + 2 * NG * k + E;                   // [NG, E], SUMS
  __shared__ int routed_s[NG];
  if constexpr (SUMS) {
    for (int e = tid; e < E; e += THREADS) cnt[e] = 0;
    __syncthreads();
  }
  pdl_wait();
  pdl_launch_dependents();
  if (SUMS && o.status && blockIdx.x == 0 && tid == 0) *o.status = 0;
  uint64_t acc[V / 2];  // two sums each
#pragma unroll
  for (int v = 0; v < V / 2; ++v) acc[v] = 0;
  int n_routed = 0;
  // (every group of a warp stays in the loop to its end: they share the shuffles)
  const long long step = static_cast<long long>(gridDim.x) * NG;
  for (long long base = static_cast<long long>(blockIdx.x) * NG; base < a.T; base += step) {
    const long long t = base + g;
    const bool in = t < a.T;
    const bool take = in && (!a.mask || a.mask[t]);
    float x[V];
    const L* row = static_cast<const L*>(a.logits) + t * a.ldl;
    if (take) {
      R::load(row, lane, E, vec, x);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = -INFINITY;
    }
    float top = NAN;
    if (k <= SOME<G>) top = choose_by_bound<L, R, G, V>(x, row, lane, k, sel_id, sel_x, some);
    if (__any_sync(0xffffffffu, top != top)) {
      top = choose_by_rounds<R, G, V>(x, lane, k, sel_id, sel_x);
      if (take) R::load(row, lane, E, vec, x);  // (no registers for it and its keys)
    }
    __syncwarp();
    const bool routed = top != -INFINITY;
    // (what is not routed gets no weights, and no NaN from -inf - -inf)
    const float m = routed ? top : 0.f;
    float inv = 0.f;  // of the softmax's sum, or of the chosen ones'
    if (SUMS || !a.renorm) {
      float total = exps(x, m);
      total = group_sum<G>(total);
      inv = routed ? reciprocal(total) : 0.f;
      if constexpr (SUMS) {
        if (routed) {
          const uint64_t by = f2_pack(inv, inv);
#pragma unroll
          for (int v = 0; v < V; v += 2) acc[v / 2] = f2_fma(f2_pack(x[v], x[v + 1]), by, acc[v / 2]);
          ++n_routed;
        }
      }
    }
    auto put = [&](int j, int id, float w) {
      o.ids[t * k + j] = id;
      if (a.w_bf16) static_cast<__nv_bfloat16*>(o.weights)[t * k + j] = __float2bfloat16_rn(w);
      else static_cast<float*>(o.weights)[t * k + j] = w;
      if (SUMS && id >= 0) atomicAdd(&cnt[id], 1);
    };
    if (k <= G) {  // a slot a lane
      const int id = lane < k ? sel_id[lane] : -1;
      float w = id >= 0 ? exp_of(sel_x[lane] - m) : 0.f;
      w *= a.renorm ? reciprocal(group_sum<G>(w)) : inv;
      if (in && lane < k) put(lane, id, id >= 0 ? w : 0.f);
    } else {
      if (a.renorm) {
        float total = 0.f;
        for (int j = lane; j < k; j += G)
          if (sel_id[j] >= 0) total += exp_of(sel_x[j] - m);
        inv = reciprocal(group_sum<G>(total));
      }
      if (in) {
        for (int j = lane; j < k; j += G)
          put(j, sel_id[j], sel_id[j] >= 0 ? exp_of(sel_x[j] - m) * inv : 0.f);
      }
    }
    __syncwarp();
  }
  if constexpr (SUMS) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = R::at(lane, v);
      const float2 two = f2_unpack(acc[v / 2]);
      if (e < E) psum[g * E + e] = v % 2 ? two.y : two.x;
    }
    if (lane == 0) routed_s[g] = n_routed;
    __syncthreads();
    int n = 0;
    for (int i = 0; i < NG; ++i) n += routed_s[i];
    const float E_k = static_cast<float>(E) / static_cast<float>(k);
    float loss = 0.f;
    for (int e = tid; e < E; e += THREADS) {
      float s = 0.f;
      for (int i = 0; i < NG; ++i) s += psum[i * E + e];
      if (gridDim.x > 1) {
        const size_t at = static_cast<size_t>(blockIdx.x) * E + e;
        o.parts.c[at] = cnt[e];
        o.parts.p[at] = s;
      } else {  // all tokens were here
        const float coef = balance_coef(E_k, cnt[e], n);
        if (o.counts) o.counts[e] = cnt[e];
        if (o.balance) o.balance[1 + e] = coef;
        loss += coef * s;
      }
    }
    if (gridDim.x > 1) {
      if (tid == 0) o.parts.n[blockIdx.x] = n;
    } else if (o.balance) {
      loss = block_sum<THREADS>(loss);
      if (tid == 0) o.balance[0] = loss;
    }
  }
}

// The blocks' sums in their order: one cluster, each CTA its share of the experts.
__global__ void __launch_bounds__(FINISH_THREADS)
    k_router_finish(const int blocks, const int E, const int top_k, const RouterParts parts,
                    int* __restrict__ counts, float* __restrict__ balance) {
  __shared__ float p_s[FINISH_THREADS];
  __shared__ int c_s[FINISH_THREADS];
  __shared__ int n_s[FINISH_THREADS / 32];
  __shared__ float loss_s[FINISH_CTAS];  // CTA 0's
  const int tid = threadIdx.x;
  const int rank = static_cast<int>(cluster_ctarank());
  const int share = (E + FINISH_CTAS - 1) / FINISH_CTAS;  // at most 128
  int wide = 1;
  while (wide < share) wide *= 2;
  const int lane = tid % wide, row = tid / wide, rows = FINISH_THREADS / wide;
  const int e = rank * share + lane;
  const bool mine = lane < share && e < E;
  cluster_sync();  // CTA 0 is there
  pdl_wait();
  pdl_launch_dependents();
  int n = 0;
  for (int b = tid; b < blocks; b += FINISH_THREADS) n += parts.n[b];
  int c = 0;
  float s = 0.f;
  if (mine) {
#pragma unroll 10
    for (int b = row; b < blocks; b += rows) {
      c += parts.c[static_cast<size_t>(b) * E + e];
      s += parts.p[static_cast<size_t>(b) * E + e];
    }
  }
  n = __reduce_add_sync(0xffffffffu, n);
  if (tid % 32 == 0) n_s[tid / 32] = n;
  c_s[tid] = c;
  p_s[tid] = s;
  __syncthreads();
  for (int i = FINISH_THREADS / 2; i >= wide; i /= 2) {
    if (tid < i) {
      c_s[tid] += c_s[tid + i];
      p_s[tid] += p_s[tid + i];
    }
    __syncthreads();
  }
  float loss = 0.f;
  if (row == 0 && mine) {
    n = 0;
#pragma unroll
    for (int i = 0; i < FINISH_THREADS / 32; ++i) n += n_s[i];
    const float coef =
        balance_coef(static_cast<float>(E) / static_cast<float>(top_k), c_s[lane], n);
    if (counts) counts[e] = c_s[lane];
    if (balance) balance[1 + e] = coef;
    loss = coef * p_s[lane];
  }
  loss = block_sum<FINISH_THREADS>(loss);
  if (tid == 0) {
    const uint32_t to = mapa_shared(smem_u32(&loss_s[rank]), 0);
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(loss) : "memory");
  }
  __syncwarp();
  cluster_sync();
  if (rank == 0 && tid == 0 && balance) {
    loss = 0.f;
    for (int i = 0; i < FINISH_CTAS; ++i) loss += loss_s[i];
    balance[0] = loss;
  }
}

template <typename L, int G, int V>
__global__ void __launch_bounds__(ROUTER_THREADS, V <= 8 ? 0 : V <= 16 ? 4 : 3)
    k_router_bwd(const RouterArgs a, const int* __restrict__ ids,
                 const float* __restrict__ balance, const void* __restrict__ dweights,
                 const float* __restrict__ dloss, void* dlogits, const bool vec, const bool vec_d) {
  constexpr int NG = ROUTER_THREADS / G;
  using R = Row<L, G, V>;
  extern __shared__ __align__(16) float router_smem[];
  const int tid = threadIdx.x, lane = tid % G, g = tid / G, E = a.E, k = a.top_k;
  // the token's exponentials by expert, then its gradients
  float* buf = router_smem + g * (G * V);
  auto put_row = [&](const float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4*>(buf + R::at(lane, i)) =
          make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  };
  pdl_wait();
  pdl_launch_dependents();
  // The loss's gradient by each expert's probability: in registers up to 256 experts, and the
  // next token's operands, too.  Above, more blocks an SM are worth more: 32768 x 1024 bf16 115 us
  // so, now 57, 65536 x 512 68 and 49; but 131072 x 256 fp32 57 without them, 48 with.
  constexpr bool ROOM = V <= 8;
  float kept[ROOM ? V : 1];
  float* coef_s = router_smem + NG * (G * V);
  {
    const float d = dloss ? *dloss : 0.f;
    if constexpr (ROOM) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = R::at(lane, v);
        kept[v] = dloss && e < E ? balance[1 + e] * d : 0.f;
      }
    } else {
      for (int e = tid; e < G * V; e += ROUTER_THREADS)
        coef_s[e] = dloss && e < E ? balance[1 + e] * d : 0.f;
      __syncthreads();
    }
  }
  auto coefs = [&](int v) {  // four of them from v
    if constexpr (ROOM) return make_float4(kept[v], kept[v + 1], kept[v + 2], kept[v + 3]);
    else return *reinterpret_cast<const float4*>(coef_s + R::at(lane, v));
  };
  const bool slots = dweights != nullptr;
  const bool one = k <= G;  // a slot a lane
  auto dw_at = [&](long long i) {
    return a.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(dweights)[i])
                    : static_cast<const float*>(dweights)[i];
  };
  // (with ROOM a token's are loaded while the one before it is worked on)
  float next_x[V], next_dw = 0.f;
  int next_id = -1;
  auto fetch = [&](long long t) {
    const bool take = t < a.T && (!a.mask || a.mask[t]);
    next_id = -1;
    if (take) {
      R::load(static_cast<const L*>(a.logits) + t * a.ldl, lane, E, vec, next_x);
      if (slots && one && lane < k) {
        next_id = ids[t * k + lane];
        next_dw = dw_at(t * k + lane);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) next_x[v] = -INFINITY;
    }
  };
  const long long step = static_cast<long long>(gridDim.x) * NG;
  if (ROOM) fetch(static_cast<long long>(blockIdx.x) * NG + g);
  for (long long base = static_cast<long long>(blockIdx.x) * NG; base < a.T; base += step) {
    const long long t = base + g;
    if (!ROOM) fetch(t);
    float x[V];
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = next_x[v];
    int id = next_id;
    const float dw = next_dw;
    if (ROOM) fetch(t + step);
    float m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = max_nan(m, x[v]);
    m = group_max<G>(m);
    const bool routed = m != -INFINITY;
    if (!routed) m = 0.f;
    if (!routed || id >= E) id = -1;
    float total = exps(x, m);
    put_row(x);
    __syncwarp();
    total = group_sum<G>(total);
    const float inv = routed ? reciprocal(total) : 0.f;
    // what the weights' gradient adds at the chosen experts: w (dw - <w, dw>), or p dw of
    // p (dw - <p, dw>).  (A caller's own ids may all be of experts whose exponentials vanish:
    // their sum is kept from zero, and nothing is added.)
    float add = 0.f, dot = 0.f, w_inv = 1.f, w_dot = 0.f;
    if (slots && one) {
      const float e = id >= 0 ? buf[id] : 0.f;
      if (a.renorm) {
        const float s = group_sum<G>(e);
        const float d = group_sum<G>(id >= 0 ? e * dw : 0.f);
        const float r = reciprocal(fmaxf(s, FLT_MIN));
        if (id >= 0) add = e * r * (dw - d * r);
      } else if (id >= 0) {
        add = dot = e * inv * dw;
      }
    } else if (slots) {
      float s = 0.f, d = 0.f;
      for (int j = lane; j < k; j += G) {
        const int i = routed && t < a.T ? ids[t * k + j] : -1;
        if (i < 0 || i >= E) continue;
        s += buf[i];
        d += buf[i] * dw_at(t * k + j);
      }
      if (a.renorm) {
        w_inv = reciprocal(fmaxf(group_sum<G>(s), FLT_MIN));
        w_dot = group_sum<G>(d) * w_inv;
      } else {
        w_inv = inv;
        dot = d * inv;
      }
    }
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      const float4 c = coefs(v);
      const float cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[v + j] *= inv;
        dot += x[v + j] * cs[j];
      }
    }
    dot = group_sum<G>(dot);
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      const float4 c = coefs(v);
      const float cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) x[v + j] *= cs[j] - dot;
    }
    if (!routed) {  // (whatever the loss's gradient is: zeros times an infinity are none)
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = 0.f;
    }
    if (slots) {
      if (one) {
        __syncwarp();  // (the exponentials have been read)
        put_row(x);
        __syncwarp();
        if (id >= 0) atomicAdd(&buf[id], add);  // (a caller's ids may name an expert twice)
      } else {  // a slot's exponential goes as its gradient comes: one at a time
        float keep[ROUTER_MAX_TOP_K / 8];
#pragma unroll
        for (int i = 0; i < ROUTER_MAX_TOP_K / 8; ++i) {
          const int j = lane + i * G;
          const int e = routed && t < a.T && j < k ? ids[t * k + j] : -1;
          keep[i] = e >= 0 && e < E ? buf[e] * w_inv * (dw_at(t * k + j) - w_dot) : 0.f;
        }
        __syncwarp();
        put_row(x);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < ROUTER_MAX_TOP_K / 8; ++i) {
          const int j = lane + i * G;
          const int e = routed && t < a.T && j < k ? ids[t * k + j] : -1;
          if (e >= 0 && e < E) atomicAdd(&buf[e], keep[i]);
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 q = *reinterpret_cast<const float4*>(buf + R::at(lane, i));
        x[i] = q.x, x[i + 1] = q.y, x[i + 2] = q.z, x[i + 3] = q.w;
      }
    }
    if (t < a.T) R::store(static_cast<L*>(dlogits) + t * a.ldd, lane, E, vec_d, x);
    __syncwarp();  // (before the next token's values go over these)
  }
}

// Lanes and values a lane of the backward by the number of experts.
template <class F>
cudaError_t by_experts_bwd(int E, F&& f) {
  if (E <= 32) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{});
  if (E <= 64) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 8>{});
  if (E <= 128) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{});
  if (E <= 256) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 8>{});
  if (E <= 512) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 32>{});
}
int lanes_bwd(int E) { return E <= 64 ? 8 : E <= 128 ? 16 : 32; }
// ... and of the forward: as few lanes as the registers allow, so that a warp chooses for up to
// four tokens at once.  (131072 x 256, 8 of them: 57 us, with 16 lanes of 16 values 62, 32 of 8
// 77; 65536 x 512, 10: 61, with 32 lanes 67.)
template <class F>
cudaError_t by_experts(int E, F&& f) {
  if (E <= 32) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{});
  if (E <= 64) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 8>{});
  if (E <= 128) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 16>{});
  if (E <= 256) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 32>{});
  if (E <= 512) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 32>{});
  return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 32>{});
}
int lanes_of(int E) { return E <= 256 ? 8 : E <= 512 ? 16 : 32; }

bool rows_aligned(const void* ptr, int ld, bool bf16) {
  return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 &&
         static_cast<long long>(ld) * (bf16 ? 2 : 4) % 16 == 0;
}

cudaLaunchConfig_t config(int blocks, size_t smem, cudaStream_t stream,
                          cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(ROUTER_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

int rounds(int T, int groups) { return (T - 1) / groups + 1; }

// Threads of the forward's blocks where the sums are wanted: as many as the registers allow (64
// a thread up to 128 experts, 128 above), since every block is a partial sum, and 256 where those
// would be too few blocks for the GPU.  (131072 x 128 with 512 threads: 29 us, now 23.)
int sum_threads(int T, int E) {
  const int many = E <= 128 ? 1024 : 512;
  return rounds(T, many / lanes_of(E)) > 152 ? many : ROUTER_THREADS;
}

}  // namespace

// (a function of the sizes alone: the workspace is, too)
int router_blocks(int T, int E) {
  const int threads = sum_threads(T, E);
  const int all = rounds(T, threads / lanes_of(E));
  if (all <= 8) return 1;  // one block, no second kernel
  const int most = threads > ROUTER_THREADS ? 152 : 2 * 152;
  return all < most ? all : most;
}

cudaError_t launch_router_fwd(const RouterArgs& a, int* ids, void* weights, int* counts,
                              float* balance, const RouterParts& parts, int* status,
                              cudaStream_t stream) {
  const bool sums = parts.n != nullptr;
  const int threads = sums ? sum_threads(a.T, a.E) : ROUTER_THREADS;
  const int all = rounds(a.T, ROUTER_THREADS / lanes_of(a.E));
  const int blocks = sums ? router_blocks(a.T, a.E) : all < 8 * 152 ? all : 8 * 152;
  const FwdOut o{ids, weights, counts, balance, parts, status};
  const bool vec = rows_aligned(a.logits, a.ldl, a.l_bf16);
  return by_experts(a.E, [&](auto g, auto v) {
    constexpr int G = decltype(g)::value, V = decltype(v)::value;
    const int ng = threads / G;
    const size_t smem =
        (2ull * ng * (SOME<G> + a.top_k) + (sums ? (ng + 1ull) * a.E : 0)) * 4;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(blocks, smem, stream, attr);
    cfg.blockDim.x = static_cast<unsigned>(threads);
    auto go = [&](auto kern) {
      // (at most 162 KB: 128 groups of 128 experts and 64 slots)
      const cudaError_t e = kern.allow_smem(200 * 1024);
      if (e != cudaSuccess) return e;
      return cudaLaunchKernelEx(&cfg, kern.kernel, a, o, vec);
    };
    if (!sums) return a.l_bf16 ? go(KernelOf<k_router_fwd<__nv_bfloat16, G, V, false, ROUTER_THREADS>>{})
                               : go(KernelOf<k_router_fwd<float, G, V, false, ROUTER_THREADS>>{});
    constexpr int MANY = V <= 16 ? 1024 : 512;
    if (threads == MANY) return a.l_bf16 ? go(KernelOf<k_router_fwd<__nv_bfloat16, G, V, true, MANY>>{})
                                         : go(KernelOf<k_router_fwd<float, G, V, true, MANY>>{});
    return a.l_bf16 ? go(KernelOf<k_router_fwd<__nv_bfloat16, G, V, true, ROUTER_THREADS>>{})
                    : go(KernelOf<k_router_fwd<float, G, V, true, ROUTER_THREADS>>{});
  });
}

cudaError_t launch_router_finish(int T, int E, int top_k, const RouterParts& parts, int* counts,
                                 float* balance, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config(FINISH_CTAS, 0, stream, attr);
  cfg.blockDim.x = FINISH_THREADS;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = FINISH_CTAS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_router_finish, router_blocks(T, E), E, top_k, parts, counts,
                            balance);
}

cudaError_t launch_router_bwd(const RouterArgs& a, const int* ids, const float* balance,
                              const void* dweights, const float* dloss, void* dlogits,
                              cudaStream_t stream) {
  const int all = rounds(a.T, ROUTER_THREADS / lanes_bwd(a.E));
  const int blocks = all < 8 * 152 ? all : 8 * 152;
  const bool vec = rows_aligned(a.logits, a.ldl, a.l_bf16);
  const bool vec_d = rows_aligned(dlogits, a.ldd, a.l_bf16);
  return by_experts_bwd(a.E, [&](auto g, auto v) {
    constexpr int G = decltype(g)::value, V = decltype(v)::value;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(blocks, (ROUTER_THREADS * V + (V > 8 ? G * V : 0)) * 4ull, stream, attr);
    auto go = [&](auto kern) {
      return cudaLaunchKernelEx(&cfg, kern, a, ids, balance, dweights, dloss, dlogits, vec, vec_d);
    };
    return a.l_bf16 ? go(k_router_bwd<__nv_bfloat16, G, V>) : go(k_router_bwd<float, G, V>);
  });
}

}  // namespace mlpk
