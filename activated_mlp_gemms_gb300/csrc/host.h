// host.h -- what the C entry points share on the host: the workspace's
// control block, TMA descriptor construction (with a cache keyed by
// pointer/shape/box), the launch builder of the tcgen05 GEMM, tracing, and
// the checks of pointers.
#pragma once
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <unordered_map>
#include <vector>

#include "gemm_params.h"
#include "mlp.h"

namespace mlpk {

// The workspace's control block (zeroed by every call): the status word
// (int 0), the tile-scheduler counters (ints 16..127) and the fused
// forward's per-block counts (ints 128..255).
constexpr size_t CTRL_BYTES = 1024;
constexpr int COUNTER_BASE = 16;
constexpr int MAX_COUNTERS = 112;
constexpr int DEP_BASE = 128;
constexpr int MAX_DEP_BLOCKS = 128;  // 256-row blocks of a fused forward: M <= 32768

inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ------------------------------------------------------------ tensor maps
inline PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
inline std::once_flag g_encode_once;

inline bool encode_fn_ok() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode != nullptr;
}

struct MapKey {
  const void* ptr;
  uint64_t inner, outer, stride;
  uint32_t box0, box1;
  int dtype, swizzle;
  uint64_t depth, stride2;
  bool operator==(const MapKey& o) const {
    return ptr == o.ptr && inner == o.inner && outer == o.outer && stride == o.stride &&
           box0 == o.box0 && box1 == o.box1 && dtype == o.dtype && swizzle == o.swizzle &&
           depth == o.depth && stride2 == o.stride2;
  }
};
struct MapKeyHash {
  size_t operator()(const MapKey& k) const {
    size_t h = reinterpret_cast<size_t>(k.ptr);
    h = h * 1000003u ^ k.inner;
    h = h * 1000003u ^ k.outer;
    h = h * 1000003u ^ k.stride;
    h = h * 1000003u ^ (static_cast<size_t>(k.box0) << 16 | k.box1);
    h = h * 1000003u ^ (static_cast<size_t>(k.dtype) << 8 | static_cast<size_t>(k.swizzle));
    h = h * 1000003u ^ k.depth;
    h = h * 1000003u ^ k.stride2;
    return h;
  }
};
inline std::mutex g_map_mu;
inline std::unordered_map<MapKey, CUtensorMap, MapKeyHash> g_map_cache;

// 2-D tensor map over a row-major [outer, inner] array with row pitch `pitch`
// elements, box {box0 (inner), box1 (outer)}; out-of-bounds elements read as
// zero and are not written.  bf16 operands use the 128-byte swizzle; the
// epilogue's 32 x 32 output boxes use the 64-byte (bf16) or 128-byte (fp32)
// swizzle of the staging buffers.
// dtype: 0 bf16, 1 fp32, 2 e4m3 bytes (uint8).  depth > 0: a stack of `depth`
// such arrays, pitch2 elements apart, as a 3-D map with boxes one array deep.
inline bool make_map(CUtensorMap* out, const void* ptr, uint64_t inner, uint64_t outer, uint64_t pitch,
              uint32_t box0, uint32_t box1, int dtype = 0,
              CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B,
                     uint64_t depth = 0, uint64_t pitch2 = 0) {
  MapKey key{ptr, inner, outer, pitch, box0, box1, dtype, static_cast<int>(swz),
             depth, pitch2};
  {
    std::lock_guard<std::mutex> lk(g_map_mu);
    auto it = g_map_cache.find(key);
    if (it != g_map_cache.end()) {
      *out = it->second;
      return true;
    }
  }
  if (!encode_fn_ok()) return false;
  const uint64_t esize = dtype == 1 ? 4 : (dtype == 2 ? 1 : 2);
  const CUtensorMapDataType dt = dtype == 1   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                 : dtype == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                              : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  cuuint64_t dims[3] = {inner, outer, depth};
  cuuint64_t strides[2] = {pitch * esize, pitch2 * esize};
  cuuint32_t box[3] = {box0, box1, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUtensorMap m;
  CUresult r = g_encode(&m, dt, depth ? 3 : 2, const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return false;
  std::lock_guard<std::mutex> lk(g_map_mu);
  if (g_map_cache.size() > 4096) g_map_cache.clear();
  g_map_cache.emplace(key, m);
  *out = m;
  return true;
}

// ------------------------------------------------------------ device info
inline int num_sms() {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64 && cache[dev]) return cache[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n;
}

inline std::atomic<unsigned long long> g_wait_ms{0};  // 0: the default below
inline std::atomic<int> g_debug_flags{0};

inline unsigned long long wait_limit_ns() {
  static unsigned long long env_ms = [] {
    const char* e = std::getenv("MLP_WAIT_TIMEOUT_MS");
    return e ? std::strtoull(e, nullptr, 10) : 0ull;
  }();
  unsigned long long ms = g_wait_ms.load();
  if (ms == 0) ms = env_ms;
  if (ms == 0) ms = 2000;  // 2 s: far above any legitimate wait (tiles take microseconds)
  return ms * 1000000ull;
}

// ------------------------------------------------------------ launch builder
// Operand roles: a K-major operand [rows, K] is loaded with boxes
// {64, rows-per-box}; an MN-major operand [K, MN] with boxes {64, 64}.
// The device activation (Act) an ABI activation applies to the gate or preact.
inline int device_act(int act) {
  switch (act) {
    case MLP_ACT_SWIGLU: return ACT_SILU;
    case MLP_ACT_RELU_SQ: return ACT_RELU_SQ;
    case MLP_ACT_GELU_TANH: return ACT_GELU_TANH;
    case MLP_ACT_RELU: return ACT_RELU;
    case MLP_ACT_REGLU: return ACT_RELU;
    case MLP_ACT_GEGLU: return ACT_GELU_TANH;
    case MLP_ACT_GLU: return ACT_SIGMOID;
    default: return ACT_SILU;
  }
}

// 0 auto, 1 single-CTA tiles, 2 CTA-pair tiles, 3 auto with the gated
// forward's two GEMMs as separate launches
inline std::atomic<int> g_tile_policy{0};

// CTA-group size for a GEMM whose output has `rows` rows: pairs (256-row
// tiles) unless the output fits one 128-row tile.
inline int pick_cg(int rows) {
  const int pol = g_tile_policy.load();
  if (pol == 1 || pol == 2) return pol;
  return rows > BM ? 2 : 1;
}

struct Gemm {
  Params p;
  int nmaps = 0;
  int cg = 1;
  bool ok = true;
  Gemm(const mlp_problem_t& pr, int* counter, int* status, int cg_)
      : Gemm(device_act(pr.act), pr.gate_mult * pr.down_mult, counter, status, cg_) {}
  Gemm(int act, float scale, int* counter, int* status, int cg_) : cg(cg_) {
    std::memset(&p, 0, sizeof(p));
    p.a_tx_bytes = BM * BK * 2;
    p.act = act;
    p.scale = scale;
    p.group_m = 16;
    p.counter = counter;
    p.status = status;
    p.timeout_ns = wait_limit_ns();
    p.debug_flags = g_debug_flags.load();
  }
  // K-major operand: array [rows, K] (row pitch K unless given), box {64, box_rows}
  int kmajor(const void* ptr, int rows, int K, int box_rows, int pitch = 0) {
    if (nmaps >= MAX_MAPS) { ok = false; return 0; }
    if (!make_map(&p.maps[nmaps], ptr, K, rows, pitch ? pitch : K, BK, box_rows)) ok = false;
    return nmaps++;
  }
  // K-major A operand [rows, K]: an output with fewer than 128 rows loads
  // boxes of its rows only (rounded up to 16); the MMA's rows beyond them
  // read stale shared memory and only produce accumulator rows past the
  // output, which the epilogue never stores.
  int kmajor_a(const void* ptr, int rows, int K, int pitch = 0) {
    const int box = rows < BM ? ((rows + 15) / 16) * 16 : BM;
    p.a_tx_bytes = box * BK * 2;
    return kmajor(ptr, rows, K, box, pitch);
  }
  // MN-major operand: array [K, MN] (row pitch MN unless given), box {64, 64}
  int mnmajor(const void* ptr, int K, int MN, int pitch = 0) {
    if (nmaps >= MAX_MAPS) { ok = false; return 0; }
    if (!make_map(&p.maps[nmaps], ptr, MN, K, pitch ? pitch : MN, 64, BK)) ok = false;
    return nmaps++;
  }
  // e4m3 operands [rows, K] (K bytes per row), boxes {128 k, box_rows}; the
  // A operand's boxes are row-sized below 128 rows, as in kmajor_a.
  int kmajor_u8(const void* ptr, int rows, int K, int box_rows) {
    if (nmaps >= MAX_MAPS) { ok = false; return 0; }
    if (!make_map(&p.maps[nmaps], ptr, K, rows, K, 2 * BK, box_rows, 2)) ok = false;
    return nmaps++;
  }
  int kmajor_a_u8(const void* ptr, int rows, int K) {
    const int box = rows < BM ? ((rows + 15) / 16) * 16 : BM;
    p.a_tx_bytes = box * BK * 2;  // 128 bytes per row, as for bf16
    return kmajor_u8(ptr, rows, K, box);
  }
  // 8-bit MN-major operand [K, MN] (MN bytes per row), boxes {128 mn, 128 k}
  int mnmajor_u8(const void* ptr, int K, int MN) {
    if (nmaps >= MAX_MAPS) { ok = false; return 0; }
    if (!make_map(&p.maps[nmaps], ptr, MN, K, MN, 2 * BK, 2 * BK, 2)) ok = false;
    return nmaps++;
  }
  // bf16 input [rows, cols] of a derivative epilogue, boxes {256, 128}: the
  // producer prefetches each tile's rows into L2 ahead of the epilogue
  int prefetch_map(const void* ptr, int rows, int cols) {
    if (!ptr) return -1;
    if (nmaps >= MAX_MAPS) { ok = false; return -1; }
    if (!make_map(&p.maps[nmaps], ptr, cols, rows, cols, MMA_N, BM, 0, CU_TENSOR_MAP_SWIZZLE_NONE))
      ok = false;
    return nmaps++;
  }
  // 8-bit epilogue output [rows, cols]: one 32-row x 128-byte box per warp
  // and tile, 128-byte swizzle; half = true: 32-row x 64-byte boxes, two per
  // warp and tile, 64-byte swizzle.
  int output_u8(void* ptr, int rows, int cols, bool half = false) {
    if (!ptr) return -1;
    if (nmaps >= MAX_MAPS) { ok = false; return -1; }
    if (!make_map(&p.maps[nmaps], ptr, cols, rows, cols, half ? 64 : 128, 32, 2,
                  half ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B))
      ok = false;
    return nmaps++;
  }
  // Epilogue output [rows, cols] (row pitch cols unless given), stored in 32 x 32
  // boxes; -1 when the output is not requested.
  int output(void* ptr, int rows, int cols, bool f32 = false, int pitch = 0) {
    if (!ptr) return -1;
    if (nmaps >= MAX_MAPS) { ok = false; return -1; }
    if (!make_map(&p.maps[nmaps], ptr, cols, rows, pitch ? pitch : cols, 32, 32, f32,
                  f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
      ok = false;
    return nmaps++;
  }
  // Stacks [depth, rows, cols] (dense): a K-major weight operand, an MN-major
  // one ([K, MN] each), and a stack of outputs
  // (or a part of each matrix: row pitch `pitch`, matrices pitch2 apart)
  int kmajor_stack(const void* ptr, int depth, int rows, int K, int box_rows, int pitch = 0,
                   uint64_t pitch2 = 0) {
    if (nmaps >= MAX_MAPS) { ok = false; return 0; }
    if (!make_map(&p.maps[nmaps], ptr, K, rows, pitch ? pitch : K, BK, box_rows, 0,
                  CU_TENSOR_MAP_SWIZZLE_128B, depth, pitch2 ? pitch2 : (uint64_t)rows * K))
      ok = false;
    return nmaps++;
  }
  int mnmajor_stack(const void* ptr, int depth, int K, int MN) {
    if (nmaps >= MAX_MAPS) { ok = false; return 0; }
    if (!make_map(&p.maps[nmaps], ptr, MN, K, MN, 64, BK, 0, CU_TENSOR_MAP_SWIZZLE_128B, depth,
                  (uint64_t)K * MN))
      ok = false;
    return nmaps++;
  }
  int output_stack(void* ptr, int depth, int rows, int cols, bool f32) {
    if (!ptr) return -1;
    if (nmaps >= MAX_MAPS) { ok = false; return -1; }
    // fp32 boxes 32 x 32, bf16 boxes 64 x 32: 128-byte rows
    if (!make_map(&p.maps[nmaps], ptr, cols, rows, cols, f32 ? 32 : 64, 32, f32,
                  CU_TENSOR_MAP_SWIZZLE_128B, depth, (uint64_t)rows * cols))
      ok = false;
    return nmaps++;
  }
  // Output of P over the sorted rows: boxes of 32 rows, and of 16 for the last
  // rows of an expert.  bf16 boxes have 32 columns (64-byte swizzle), or 64
  // (ROWS_WIDE, the plain store's; 128-byte swizzle), fp32 boxes 32.
  enum RowsKind { ROWS_BF16, ROWS_WIDE, ROWS_F32 };
  void output_rows(Prob& P, int i, void* ptr, int rows, int cols, RowsKind kind = ROWS_BF16,
                   int pitch = 0) {
    P.mapO[i] = P.mapO16[i] = -1;
    if (ptr) row_boxes(ptr, rows, cols, kind, pitch, P.mapO[i], P.mapO16[i]);
  }
  void row_boxes(void* ptr, int rows, int cols, RowsKind kind, int pitch, int& map32, int& map16) {
    for (int box : {32, 16}) {
      if (nmaps >= MAX_MAPS) { ok = false; return; }
      if (!make_map(&p.maps[nmaps], ptr, cols, rows, pitch ? pitch : cols,
                    kind == ROWS_WIDE ? 64 : 32, box, kind == ROWS_F32,
                    kind == ROWS_BF16 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B))
        ok = false;
      (box == 32 ? map32 : map16) = nmaps++;
    }
  }
  // ke: K elements per k-block (bf16 64, e4m3 128: a 128-byte row either way)
  Prob& add(int M, int N, int K0, int K1, int tile_n, int ksplit = 1, int ke = BK) {
    Prob& P = p.prob[p.nprob++];
    P.M = M;
    P.N = N;
    P.kb0 = (K0 + ke - 1) / ke;
    P.kb1 = (K1 + ke - 1) / ke;
    P.tiles_m = (M + BM * cg - 1) / (BM * cg);
    P.tiles_n = (N + tile_n - 1) / tile_n;
    const int kbt = P.kb0 + P.kb1;
    if (ksplit < 1) ksplit = 1;
    if (ksplit > kbt) ksplit = kbt;
    P.kper = (kbt + ksplit - 1) / ksplit;
    P.ksplit = (kbt + P.kper - 1) / P.kper;  // no empty splits
    P.unit_begin = p.total_units;
    P.units = P.tiles_m * P.tiles_n * P.ksplit;
    p.total_units += P.units;
    P.ld = N;
    P.mapO[0] = P.mapO[1] = P.mapO[2] = -1;
    P.mapI0 = P.mapI1 = -1;
    P.mapE = -1;
    P.l2a = P.l2b = 0;
    return P;
  }
  // B rows per K-major box: a CTA stages 256 / cg of the 256 B rows
  int b_rows() const { return MMA_N / cg; }
};

struct Call {
  cudaStream_t stream;
  int* status;
  int* counters;
  int next_counter = 0;
  int launches = 0;
  bool one_wave = false;      // its GEMMs claim no units (begin_one_wave)
  bool clear_status = false;  // its next GEMM clears the status word
  int* counter() { return counters + (next_counter++ % MAX_COUNTERS); }
  bool pdl() { return launches++ > 0; }  // the first kernel follows the memset or the caller's work
};

inline int cuda_err(cudaError_t e) { return e == cudaSuccess ? MLP_OK : MLP_ERR_CUDA; }

// A second stream per device for GEMMs that may run beside the caller's
// (the weight gradients beside dx), with the events of the fork and the
// join.  `mu` is held from the fork to the join so that concurrent calls do
// not interleave their records and waits.
struct Side {
  std::mutex mu;
  cudaStream_t stream = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
  bool ok = false;
};
inline Side g_side[64];
inline std::mutex g_side_mu;

// The current device's side stream, created on first use; nullptr when it
// cannot be had (no device, creation failed, or first asked for while
// `caller` is being captured into a graph).
inline Side* side_stream(cudaStream_t caller) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  Side& sd = g_side[dev];
  std::lock_guard<std::mutex> lk(g_side_mu);
  if (sd.ok) return &sd;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(caller, &cs) != cudaSuccess || cs != cudaStreamCaptureStatusNone)
    return nullptr;
  if (cudaStreamCreateWithFlags(&sd.stream, cudaStreamNonBlocking) != cudaSuccess) return nullptr;
  if (cudaEventCreateWithFlags(&sd.fork, cudaEventDisableTiming) != cudaSuccess ||
      cudaEventCreateWithFlags(&sd.join, cudaEventDisableTiming) != cudaSuccess)
    return nullptr;
  sd.ok = true;
  return &sd;
}

// ------------------------------------------------------------ tracing
// When enabled, every kernel launch is bracketed by a pair of CUDA events on
// its stream; mlp_trace_read returns (kernel tag, milliseconds) per launch.
struct TraceRec {
  int tag;
  cudaEvent_t a, b;
};
inline std::mutex g_trace_mu;
inline bool g_trace_on = false;
inline std::atomic<bool> g_trace_flag{false};  // g_trace_on, readable without the lock
inline std::vector<TraceRec> g_trace;
inline std::vector<cudaEvent_t> g_event_pool;

inline cudaEvent_t trace_event() {
  if (!g_event_pool.empty()) {
    cudaEvent_t e = g_event_pool.back();
    g_event_pool.pop_back();
    return e;
  }
  cudaEvent_t e = nullptr;
  if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
  return e;
}

template <class F>
int traced(int tag, cudaStream_t s, F&& launch) {
  std::unique_lock<std::mutex> lk(g_trace_mu);
  if (!g_trace_on) {
    lk.unlock();
    return cuda_err(launch());
  }
  TraceRec r{tag, trace_event(), trace_event()};
  if (!r.a || !r.b) return MLP_ERR_CUDA;
  if (cudaEventRecord(r.a, s) != cudaSuccess) return MLP_ERR_CUDA;
  cudaError_t e = launch();
  if (cudaEventRecord(r.b, s) != cudaSuccess) return MLP_ERR_CUDA;
  g_trace.push_back(r);
  return cuda_err(e);
}

// Co-resident CTA groups of a kernel instance on the current device (cached).
template <int EPI, bool A_MN, bool B_MN, int CG, int ACT, bool GRP = false>
int groups_cached() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) {
    int v = cache[dev].load();
    if (v > 0) return v;
  }
  int v = max_groups<EPI, A_MN, B_MN, CG, ACT, GRP>();
  if (v > 0 && dev >= 0 && dev < 64) cache[dev].store(v);
  return v;
}

// Kernels that are built for single CTAs only (few slots' rows).
template <int EPI, bool A_MN, bool GRP>
constexpr bool singles_only() {
  return EPI == EPI_GATED_FINE || EPI == EPI_ACT_FINE || (EPI == EPI_ACCUM_F32 && !A_MN && GRP);
}

template <int EPI, bool A_MN, bool B_MN, int ACT, bool GRP = false>
int run_act(Gemm& g, Call& c, int tag) {
  if (!g.ok) return MLP_ERR_CUDA;
  if (g.p.total_units == 0) return MLP_OK;
  g.p.nmaps = g.nmaps;
  g.p.one_wave = c.one_wave;
  g.p.clear_status = c.clear_status;
  c.clear_status = false;
  const bool pdl = c.pdl();
  if constexpr (singles_only<EPI, A_MN, GRP>()) {
    if (g.cg != 1) return MLP_ERR_UNSUPPORTED;
  } else if (g.cg == 2) {
    const int groups = groups_cached<EPI, A_MN, B_MN, 2, ACT, GRP>();
    if (groups <= 0) return MLP_ERR_CUDA;
    const int n = g.p.total_units < groups ? g.p.total_units : groups;
    if (c.one_wave && n < g.p.total_units) return MLP_ERR_CUDA;  // (see one_wave_units)
    return traced(tag, c.stream,
                  [&] { return launch_gemm<EPI, A_MN, B_MN, 2, ACT, GRP>(g.p, 2 * n, c.stream, pdl); });
  }
  if constexpr (EPI == EPI_FWD_FUSED) {
    return MLP_ERR_UNSUPPORTED;  // CTA pairs only
  } else {
    const int sms = num_sms();
    const int n = g.p.total_units < sms ? g.p.total_units : sms;
    if (c.one_wave && n < g.p.total_units) return MLP_ERR_CUDA;
    return traced(tag, c.stream, [&] {
      return launch_gemm<EPI, A_MN, B_MN, 1, ACT, GRP>(g.p, n < 1 ? 1 : n, c.stream, pdl);
    });
  }
}

// Kernels without an activation epilogue.
template <int EPI, bool A_MN, bool B_MN, bool GRP = false>
int run(Gemm& g, Call& c, int tag) {
  return run_act<EPI, A_MN, B_MN, 0, GRP>(g, c, tag);
}

// Activation epilogues: one kernel instance per activation.
template <int EPI, bool A_MN, bool B_MN, bool GRP = false>
int run_gated(Gemm& g, Call& c, int tag) {
  switch (g.p.act) {
    case ACT_RELU: return run_act<EPI, A_MN, B_MN, ACT_RELU, GRP>(g, c, tag);
    case ACT_GELU_TANH: return run_act<EPI, A_MN, B_MN, GRP ? ACT_GELU_EXP : ACT_GELU_TANH, GRP>(g, c, tag);
    case ACT_SIGMOID: return run_act<EPI, A_MN, B_MN, ACT_SIGMOID, GRP>(g, c, tag);
    default: return run_act<EPI, A_MN, B_MN, ACT_SILU, GRP>(g, c, tag);
  }
}
template <int EPI, bool A_MN, bool B_MN, bool GRP = false>
int run_nongated(Gemm& g, Call& c, int tag) {
  switch (g.p.act) {
    case ACT_RELU: return run_act<EPI, A_MN, B_MN, ACT_RELU, GRP>(g, c, tag);
    case ACT_GELU_TANH: return run_act<EPI, A_MN, B_MN, GRP ? ACT_GELU_EXP : ACT_GELU_TANH, GRP>(g, c, tag);
    default: return run_act<EPI, A_MN, B_MN, ACT_RELU_SQ, GRP>(g, c, tag);
  }
}

// Required pointer present and 16-byte aligned; optional pointer aligned if present.
inline int need(const void* ptr) {
  if (!ptr) return MLP_ERR_INVALID_ARG;
  return aligned16(ptr) ? MLP_OK : MLP_ERR_ALIGNMENT;
}
inline int opt(const void* ptr) { return (!ptr || aligned16(ptr)) ? MLP_OK : MLP_ERR_ALIGNMENT; }

#define MLP_TRY(...)                 \
  do {                               \
    int _rc = (__VA_ARGS__);         \
    if (_rc != MLP_OK) return _rc;   \
  } while (0)

// Split-K factor of a bf16-output GEMM [rows, cols] x K whose output tiles
// cannot fill the GPU: the splits' fp32 partial sums meet in a zeroed region
// of the workspace (TMA reduce-add) and one elementwise pass converts it to
// bf16.  It depends on the shape only (a nominal 152 SMs), so the workspace
// size does too.
//  - Decode-sized token counts (at most 32 tiles of 128 x 256): about 128
//    work units with at least 8 k-blocks each.
//  - `fill` (the forward's down projection): when its 256 x 256 tiles (CTA
//    pairs) would occupy at most half of the 76 pairs, the smallest split
//    whose units fill at least 80 % of their last wave, again with at least
//    8 k-blocks a unit.  (A 512-token Llama-3-8B down projection is 32 such
//    tiles.)  Measured against the unsplit forward (the gated forward then
//    runs as one launch): 9-13 % faster at 384 and 512 tokens of the
//    4096-wide shapes, 3-10 % at 640-1024 tokens of a 2048-wide one; with
//    more tiles, splitting until the units filled their waves lost to the
//    one-launch forward.  The backward's dx is left whole: its last wave
//    shares the GPU with the weight gradients on the second stream.
constexpr int SPLIT_NOMINAL_SMS = 152;
inline int bf16_split(int rows, int cols, int K, bool fill) {
  const long long tiles =
      (long long)((rows + BM - 1) / BM) * (long long)((cols + MMA_N - 1) / MMA_N);
  const int kb = (K + BK - 1) / BK;
  if (kb < 16) return 1;
  if (tiles <= 32) {
    int split = static_cast<int>(128 / tiles);
    if (split > kb / 8) split = kb / 8;
    return split < 2 ? 1 : split;
  }
  if (!fill) return 1;
  // 256 x 256 tiles on CTA pairs (rows > 128 take pairs)
  const int pairs = SPLIT_NOMINAL_SMS / 2;
  const long long ptiles =
      (long long)((rows + 2 * BM - 1) / (2 * BM)) * (long long)((cols + MMA_N - 1) / MMA_N);
  if (2 * ptiles > pairs) return 1;
  for (int s = 2; s <= 8 && kb / s >= 8; ++s) {
    const long long units = ptiles * s;
    const long long waves = (units + pairs - 1) / pairs;
    if (units * 5 >= waves * pairs * 4) return s;
  }
  return 1;
}

// Output tiles (256 columns, 128 x cg rows) of a GEMM output [rows, cols].
inline long long out_tiles(int rows, int cols, int cg) {
  return (long long)((rows + BM * cg - 1) / (BM * cg)) * ((cols + MMA_N - 1) / MMA_N);
}

// Split-K factor of the weight-gradient launch: when its output tiles cannot
// fill the GPU, the token reduction (K = M) is split so that the work units
// do, with at least 8 k-blocks per unit (fp32 accumulation only: the
// partial sums meet through atomic adds in dW).
inline int wgrad_split(int M, long long tiles, int cg, int fuse) {
  if (!fuse || tiles <= 0) return 1;
  const int slots = num_sms() / cg;
  const int kb = (M + BK - 1) / BK;
  int ksplit = 1;
  if (tiles < slots) {
    ksplit = (int)(slots / tiles);
    while (ksplit > 1 && kb / ksplit < 8) --ksplit;
  }
  return ksplit;
}

// clear = false: the call's first kernel clears the status word itself (the
// decode weight streams, which use no counter of the control block), so the
// call enqueues no memset.
inline int begin_call(Call& c, void* ws, void* stream, bool clear = true) {
  c.stream = static_cast<cudaStream_t>(stream);
  c.status = static_cast<int*>(ws);
  c.counters = static_cast<int*>(ws) + COUNTER_BASE;
  return clear ? cuda_err(cudaMemsetAsync(ws, 0, CTRL_BYTES, c.stream)) : MLP_OK;
}

// A call whose GEMMs all have a unit for every cluster: they claim none, the
// control block needs no memset, and the call's first GEMM clears the status
// word (clear = false: another kernel of the call does).  Every kernel waits
// for the end of the one before it, so the first is launched while that, whatever
// it is, still runs.
inline void begin_one_wave(Call& c, void* ws, void* stream, bool clear = true) {
  begin_call(c, ws, stream, false);
  c.one_wave = true;
  c.clear_status = clear;
  c.launches = 1;
}
// Units up to which a GEMM is one wave: the clusters that are resident together
// (every instance holds an SM's shared memory: 76 pairs, 152 single CTAs).
inline int one_wave_units(int cg) {
  return cg == 2 ? groups_cached<EPI_STORE_BF16, false, false, 2, 0>() : num_sms();
}

// fp32 [n] -> bf16 [n] (the split-K partial-sum region to the output), plus
// alpha * resid when the block's residual is given.
inline int convert_out(Call& c, const float* part, void* out, long long n, const void* resid = nullptr,
                float alpha = 0.f) {
  const bool pdl = c.pdl();
  return traced(MLP_KERNEL_CONVERT, c.stream,
                [&] { return launch_f32_to_bf16(part, out, n, c.stream, pdl, resid, alpha); });
}

}  // namespace mlpk
