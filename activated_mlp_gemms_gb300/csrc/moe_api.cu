// moe_api.cu -- the C entry points of mlp_moe.h: argument validation and the
// launch sequences of the mixture-of-experts MLP.
#include "mlp_moe.h"

#include "host.h"
#include "moe.h"

using namespace mlpk;

namespace {

int check_moe(const mlp_moe_t* p) {
  if (!p) return MLP_ERR_INVALID_ARG;
  if (p->T <= 0 || p->E <= 0 || p->top_k <= 0 || p->H <= 0) return MLP_ERR_INVALID_ARG;
  if (p->weights_type != MLP_MOE_W_F32 && p->weights_type != MLP_MOE_W_BF16)
    return MLP_ERR_INVALID_ARG;
  if (p->H % 8) return MLP_ERR_ALIGNMENT;
  if (p->E > MLP_MOE_MAX_EXPERTS || p->top_k > MLP_MOE_MAX_TOP_K) return MLP_ERR_UNSUPPORTED;
  // rows and slots are 32-bit, the token kernels' grids and rounded-up widths too
  if (p->H > 0x7fffffff - 8191) return MLP_ERR_UNSUPPORTED;
  if ((long long)p->T * p->top_k > (1LL << 30) || (long long)p->T * p->H >= (1LL << 40))
    return MLP_ERR_UNSUPPORTED;
  return MLP_OK;
}

MoePlan plan_of(const mlp_moe_t* p) { return moe_plan(p->T, p->E, p->top_k, p->H); }
// The inference layer's own: no gradient follows.
MoePlan plan_of_infer(const mlp_moe_t* p) { return moe_plan(p->T, p->E, p->top_k, 0); }

bool w_bf16(const mlp_moe_t* p) { return p->weights_type == MLP_MOE_W_BF16; }

// The ids and the routing weights are read one by one: aligned as their type.
int need_ids(const void* ptr) {
  if (!ptr) return MLP_ERR_INVALID_ARG;
  return (reinterpret_cast<uintptr_t>(ptr) & 3u) ? MLP_ERR_ALIGNMENT : MLP_OK;
}
int need_w(const mlp_moe_t* p, const void* ptr) {
  if (!ptr) return MLP_ERR_INVALID_ARG;
  const uintptr_t low = w_bf16(p) ? 1u : 3u;
  return (reinterpret_cast<uintptr_t>(ptr) & low) ? MLP_ERR_ALIGNMENT : MLP_OK;
}

bool gated(const mlp_moe_t* p) {
  return p->act == MLP_ACT_SWIGLU || p->act == MLP_ACT_REGLU || p->act == MLP_ACT_GEGLU ||
         p->act == MLP_ACT_GLU;
}

// The calls that run the experts.
int check_experts(const mlp_moe_t* p) {
  MLP_TRY(check_moe(p));
  if (p->I <= 0 || p->act < MLP_ACT_SWIGLU || p->act > MLP_ACT_GLU) return MLP_ERR_INVALID_ARG;
  if (!std::isfinite(p->gate_mult) || !std::isfinite(p->down_mult)) return MLP_ERR_INVALID_ARG;
  if (p->I % 8) return MLP_ERR_ALIGNMENT;
  if (p->I > 0x7fffffff - 8191) return MLP_ERR_UNSUPPORTED;
  const MoePlan L = plan_of(p);
  // 32-bit work units (three weight gradients of 128 x 256 tiles at most)
  const long long tiles = out_tiles(p->I, p->H, 1) + out_tiles(p->H, p->I, 1);
  if (L.rows * p->I >= (1LL << 40) || tiles * 2 * p->E >= (1LL << 31) ||
      (L.tile_cap[0]) * ((p->H > p->I ? p->H : p->I) / 128 + 1) >= (1LL << 31))
    return MLP_ERR_UNSUPPORTED;
  return MLP_OK;
}

int check_weights(const mlp_moe_t* p, const void* Wg, const void* Wu, const void* Wd) {
  MLP_TRY(need(Wg));
  MLP_TRY(need(Wd));
  return gated(p) ? need(Wu) : (Wu ? MLP_ERR_INVALID_ARG : MLP_OK);
}

// The workspace after the control block.
struct Layout {
  size_t inter;              // the postact [rows, I]
  size_t plan, xs, y, total; // MLP_MODE_INFER: the plan and the sorted rows
};
Layout layout(const mlp_moe_t* p, int mode) {
  const MoePlan L = plan_of_infer(p);
  Layout w = {};
  size_t at = CTRL_BYTES;
  w.inter = at;
  at += round256((size_t)L.rows * p->I * 2);
  if (mode == MLP_MODE_INFER) {
    w.plan = at;
    at += round256((size_t)L.ints * 4);
    w.xs = at;
    at += round256((size_t)L.rows * p->H * 2);
    // y in fp32: the sum over a token's experts rounds once (in bf16 the layer's
    // error was 0.0029 of its result, now 0.0024; the fp32 rows cost 1 %)
    w.y = at;
    at += round256((size_t)L.rows * p->H * 4);
  }
  w.total = at;
  return w;
}

int check_ws(const mlp_moe_t* p, int mode, const void* ws, size_t ws_bytes) {
  if (!ws) return MLP_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return MLP_ERR_ALIGNMENT;
  return ws_bytes < layout(p, mode).total ? MLP_ERR_WORKSPACE_TOO_SMALL : MLP_OK;
}

// CTA pairs (256-row tiles) from an average of 160 rows an expert, for the weight
// gradients from 256: an expert's last tile is half empty on average, 128 rows of a
// pair's tile or 64 of a single CTA's, while a pair's tile is the faster one per row.
// What decides is how the rows of each expert fill whole tiles, which only the device
// knows; the average decides well enough.  Measured (time on pairs / on singles;
// gate/up, down, dgated, dx | weight gradients; 16 experts of 2048 x 4864):
//   rows   96   1.03 1.10 1.01 1.11 | 1.11    uneven counts 1.05  .79  .99  .78 | 1.05
//         128   1.04 1.10 1.00 1.11 | 1.13                  1.02  .83 1.08  .82 | 1.09
//         160    .85  .87  .98  .86 | 1.06                   .97  .85 1.02  .85 | 1.07
//         192    .86  .88  .96  .87 | 1.09                   .91 1.09  .90 1.13 | 1.04
//         256    .88  .90  .97  .87 |  .98                   .88  .82  .90  .83 | 1.01
//         320   1.01 1.00 1.03 1.05 |  .99                   .92  .84  .96  .86 |  .98
//         384   1.02 1.00 1.03 1.05 |  .90                   .92  .99  .95 1.05 |  .96
//         512    .85  .82  .91  .88 |  .92                   .94  .97  .99 1.04 |  .94
//        1024    .85  .83  .86  .87 |  .90                   .88  .83  .91  .88 |  .92
// (the entries above 1.0 at 320 and 384 rows are pairs' tiles half empty in every
// expert, those of the uneven counts one more tile in the last wave).
constexpr int MOE_PAIR_ROWS = 160, MOE_PAIR_ROWS_W = 256;
int moe_cg(const mlp_moe_t* p, int rows = MOE_PAIR_ROWS) {
  const int pol = g_tile_policy.load();
  if (pol == 1 || pol == 2) return pol;
  return (long long)p->T * p->top_k >= (long long)rows * p->E ? 2 : 1;
}

// Whether the inference layer streams the touched experts' weights: few tokens
// whose experts' weights are at most 1 GB, unless a tile policy asks for the
// tiles.  The stream saves the sort, the sorted rows and their launches, about
// 12 us; the tiles' TMA loads get 6-10 % more of HBM.  Measured (stream /
// tiles): 8 slots of 17 MB each 33 / 45 us, 32 of them 88 / 92, 64 134 / 130.
constexpr long long MOE_DECODE_MAX_BYTES = 1ll << 30;
bool decode_moe(const mlp_moe_t* p) {
  const int pol = g_tile_policy.load();
  const long long n = (long long)p->T * p->top_k;
  if ((pol != 0 && pol != 3) || p->T > MOE_DECODE_MAX_T || n > MOE_DECODE_MAX_SLOTS) return false;
  const long long expert = (long long)(gated(p) ? 3 : 2) * p->H * p->I * 2;
  return (n < p->E ? n : p->E) * expert <= MOE_DECODE_MAX_BYTES;
}

// A GEMM over the sorted rows: its output tiles are the plan's.
struct RowGemm : Gemm {
  RowGemm(const mlp_moe_t* p, Call& c, const int* plan) : RowGemm(p, c, plan, moe_cg(p)) {}
  RowGemm(const mlp_moe_t* p, Call& c, const int* plan, int cg_)
      : Gemm(device_act(p->act), p->gate_mult * p->down_mult, c.counter(), c.status, cg_),
        L(plan_of(p)) {
    this->p.tiles = reinterpret_cast<const MoeTile*>(plan + L.tiles[cg - 1]);
    this->p.ntiles = plan + L.ntiles + cg - 1;
    this->p.offsets = plan + L.offsets;
    this->p.rows = static_cast<int>(L.rows);
  }
  Prob& add_rows(int N, int K0, int K1, int tile_n) {
    Prob& P = add(static_cast<int>(L.rows), N, K0, K1, tile_n);
    P.units = static_cast<int>(L.tile_cap[cg - 1] * P.tiles_n);  // at most; the plan has the number
    p.total_units = P.units;
    return P;
  }
  int rows_a(const void* ptr, int K) { return kmajor(ptr, static_cast<int>(L.rows), K, BM); }
  MoePlan L;
};

// Output tiles of a GEMM over the rows with `cols` columns in tiles of tile_n, at
// most (the plan has their number).
long long row_units(const mlp_moe_t* p, int cols, int tile_n) {
  const int cg = moe_cg(p);
  return plan_of(p).tile_cap[cg - 1] * ((cols + tile_n - 1) / tile_n);
}
// The forward's GEMMs are one wave each.  (Up to MOE_FINE_SLOTS slots, too, where they
// are single CTAs whatever the tile policy: an expert's rows are one tile either way.)
bool fwd_one_wave(const mlp_moe_t* p) {
  const int most = one_wave_units(moe_cg(p));
  return row_units(p, p->I, gated(p) ? 128 : MMA_N) <= most && row_units(p, p->H, MMA_N) <= most;
}

int launch_experts_act(const mlp_moe_t* p, Call& c, const int* plan, const void* xs, const void* Wg,
                       const void* Wu, void* a, void* G, void* U) {
  RowGemm g(p, c, plan);
  const int rows = static_cast<int>(g.L.rows);
  const int mA = g.rows_a(xs, p->H);
  if (gated(p)) {
    const int mG = g.kmajor_stack(Wg, p->E, p->I, p->H, 128);
    const int mU = g.kmajor_stack(Wu, p->E, p->I, p->H, 128);
    Prob& P = g.add_rows(p->I, p->H, 0, 128);
    P.l2a = L2_EVICT_LAST;   // the rows: every tile column re-reads them
    P.l2b = L2_EVICT_FIRST;  // the weights: a panel's reuse is by consecutive row tiles
    P.mapA0 = mA;
    P.mapB0 = mG;
    P.mapB1 = mU;
    g.output_rows(P, 0, a, rows, p->I);
    g.output_rows(P, 1, G, rows, p->I);
    g.output_rows(P, 2, U, rows, p->I);
    return run_gated<EPI_GATED_FWD, false, false, true>(g, c, MLP_KERNEL_GATE_UP);
  }
  const int mW = g.kmajor_stack(Wg, p->E, p->I, p->H, g.b_rows());
  Prob& P = g.add_rows(p->I, p->H, 0, MMA_N);
  P.l2a = L2_EVICT_LAST;
  P.l2b = L2_EVICT_FIRST;
  P.mapA0 = mA;
  P.mapB0 = mW;
  g.output_rows(P, 0, a, rows, p->I);
  g.output_rows(P, 1, G, rows, p->I);
  return run_nongated<EPI_ACT_FWD, false, false, true>(g, c, MLP_KERNEL_GATE_UP);
}

// y32: y is fp32
int launch_experts_down(const mlp_moe_t* p, Call& c, const int* plan, const void* a, const void* Wd,
                        void* y, bool y32) {
  RowGemm g(p, c, plan);
  const int mA = g.rows_a(a, p->I);
  const int mB = g.kmajor_stack(Wd, p->E, p->H, p->I, g.b_rows());
  Prob& P = g.add_rows(p->H, p->I, 0, MMA_N);
  P.l2a = L2_EVICT_LAST;
  P.l2b = L2_EVICT_FIRST;
  P.mapA0 = mA;
  P.mapB0 = mB;
  g.output_rows(P, 0, y, static_cast<int>(g.L.rows), p->H, y32 ? Gemm::ROWS_F32 : Gemm::ROWS_WIDE);
  return y32 ? run<EPI_STORE_F32, false, false, true>(g, c, MLP_KERNEL_DOWN)
             : run<EPI_STORE_BF16, false, false, true>(g, c, MLP_KERNEL_DOWN);
}

// Few slots (MOE_FINE_SLOTS): y in fp32 into the plan, for the routing weights'
// gradient (k_moe_combine_bwd), from the postact as two bf16 terms: the k-blocks of
// both alternate against the same Wd, which the second finds in L2.  (y in fp32 from a postact of one
// term leaves 5 % of the steps of up to eight slots over 0.005.)  The first term has
// the workspace, the second waits in y, at most H columns of the postact at a time;
// y itself is written last, from the fp32 rows.  Single CTAs.
int launch_experts_fine(const mlp_moe_t* p, Call& c, int* plan, const void* xs, const void* Wg,
                        const void* Wu, const void* Wd, void* a, void* y, void* G, void* U) {
  const MoePlan L = plan_of(p);
  const int rows = static_cast<int>(L.rows), H = p->H, I = p->I;
  const bool gt = gated(p);
  const int tile_n = gt ? 128 : MMA_N;
  auto at = [](const void* ptr, long long n) {  // n bf16 values on
    return ptr ? const_cast<char*>(static_cast<const char*>(ptr)) + 2 * n : nullptr;
  };
  void* y32 = plan + L.fine;
  const int parts = (I + H - 1) / H;
  int most = ((I + parts - 1) / parts + 127) / 128 * 128;  // equal parts, whole tiles
  if (most > H) most = H;
  for (int c0 = 0; c0 < I; c0 += most) {
    const int w = I - c0 < most ? I - c0 : most;
    if (!c.one_wave && c.next_counter + 2 > MAX_COUNTERS) {  // (I above 56 H) counters to use again
      MLP_TRY(cuda_err(cudaMemsetAsync(c.counters, 0, MAX_COUNTERS * sizeof(int), c.stream)));
      c.next_counter = c.launches = 0;
    }
    {
      RowGemm g(p, c, plan, 1);
      const int mA = g.rows_a(xs, H);
      const int mG = g.kmajor_stack(at(Wg, (long long)c0 * H), p->E, w, H, tile_n, H, (uint64_t)I * H);
      const int mU = gt ? g.kmajor_stack(at(Wu, (long long)c0 * H), p->E, w, H, tile_n, H,
                                         (uint64_t)I * H) : 0;
      Prob& P = g.add_rows(w, H, 0, tile_n);
      P.l2a = L2_EVICT_LAST;
      P.l2b = L2_EVICT_FIRST;
      P.mapA0 = mA;
      P.mapB0 = mG;
      P.mapB1 = mU;
      g.output_rows(P, 0, at(a, c0), rows, w, Gemm::ROWS_BF16, I);
      g.output_rows(P, 1, at(G, c0), rows, w, Gemm::ROWS_BF16, I);
      g.output_rows(P, 2, at(U, c0), rows, w, Gemm::ROWS_BF16, I);
      g.row_boxes(y, rows, w, Gemm::ROWS_BF16, H, P.mapE, P.mapI1);
      MLP_TRY(gt ? run_gated<EPI_GATED_FINE, false, false, true>(g, c, MLP_KERNEL_GATE_UP)
                 : run_nongated<EPI_ACT_FINE, false, false, true>(g, c, MLP_KERNEL_GATE_UP));
    }
    RowGemm g(p, c, plan, 1);
    const int mA0 = g.kmajor(at(a, c0), rows, w, BM, I);
    const int mA1 = g.kmajor(y, rows, w, BM, H);
    const int mB = g.kmajor_stack(at(Wd, c0), p->E, H, w, MMA_N, I, (uint64_t)H * I);
    Prob& P = g.add_rows(H, w, w, MMA_N);
    P.l2a = L2_EVICT_LAST;
    P.mapA0 = mA0;
    P.mapA1 = mA1;
    P.mapB0 = P.mapB1 = mB;
    g.output_rows(P, 0, y32, rows, H, Gemm::ROWS_F32);
    MLP_TRY(c0 == 0 ? (run<EPI_STORE_F32, false, false, true>(g, c, MLP_KERNEL_DOWN))
                    : (run<EPI_ACCUM_F32, false, false, true>(g, c, MLP_KERNEL_DOWN)));
  }
  const bool pdl = c.pdl();
  return traced(MLP_KERNEL_CONVERT, c.stream,
                [&] { return launch_moe_fine_rows(plan, L, p->E, H, y, c.stream, pdl); });
}

// The sort and the token kernels start while the kernel before them on the
// stream, whatever it is, still runs (programmatic launch): each waits for its
// end before it touches memory, and what is saved is the launch itself.

}  // namespace

extern "C" {

long long mlp_moe_rows(const mlp_moe_t* p) {
  return check_moe(p) == MLP_OK ? plan_of(p).rows : 0;
}

int mlp_moe_plan_layout(const mlp_moe_t* p, mlp_moe_plan_t* layout) {
  MLP_TRY(check_moe(p));
  if (!layout) return MLP_ERR_INVALID_ARG;
  const MoePlan L = plan_of(p);
  layout->ints = L.ints;
  layout->offsets = L.offsets;
  layout->counts = L.counts;
  layout->pos = L.pos;
  layout->src = L.src;
  return MLP_OK;
}

int mlp_moe_sort(const mlp_moe_t* p, const int* ids, void* plan, void* stream) {
  MLP_TRY(check_moe(p));
  MLP_TRY(need_ids(ids));
  MLP_TRY(need(plan));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(MLP_KERNEL_MOE_SORT, s, [&] {
    return launch_moe_sort(ids, static_cast<int*>(plan), plan_of(p), p->E, s, true);
  });
}

int mlp_moe_dispatch(const mlp_moe_t* p, const void* plan, const void* x, void* xs, void* stream) {
  MLP_TRY(check_moe(p));
  MLP_TRY(need(plan));
  MLP_TRY(need(x));
  MLP_TRY(need(xs));
  if (xs == x) return MLP_ERR_INVALID_ARG;  // other blocks still read x
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(MLP_KERNEL_MOE_DISPATCH, s, [&] {
    return launch_moe_dispatch(x, static_cast<const int*>(plan), plan_of(p), p->T, p->top_k, p->H,
                               xs, s, true);
  });
}

int mlp_moe_dispatch_bwd(const mlp_moe_t* p, const void* plan, const void* dxs, void* dx,
                         void* stream) {
  MLP_TRY(check_moe(p));
  MLP_TRY(need(plan));
  MLP_TRY(need(dxs));
  MLP_TRY(need(dx));
  if (dx == dxs) return MLP_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(MLP_KERNEL_MOE_COMBINE, s, [&] {
    return launch_moe_combine(dxs, false, static_cast<const int*>(plan), plan_of(p), p->T, p->top_k, p->H,
                              nullptr, false, nullptr, dx, s, true);
  });
}

int mlp_moe_combine(const mlp_moe_t* p, const void* plan, const void* y, const void* weights,
                    const void* residual, void* out, void* stream) {
  MLP_TRY(check_moe(p));
  MLP_TRY(need(plan));
  MLP_TRY(need(y));
  MLP_TRY(need_w(p, weights));
  MLP_TRY(opt(residual));
  MLP_TRY(need(out));
  if (out == y) return MLP_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(MLP_KERNEL_MOE_COMBINE, s, [&] {
    return launch_moe_combine(y, false, static_cast<const int*>(plan), plan_of(p), p->T, p->top_k, p->H,
                              weights, w_bf16(p), residual, out, s, true);
  });
}

int mlp_moe_combine_bwd(const mlp_moe_t* p, const void* plan, const void* dout, const void* y,
                        const void* weights, void* dy, void* dweights, void* stream) {
  MLP_TRY(check_moe(p));
  MLP_TRY(need(plan));
  MLP_TRY(need(dout));
  if (dy) {
    MLP_TRY(need(dy));
    MLP_TRY(need_w(p, weights));
  }
  if (dweights) {
    MLP_TRY(need_w(p, dweights));
    MLP_TRY(need(y));
  }
  if (!dy && !dweights) return MLP_OK;
  if (dy && (dy == dout || (dweights && dy == y))) return MLP_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return traced(MLP_KERNEL_MOE_COMBINE_BWD, s, [&] {
    return launch_moe_combine_bwd(dout, y, static_cast<const int*>(plan), plan_of(p), p->T,
                                  p->top_k, p->H, weights, w_bf16(p), dy, dweights, s, true);
  });
}

size_t mlp_moe_workspace_size(const mlp_moe_t* p, int mode) {
  if (check_experts(p) != MLP_OK) return 0;
  if (mode != MLP_MODE_FWD && mode != MLP_MODE_BWD && mode != MLP_MODE_INFER) return 0;
  return layout(p, mode).total;
}

int mlp_moe_experts_fwd(const mlp_moe_t* p, void* plan, const void* xs, const void* Wg,
                        const void* Wu, const void* Wd, void* y, void* G_save, void* U_save,
                        void* ws, size_t ws_bytes, void* stream) {
  MLP_TRY(check_experts(p));
  MLP_TRY(need(plan));
  MLP_TRY(need(xs));
  MLP_TRY(check_weights(p, Wg, Wu, Wd));
  MLP_TRY(need(y));
  MLP_TRY(opt(G_save));
  MLP_TRY(opt(U_save));
  if (!gated(p) && U_save) return MLP_ERR_INVALID_ARG;
  MLP_TRY(check_ws(p, MLP_MODE_FWD, ws, ws_bytes));
  if (y == xs) return MLP_ERR_INVALID_ARG;  // (few slots: y is written while xs is read)
  Call c;
  if (fwd_one_wave(p)) begin_one_wave(c, ws, stream);
  else MLP_TRY(begin_call(c, ws, stream));
  void* a = static_cast<char*>(ws) + layout(p, MLP_MODE_FWD).inter;
  int* pl = static_cast<int*>(plan);
  if (plan_of(p).fine >= 0)
    return launch_experts_fine(p, c, pl, xs, Wg, Wu, Wd, a, y, G_save, U_save);
  MLP_TRY(launch_experts_act(p, c, pl, xs, Wg, Wu, a, G_save, U_save));
  return launch_experts_down(p, c, pl, a, Wd, y, false);
}

int mlp_moe_experts_bwd(const mlp_moe_t* p, const void* plan, const void* dy, const void* xs,
                        const void* Wg, const void* Wu, const void* Wd, void* G, void* U,
                        void* dxs, void* dWg, void* dWu, void* dWd, int fuse_grad_accum, void* ws,
                        size_t ws_bytes, void* stream) {
  MLP_TRY(check_experts(p));
  if (fuse_grad_accum != 0 && fuse_grad_accum != 1) return MLP_ERR_INVALID_ARG;
  MLP_TRY(need(plan));
  MLP_TRY(need(dy));
  MLP_TRY(need(xs));
  MLP_TRY(check_weights(p, Wg, Wu, Wd));
  MLP_TRY(need(G));
  const bool gt = gated(p);
  if (gt) {
    MLP_TRY(need(U));
  } else if (U || dWu) {
    return MLP_ERR_INVALID_ARG;
  }
  MLP_TRY(opt(dxs));
  MLP_TRY(opt(dWg));
  MLP_TRY(opt(dWu));
  MLP_TRY(opt(dWd));
  MLP_TRY(check_ws(p, MLP_MODE_BWD, ws, ws_bytes));
  const bool need_dact = dxs || dWg || dWu;
  if (!need_dact && !dWd) return MLP_OK;
  // the weight gradients still read dy and xs while dxs is stored
  if (dxs && ((dWd && dxs == dy) || ((dWg || dWu) && dxs == xs))) return MLP_ERR_INVALID_ARG;
  const int cgw = p->H > BM && p->I > BM ? moe_cg(p, MOE_PAIR_ROWS_W)
                                         : pick_cg(p->H < p->I ? p->H : p->I);
  const long long w_units = ((dWg ? 1 : 0) + (dWu ? 1 : 0)) * out_tiles(p->I, p->H, cgw) +
                            (dWd ? 1 : 0) * out_tiles(p->H, p->I, cgw);
  const int most = one_wave_units(moe_cg(p));
  Call c;
  if (need_dact && row_units(p, p->I, MMA_N) <= most && row_units(p, p->H, MMA_N) <= most &&
      w_units * p->E <= one_wave_units(cgw))
    begin_one_wave(c, ws, stream);
  else
    MLP_TRY(begin_call(c, ws, stream));
  void* a = static_cast<char*>(ws) + layout(p, MLP_MODE_BWD).inter;
  const int* pl = static_cast<const int*>(plan);
  const int rows = static_cast<int>(plan_of(p).rows);

  if (need_dact) {
    // dh = dy Wd; dG, dU over G, U, and the postact for dWd
    RowGemm g(p, c, pl);
    const int mA = g.rows_a(dy, p->H);
    const int mB = g.mnmajor_stack(Wd, p->E, p->H, p->I);
    Prob& P = g.add_rows(p->I, p->H, 0, MMA_N);
    P.l2a = L2_EVICT_LAST;
    P.mapA0 = mA;
    P.mapB0 = mB;
    P.in0 = G;
    P.in1 = U;
    g.output_rows(P, 0, G, rows, p->I);
    if (gt) {
      g.output_rows(P, 1, U, rows, p->I);
      g.output_rows(P, 2, dWd ? a : nullptr, rows, p->I);
      MLP_TRY((run_gated<EPI_DGATED, false, true, true>(g, c, MLP_KERNEL_DGATED)));
    } else {
      g.output_rows(P, 1, dWd ? a : nullptr, rows, p->I);
      MLP_TRY((run_nongated<EPI_DACT, false, true, true>(g, c, MLP_KERNEL_DGATED)));
    }
  } else {
    const bool pdl = c.pdl();
    MLP_TRY(traced(MLP_KERNEL_POSTACT, c.stream, [&] {
      return launch_postact(G, U, a, (long long)rows * p->I, device_act(p->act),
                            p->gate_mult * p->down_mult, c.stream, pdl);
    }));
  }

  // the input gradient, and the weight gradients beside it (mlp_bwd's reasons;
  // small ones after it: the events cost more than the overlap gives)
  const bool want_w = dWg || dWu || dWd;
  Side* side = (dxs && want_w && !c.one_wave && !g_trace_flag.load()) ? side_stream(c.stream) : nullptr;
  std::unique_lock<std::mutex> side_lk;
  if (side) {
    side_lk = std::unique_lock<std::mutex>(side->mu);
    MLP_TRY(cuda_err(cudaEventRecord(side->fork, c.stream)));
  }
  if (dxs) {
    RowGemm g(p, c, pl);
    const int mA0 = g.rows_a(G, p->I);
    const int mB0 = g.mnmajor_stack(Wg, p->E, p->I, p->H);
    int mA1 = 0, mB1 = 0;
    if (gt) {
      mA1 = g.rows_a(U, p->I);
      mB1 = g.mnmajor_stack(Wu, p->E, p->I, p->H);
    }
    Prob& P = g.add_rows(p->H, p->I, gt ? p->I : 0, MMA_N);
    P.l2a = L2_EVICT_LAST;
    P.l2b = L2_EVICT_FIRST;
    P.mapA0 = mA0;
    P.mapB0 = mB0;
    P.mapA1 = mA1;
    P.mapB1 = mB1;
    g.output_rows(P, 0, dxs, rows, p->H, Gemm::ROWS_WIDE);
    MLP_TRY((run<EPI_STORE_BF16, false, true, true>(g, c, MLP_KERNEL_DX)));
  }
  if (want_w) {
    Call cw = c;
    if (side) {
      cw.stream = side->stream;
      cw.launches = 0;  // its first kernel follows an event wait, not a kernel
      MLP_TRY(cuda_err(cudaStreamWaitEvent(side->stream, side->fork, 0)));
    }
    const int fuse = fuse_grad_accum;
    Gemm g(device_act(p->act), 1.f, cw.counter(), cw.status, cgw);
    g.p.offsets = pl + plan_of(p).offsets;
    g.p.rows = rows;
    struct W { const void* A; int m; const void* B; int n; void* out; };
    W list[3];
    int n = 0;
    if (dWg) list[n++] = {G, p->I, xs, p->H, dWg};
    if (dWu) list[n++] = {U, p->I, xs, p->H, dWu};
    if (dWd) list[n++] = {dy, p->H, a, p->I, dWd};
    for (int i = 0; i < n; ++i) {
      const int mA = g.mnmajor(list[i].A, rows, list[i].m);
      const int mB = g.mnmajor(list[i].B, rows, list[i].n);
      const int oW = g.output_stack(list[i].out, p->E, list[i].m, list[i].n, fuse != 0);
      Prob& P = g.add(list[i].m, list[i].n, BK, 0, MMA_N);  // K: each expert's rows
      g.p.total_units += P.units * (p->E - 1);
      P.units *= p->E;
      P.l2b = L2_EVICT_LAST;
      P.mapA0 = mA;
      P.mapB0 = mB;
      P.mapO[0] = oW;
    }
    if (fuse) MLP_TRY((run<EPI_ACCUM_F32, true, true, true>(g, cw, MLP_KERNEL_WGRAD)));
    else MLP_TRY((run<EPI_STORE_BF16, true, true, true>(g, cw, MLP_KERNEL_WGRAD)));
    if (side) {
      MLP_TRY(cuda_err(cudaEventRecord(side->join, side->stream)));
      MLP_TRY(cuda_err(cudaStreamWaitEvent(c.stream, side->join, 0)));
    }
  }
  return MLP_OK;
}

int mlp_moe_fwd_infer(const mlp_moe_t* p, const void* x, const int* ids, const void* weights,
                      const void* Wg, const void* Wu, const void* Wd, const void* residual,
                      void* out, void* ws, size_t ws_bytes, void* stream) {
  MLP_TRY(check_experts(p));
  MLP_TRY(need(x));
  MLP_TRY(need_ids(ids));
  MLP_TRY(need_w(p, weights));
  MLP_TRY(check_weights(p, Wg, Wu, Wd));
  MLP_TRY(opt(residual));
  MLP_TRY(need(out));
  MLP_TRY(check_ws(p, MLP_MODE_INFER, ws, ws_bytes));
  const Layout w = layout(p, MLP_MODE_INFER);
  const MoePlan L = plan_of_infer(p);
  char* base = static_cast<char*>(ws);
  int* plan = reinterpret_cast<int*>(base + w.plan);
  void *a = base + w.inter, *xs = base + w.xs, *y = base + w.y;
  const bool stream_weights = decode_moe(p);  // (clears the status word itself)
  Call c;
  if (stream_weights || fwd_one_wave(p)) begin_one_wave(c, ws, stream, !stream_weights);
  else MLP_TRY(begin_call(c, ws, stream));
  bool pdl = c.pdl();
  if (stream_weights) {
    MLP_TRY(traced(MLP_KERNEL_GATE_UP, c.stream, [&] {
      return launch_moe_decode_act(x, ids, Wg, Wu, Wd, a, p->T, p->top_k, p->E, p->H, p->I,
                                   device_act(p->act), gated(p), p->gate_mult * p->down_mult,
                                   c.stream, pdl, c.status);
    }));
    pdl = c.pdl();
    return traced(MLP_KERNEL_DOWN, c.stream, [&] {
      return launch_moe_decode_down(a, ids, weights, w_bf16(p), Wd, residual, out, p->T, p->top_k,
                                    p->E, p->H, p->I, c.stream, pdl);
    });
  }
  MLP_TRY(traced(MLP_KERNEL_MOE_SORT, c.stream,
                 [&] { return launch_moe_sort(ids, plan, L, p->E, c.stream, pdl); }));
  pdl = c.pdl();
  MLP_TRY(traced(MLP_KERNEL_MOE_DISPATCH, c.stream, [&] {
    return launch_moe_dispatch(x, plan, L, p->T, p->top_k, p->H, xs, c.stream, pdl);
  }));
  MLP_TRY(launch_experts_act(p, c, plan, xs, Wg, Wu, a, nullptr, nullptr));
  MLP_TRY(launch_experts_down(p, c, plan, a, Wd, y, true));
  pdl = c.pdl();
  return traced(MLP_KERNEL_MOE_COMBINE, c.stream, [&] {
    return launch_moe_combine(y, true, plan, L, p->T, p->top_k, p->H, weights, w_bf16(p), residual, out,
                              c.stream, pdl);
  });
}

}  // extern "C"
