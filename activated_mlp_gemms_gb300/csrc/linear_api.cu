// linear_api.cu -- the C entry points of mlp_linear.h: argument validation,
// workspace layout and launch sequences.
//   mlp_linear_fwd   one kernel with the bias / activation / residual epilogue: the
//                    weight stream, the skinny kernel or the GEMM (route)
//   mlp_linear_bwd   dz = dout act'(z) and the bias gradient's partial sums in
//                    one pass (no activation: only those sums, dz is dout),
//                    dx = dz W, and dW = dz^T x on the second stream beside it
#include "mlp_linear.h"

#include "host.h"
#include "linear.h"

using namespace mlpk;

namespace {

int check_linear(const mlp_linear_t* p) {
  if (!p) return MLP_ERR_INVALID_ARG;
  if (p->M <= 0 || p->N <= 0 || p->K <= 0) return MLP_ERR_INVALID_ARG;
  if (p->act < MLP_LINEAR_NONE || p->act > MLP_LINEAR_SIGMOID) return MLP_ERR_INVALID_ARG;
  if (!std::isfinite(p->resid_scale)) return MLP_ERR_INVALID_ARG;
  auto pitch = [](int ld, int row) { return ld == 0 || ld >= row; };
  if (!pitch(p->ldx, p->K) || !pitch(p->ldr, p->N) || !pitch(p->ldo, p->N))
    return MLP_ERR_INVALID_ARG;
  if (p->N % 8 || p->K % 8 || p->ldx % 8 || p->ldr % 8 || p->ldo % 8) return MLP_ERR_ALIGNMENT;
  if ((long long)p->M * p->N >= (1LL << 40) || (long long)p->M * p->K >= (1LL << 40))
    return MLP_ERR_UNSUPPORTED;
  // rows and columns rounded up to whole tiles are 32-bit
  constexpr int MOST = 0x7fffffff - 1023;
  if (p->M > MOST || p->N > MOST || p->K > MOST) return MLP_ERR_UNSUPPORTED;
  return MLP_OK;
}

int linear_act(int act) {
  switch (act) {
    case MLP_LINEAR_RELU: return ACT_RELU;
    case MLP_LINEAR_RELU_SQ: return ACT_RELU_SQ;
    case MLP_LINEAR_GELU_TANH: return ACT_GELU_EXP;
    case MLP_LINEAR_SILU: return ACT_SILU_EXP;
    case MLP_LINEAR_SIGMOID: return ACT_SIGMOID_EXP;
    default: return ACT_NONE;
  }
}

// Which kernel a product [M, N] over K runs as: 128 x 256 tiles of single CTAs, 256
// x 256 tiles of CTA pairs, or the skinny kernel's 128 features by up to 256 rows
// with K shared by clusters.  (A tile policy of 1 or 2 asks for the first two.)
// The least of three estimates, in units of one 256 x 256 k-block of a pair (0.33 us),
// from the start of a single-CTA launch on: a pair's launch costs 4 more than that;
// single-CTA MMAs draw more shared-memory bandwidth per flop, 13 % of the time; a
// skinny tile of mp rows takes (160 + mp) / 400 of a k-block, its CTAs, which are not
// persistent, 6 a wave and mp / 50 for their end, the exchange of the sums mp / 20,
// and its start 6 less (2 for dx, whose tiles have the shorter epilogue).  Rows that
// are no multiple of 128 bytes straddle L2 lines, and those MMAs' larger share of
// loads costs 40 %.  Measured (skinny / singles / pairs, us): 128 x 768 x 768 7.7 /
// 8.6 / 9.0, 192 x 768 x 768 9.3 / 8.5 / 8.9, 192 x 1024 x 1024 9.0 / 9.5 / 10, 300 x
// 4096 x 4096 16.5 / 27 / 25, 512 x 2048 x 8192 22.8 / 27.6 / 28.5, 777 x 14336 x 4096
// 76 / 78 / 69, 777 x 4864 x 2048 16.5 / 15.7 / 16.6, 1000 x 1024 x 1024 11.2 / 10.0 /
// 10.4.
enum Route { ROUTE_SINGLES = 1, ROUTE_PAIRS = 2, ROUTE_SKINNY = 3 };
Route route(int M, int N, int K, bool whole_lines, bool forward) {
  const int pol = g_tile_policy.load();
  if (pol == 1 || pol == 2) return static_cast<Route>(pol);
  const SkinnyShape s = linear_skinny_shape(M, N, K);
  const double kbs = (K + BK - 1) / BK, loads = whole_lines ? 1.13 : 1.4;
  auto waves = [](long long units, int slots) { return (double)((units + slots - 1) / slots); };
  const double pairs = waves(out_tiles(M, N, 2), 76) * kbs + 5;
  const double singles = loads * waves(out_tiles(M, N, 1), 152) * kbs + 1;
  const double skinny = waves((long long)s.blocks * s.tiles * s.share, 152) *
                            (loads * kbs / s.share * (160 + s.mp) / 400 + 6 + 0.02 * s.mp) +
                        (s.share > 1 ? 0.05 * s.mp : 0) - (forward ? 6 : 2);
  if (skinny < pairs && skinny < singles) return ROUTE_SKINNY;
  return singles < pairs ? ROUTE_SINGLES : ROUTE_PAIRS;
}

// The workspace after the control block: the backward's dz and the bias
// gradient's partial sums.
struct Layout {
  size_t dz, db, total;
};
Layout layout(const mlp_linear_t* p, bool backward) {
  Layout L = {};
  size_t at = CTRL_BYTES;
  L.dz = at;
  if (backward && p->act != MLP_LINEAR_NONE) at += round256((size_t)p->M * p->N * 2);
  L.db = at;
  if (backward) at += round256((size_t)linear_db_chunks(p->M, p->N) * p->N * 4);
  L.total = at;
  return L;
}

int check_ws(const Layout& L, const void* ws, size_t ws_bytes) {
  if (!ws) return MLP_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return MLP_ERR_ALIGNMENT;
  return ws_bytes < L.total ? MLP_ERR_WORKSPACE_TOO_SMALL : MLP_OK;
}

template <int ACT>
int run_linear(Gemm& g, Call& c) {
  return run_act<EPI_LINEAR, false, false, ACT>(g, c, MLP_KERNEL_LINEAR);
}

}  // namespace

extern "C" {

size_t mlp_linear_workspace_size(const mlp_linear_t* p, int backward) {
  if (check_linear(p) != MLP_OK || (backward != 0 && backward != 1)) return 0;
  return layout(p, backward == 1).total;
}

int mlp_linear_fwd(const mlp_linear_t* p, const void* x, const void* W, const void* bias,
                   const void* residual, void* out, void* pre_save, void* ws, size_t ws_bytes,
                   void* stream) {
  MLP_TRY(check_linear(p));
  MLP_TRY(need(x));
  MLP_TRY(need(W));
  MLP_TRY(opt(bias));
  MLP_TRY(opt(residual));
  MLP_TRY(need(out));
  MLP_TRY(opt(pre_save));
  // other tiles still read x when a tile of out is stored
  if (out == x || pre_save == x || pre_save == out) return MLP_ERR_INVALID_ARG;
  const Layout L = layout(p, false);
  MLP_TRY(check_ws(L, ws, ws_bytes));
  const int M = p->M, N = p->N, K = p->K, act = linear_act(p->act);
  const int ldx = p->ldx ? p->ldx : K, ldr = p->ldr ? p->ldr : N, ldo = p->ldo ? p->ldo : N;
  const bool streamed = M <= LINEAR_STREAM_MAX_M;
  const Route way = streamed ? ROUTE_SKINNY : route(M, N, K, ldx % 64 == 0 && K % 64 == 0, true);
  const bool tiles = way != ROUTE_SKINNY;
  Call c;
  // (one wave of tiles: 22.7 -> 18.9 us for 777 x 4864 x 2048; the stream and the
  // skinny kernel use no counter and clear the status word themselves)
  if (!tiles || out_tiles(M, N, way) <= one_wave_units(way)) begin_one_wave(c, ws, stream, tiles);
  else MLP_TRY(begin_call(c, ws, stream));
  if (streamed) {
    const bool pdl = c.pdl();
    return traced(MLP_KERNEL_LINEAR, c.stream, [&] {
      return launch_linear_stream(x, ldx, W, bias, residual, ldr, p->resid_scale, out, ldo,
                                  pre_save, M, N, K, act, c.stream, pdl, c.status);
    });
  }
  if (!tiles) {
    CUtensorMap map_w, map_x;
    if (!make_map(&map_w, W, K, N, K, BK, 128) ||
        !make_map(&map_x, x, K, M, ldx, BK, linear_skinny_shape(M, N, K).mp))
      return MLP_ERR_CUDA;
    const bool pdl = c.pdl();
    return traced(MLP_KERNEL_LINEAR, c.stream, [&] {
      return launch_linear_skinny(map_w, map_x, bias, residual, ldr, p->resid_scale, out, ldo,
                                  pre_save, M, N, K, act, false, true,
                                  g_debug_flags.load() & MLP_DEBUG_NO_WORK, c.status,
                                  wait_limit_ns(), c.stream, pdl);
    });
  }
  Gemm g(act, 1.f, c.counter(), c.status, way);
  const int mA = g.kmajor_a(x, M, K, ldx);
  const int mB = g.kmajor(W, N, K, g.b_rows());
  const int oO = g.output(out, M, N, false, ldo);
  const int oZ = g.output(pre_save, M, N);
  Prob& P = g.add(M, N, K, 0, MMA_N);
  P.l2a = L2_EVICT_LAST;
  P.l2b = L2_EVICT_FIRST;
  P.mapA0 = mA;
  P.mapB0 = mB;
  P.mapO[0] = oO;
  P.mapO[1] = oZ;
  P.in0 = residual;
  P.in1 = bias;
  P.ld = ldr;
  P.alpha = p->resid_scale;
  switch (act) {
    case ACT_RELU: return run_linear<ACT_RELU>(g, c);
    case ACT_RELU_SQ: return run_linear<ACT_RELU_SQ>(g, c);
    case ACT_GELU_EXP: return run_linear<ACT_GELU_EXP>(g, c);
    case ACT_SILU_EXP: return run_linear<ACT_SILU_EXP>(g, c);
    case ACT_SIGMOID_EXP: return run_linear<ACT_SIGMOID_EXP>(g, c);
    default: return run_linear<ACT_NONE>(g, c);
  }
}

int mlp_linear_bwd(const mlp_linear_t* p, const void* dout, const void* x, const void* W,
                   const void* pre, void* dx, void* dW, void* db, int fuse_grad_accum, void* ws,
                   size_t ws_bytes, void* stream) {
  MLP_TRY(check_linear(p));
  if (fuse_grad_accum != 0 && fuse_grad_accum != 1) return MLP_ERR_INVALID_ARG;
  const int fuse = fuse_grad_accum;
  MLP_TRY(need(dout));
  MLP_TRY(dW ? need(x) : opt(x));
  MLP_TRY(dx ? need(W) : opt(W));
  const bool has_act = p->act != MLP_LINEAR_NONE;
  MLP_TRY(has_act ? need(pre) : opt(pre));
  MLP_TRY(opt(dx));
  MLP_TRY(opt(dW));
  MLP_TRY(opt(db));
  // dW still reads dout and x while dx is stored
  if (dx && (dx == dout || dx == x)) return MLP_ERR_INVALID_ARG;
  const Layout L = layout(p, true);
  MLP_TRY(check_ws(L, ws, ws_bytes));
  if (!dx && !dW && !db) return MLP_OK;
  const int M = p->M, N = p->N, K = p->K, act = linear_act(p->act);
  const int ldx = p->ldx ? p->ldx : K, ldd = p->ldo ? p->ldo : N;
  char* base = static_cast<char*>(ws);
  const Route way = route(M, K, N, ldd % 64 == 0 && K % 64 == 0, false);  // dx
  const bool skinny_dx = dx && way == ROUTE_SKINNY;
  const int cgx = skinny_dx ? 1 : way, cgw = pick_cg(N < K ? N : K);
  // dz_out or db: the derivative pass comes first and clears the status word
  const bool pass = (has_act && (dx || dW)) || db;
  Call c;
  if ((!dx || skinny_dx || out_tiles(M, K, cgx) <= one_wave_units(cgx)) &&
      (!dW || (!fuse && out_tiles(N, K, cgw) <= one_wave_units(cgw))))
    begin_one_wave(c, ws, stream, !pass);
  else
    MLP_TRY(begin_call(c, ws, stream));

  const void* dz = dout;
  int ldz = ldd;
  float* sums = reinterpret_cast<float*>(base + L.db);
  void* dz_out = has_act && (dx || dW) ? base + L.dz : nullptr;
  if (dz_out || db) {
    const bool pdl = c.pdl();
    MLP_TRY(traced(MLP_KERNEL_LINEAR_DACT, c.stream, [&] {
      return launch_linear_dact(dout, ldd, pre, dz_out, db ? sums : nullptr, db, fuse != 0, M, N,
                                act, c.one_wave ? c.status : nullptr, c.stream, pdl);
    }));
  }
  if (dz_out) {
    dz = dz_out;
    ldz = N;
  }

  // a single chunk of rows: the pass has written db itself
  const bool db_left = db && linear_db_chunks(M, N) > 1;
  // dW and db go to the second stream when dx runs too (mlp_bwd's reasons),
  // unless all are small: then the events cost more than the overlap gives
  Side* side = dx && (dW || db_left) && !c.one_wave && !g_trace_flag.load()
                   ? side_stream(c.stream) : nullptr;
  std::unique_lock<std::mutex> side_lk;
  if (side) {
    side_lk = std::unique_lock<std::mutex>(side->mu);
    MLP_TRY(cuda_err(cudaEventRecord(side->fork, c.stream)));
  }
  if (skinny_dx) {
    CUtensorMap map_w, map_z;
    if (!make_map(&map_w, W, K, N, K, 64, BK) ||
        !make_map(&map_z, dz, N, M, ldz, BK, linear_skinny_shape(M, K, N).mp))
      return MLP_ERR_CUDA;
    const bool pdl = c.pdl();
    MLP_TRY(traced(MLP_KERNEL_DX, c.stream, [&] {
      return launch_linear_skinny(map_w, map_z, nullptr, nullptr, 0, 0.f, dx, K, nullptr, M, K, N,
                                  ACT_NONE, true, c.clear_status,
                                  g_debug_flags.load() & MLP_DEBUG_NO_WORK, c.status,
                                  wait_limit_ns(), c.stream, pdl);
    }));
    c.clear_status = false;
  } else if (dx) {
    Gemm g(act, 1.f, c.counter(), c.status, cgx);
    const int mA = g.kmajor_a(dz, M, N, ldz);
    const int mB = g.mnmajor(W, N, K);  // W [N,K]: B(n=k, k=n) is contiguous along K
    const int oX = g.output(dx, M, K);
    Prob& P = g.add(M, K, N, 0, MMA_N);
    P.l2a = L2_EVICT_LAST;   // dz: re-read by every tile column
    P.l2b = L2_EVICT_FIRST;  // W
    P.mapA0 = mA;
    P.mapB0 = mB;
    P.mapO[0] = oX;
    MLP_TRY((run<EPI_STORE_BF16, false, true>(g, c, MLP_KERNEL_DX)));
  }
  if (dW || db_left) {
    Call cw = c;
    if (side) {
      cw.stream = side->stream;
      cw.launches = 0;  // its first kernel follows an event wait, not a kernel
      MLP_TRY(cuda_err(cudaStreamWaitEvent(side->stream, side->fork, 0)));
    }
    if (db_left) {
      const bool pdl = cw.pdl();
      MLP_TRY(traced(MLP_KERNEL_LINEAR_DB, cw.stream, [&] {
        return launch_linear_db(sums, linear_db_chunks(M, N), db, N, fuse != 0, cw.stream, pdl);
      }));
    }
    if (dW) {
      Gemm g(act, 1.f, cw.counter(), cw.status, cgw);
      const int mA = g.mnmajor(dz, M, N, ldz);
      const int mB = g.mnmajor(x, M, K, ldx);
      const int oW = g.output(dW, N, K, fuse != 0);
      Prob& P = g.add(N, K, M, 0, MMA_N, wgrad_split(M, out_tiles(N, K, g.cg), g.cg, fuse));
      P.l2b = L2_EVICT_LAST;  // x: shared by the tile rows
      P.mapA0 = mA;
      P.mapB0 = mB;
      P.mapO[0] = oW;
      if (fuse) MLP_TRY((run<EPI_ACCUM_F32, true, true>(g, cw, MLP_KERNEL_WGRAD)));
      else MLP_TRY((run<EPI_STORE_BF16, true, true>(g, cw, MLP_KERNEL_WGRAD)));
    }
    if (side) {
      MLP_TRY(cuda_err(cudaEventRecord(side->join, side->stream)));
      MLP_TRY(cuda_err(cudaStreamWaitEvent(c.stream, side->join, 0)));
    }
  }
  return MLP_OK;
}

}  // extern "C"
