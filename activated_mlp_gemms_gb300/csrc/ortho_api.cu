// ortho_api.cu -- the C entry points of mlp_ortho.h: argument validation, workspace layout
// and the launch sequence.
#include "mlp_ortho.h"

#include "host.h"
#include "ortho.h"

using namespace mlpk;

namespace {

int check_ortho(const mlp_ortho_t* p) {
  if (!p) return MLP_ERR_INVALID_ARG;
  if (p->rows <= 0 || p->cols <= 0 || p->batch <= 0) return MLP_ERR_INVALID_ARG;
  if (p->steps < 1 || p->steps > 32) return MLP_ERR_INVALID_ARG;
  for (float c : p->coeff)
    if (!std::isfinite(c)) return MLP_ERR_INVALID_ARG;
  if (!std::isfinite(p->eps) || p->eps < 0.f || !std::isfinite(p->scale))
    return MLP_ERR_INVALID_ARG;
  auto type = [](int t) { return t == MLP_ORTHO_F32 || t == MLP_ORTHO_BF16; };
  if (!type(p->type) || !type(p->out_type)) return MLP_ERR_INVALID_ARG;
  if (p->rows % 8 || p->cols % 8) return MLP_ERR_ALIGNMENT;
  // one side up to 32768 (the symmetric products' units and fp16's range), the grids' limits
  const long long m = p->rows < p->cols ? p->rows : p->cols;
  const long long n = p->rows < p->cols ? p->cols : p->rows;
  if (m > 32768 || n > (1 << 21) || p->batch > 65535 || m * n * p->batch > (1LL << 36))
    return MLP_ERR_UNSUPPORTED;
  const long long tm = (m + 127) / 128, tn = (n + 127) / 128;
  if (tm * tn * p->batch >= (1LL << 31)) return MLP_ERR_UNSUPPORTED;
  return MLP_OK;
}

// After the control block (of which only the status word is used): the norms' partial sums, X
// in two terms twice, and P = b A + c A A and A in one term or two.  Their rows begin at multiples
// of 128 bytes: boxes of rows that straddle L2's lines took 1.5-1.8 times as long (3000 x 3000).
//
// Up to 128 rows P X takes both terms of both for a bf16 result, too, as in the one launch: the
// result is as exact whichever way a matrix goes, alone or in a stack, and K is two k-blocks at
// most (16 x 128 x 2048 2.8e-3 -> 2.0e-3 off, 125 -> 138 us; 1 x 128 x 2056 2.7e-3 -> 1.9e-3, 97 ->
// 111; 1 x 64 x 4096 2.5e-3 -> 1.7e-3, 101 -> 107).  P's second term then goes over A, which lies
// behind P.  A is one tile there: all of it has been multiplied before any of P is stored, and
// the boxes of it that are added to P are read by the warp that stores there, before it does.
struct Layout {
  int m, n, terms, p_terms;  // terms: of A, and of the products' operands but P X's
  int mp, np;                // row pitches of A and P, and of X
  size_t part, x[2], poly, a, total;
};
Layout layout(const mlp_ortho_t* p) {
  Layout w;
  w.m = p->rows < p->cols ? p->rows : p->cols;
  w.n = p->rows < p->cols ? p->cols : p->rows;
  w.terms = p->out_type == MLP_ORTHO_F32 ? 2 : 1;
  w.p_terms = w.terms == 2 || w.m <= ORTHO_SMALL_M ? 2 : 1;
  w.mp = (w.m + 63) / 64 * 64;
  w.np = (w.n + 63) / 64 * 64;
  const size_t x = round256((size_t)p->batch * w.m * w.np * 4);
  const size_t a = round256((size_t)p->batch * w.m * w.mp * 2 * w.terms);
  size_t at = CTRL_BYTES;
  w.part = at;
  at += round256((size_t)p->batch * ORTHO_PARTS * 4);
  w.x[0] = at;
  w.x[1] = at + x;
  w.poly = at + 2 * x;
  w.a = w.poly + a;  // (m is a multiple of 8, mp of 64: nothing between them)
  w.total = w.a + a;
  return w;
}

// Products run on CTA pairs (256 x 256 tiles) unless the singles' 128 x 128 fill the GPU that
// much better: a wave of 76 pairs takes 1.3 times one of 152 singles, for twice the work
// (their tiles load half as much for a flop).  Measured (pairs / singles, us): 4096 x 14336 step
// 299 / 460, 16 x 1408 x 2048 step 118 / 155, gram 64 / 74; 2048 x 4864 step 37 / 49, gram 33 /
// 29; 1024 x 1024 16 / 12.
int pick(const OrthoGemm& g, bool sym) {
  const int pol = g_tile_policy.load();
  if (pol == 1 || pol == 2) return pol;
  auto waves = [&](int tile, int slots) {
    const long long tm = (g.M + tile - 1) / tile, tn = (g.N + tile - 1) / tile;
    const long long units = (sym ? tm * (tm + 1) / 2 : tm * tn) * g.batch;
    return (units + slots - 1) / slots;
  };
  return 1.3 * waves(256, 76) <= waves(128, 152) ? 2 : 1;
}

// CTAs that share the k-blocks of a 128 x 128 tile where the tiles are few (1: none do).  The
// least estimate in us: 0.27 a k-block of one CTA (its loads' latency over the stages in
// flight), and 3.2 + 0.3 a CTA for the cluster's launch, its two barriers and the exchange of
// the sums.  Measured (1 / 2 / 4 / 8 CTAs, us of an X X^T with 5 of event time): 64 x 1024 10 / 12 /
// 12 / 12, 64 x 2048 16 / 14 / 12 / 13, 64 x 4096 24 / 18 / 14 / 14, 256 x 14336 65 / 43 / 27 / 20,
// 1024 x 2048 16 / 18 / 16 / 35 (more CTAs than SMs).
double share_us(int share, int kblocks, int products) {
  return 0.27 * products * ((kblocks + share - 1) / share) + (share > 1 ? 3.2 + 0.3 * share : 0.);
}
int pick_share(int units, int kblocks, int products) {
  int best = 1;
  for (int share = 2; share <= 8 && units * share <= 144; share *= 2)
    if (share_us(share, kblocks, products) < share_us(best, kblocks, products)) best = share;
  return best;
}

// Whether two CTA pairs share the k-blocks of a symmetric product's 256 x 256 tiles: these are
// too few for the GPU's pairs, and singles with their 128 x 128 ones load twice as much for a
// flop.  At most one wave of such clusters (36 on this GPU); 0.14 us a k-block and 12 for the
// cluster's launch and the exchange of half a tile's sums, with three products 0.2 and 5 (the
// singles' own epilogues are longer, too).  Measured (pairs / singles or clusters of them, us of
// an X X^T with 5 of event time): 2048 x 14336 51 / 69, 1536 x 8192 35 / 43, 2048 x 4864 31 / 29,
// 1024 x 4096 25 / 17; for an fp32 result 145 / 201, 80 / 117, 57 / 75, 49 / 26; 2048 x 2048 37 / 37.
bool share_pairs(const OrthoGemm& g) {
  if (g_tile_policy.load() != 0 || g.kblocks < 2) return false;
  const long long t = (g.M + 255) / 256, s = (g.M + 127) / 128;
  if (t * (t + 1) / 2 * g.batch > ortho_pairs_clusters()) return false;
  const int products = g.terms == 2 ? 3 : 1, units = static_cast<int>(s * (s + 1) / 2) * g.batch;
  const double us = products == 3 ? 0.6 * g.kblocks + 5 : 0.14 * g.kblocks + 12;
  return us < share_us(pick_share(units, g.kblocks, products), g.kblocks, products);
}

// Columns a CTA where the whole call runs on one cluster a matrix (0: it does not): what fits
// its shared memory, X in two terms and A in `terms`, P in two, and at most one wave of such
// clusters (15 of eight CTAs are resident together), two up to 64 rows.  Measured, five steps in us
// (one launch / a launch a product): 64 x 1024 33 / 90, 64 x 2048 45 / 98, 128 x 2048 76 / 109, 128 x
// 128 34 / 85; fp32 results 64 x 1024 45 / 107, 128 x 1024 76 / 125; two waves, 30 x 64 x 1024 70 / 114,
// 16 x 128 x 2048 155 / 138, 30 x 128 x 1024 133 / 130.
int small_width(const mlp_ortho_t* p, const Layout& w) {
  if (g_tile_policy.load() != 0 || w.m > ORTHO_SMALL_M) return 0;
  const int width = w.n <= 128 * ORTHO_SMALL_CTAS ? 128 : w.terms == 1 ? 256 : 0;
  int ctas = 1;
  while (ctas * width < w.n && ctas <= ORTHO_SMALL_CTAS) ctas *= 2;
  if (width == 0 || ctas > ORTHO_SMALL_CTAS) return 0;
  const long long waves = ((long long)p->batch * ctas + 119) / 120;
  return waves <= (w.m <= 64 ? 2 : 1) ? width : 0;
}

// k-blocks of a leading product that one accumulator sums up where both terms are taken (the
// tensor cores truncate it at every instruction).  X X^T and A A half as long: their errors are
// stretched by two more products and one.  Up to 512 rows, whose own error is small, one and
// two, so that an fp32 result is as exact as with products of fp32; above, where it grows by the
// sums' length, four and eight are, for 5-20 % less time.  Measured (off by and us, short / long;
// products of fp32): 256 x 14336 2.2e-6, 331 / 7.6e-6, 291; 2.0e-6 -- 256 x 512 1.7e-6, 147 / 5.7e-6,
// 140; 2.2e-6 -- 4 x 512 x 1408 2.0e-6, 274 / 5.8e-6, 247; 3.2e-6 -- 640 x 4096 2.1e-6, 270 / 4.9e-6, 251;
// 3.7e-6 -- 4864 x 2048 1.6e-6, 1030 / 4.7e-6, 844; 5.0e-6.
int chunk_of(int m, bool sym) { return (m <= 512 ? 2 : 8) / (sym ? 2 : 1); }

struct Products {
  const mlp_ortho_t* p;
  Layout w;
  cudaStream_t stream;
  int* status;
  bool ok = true;
  // Each product walks over the stack against the one before it, whose last results are still in
  // L2.
  bool backwards = false;

  // A stack [depth, rows, cols] of fp16 (or bf16, fp32) matrices in boxes {c, r}.
  CUtensorMap map(const void* ptr, int depth, int rows, int cols, int pitch, int c, int r,
                  CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B, int f32 = 0) {
    CUtensorMap m;
    if (!make_map(&m, ptr, cols, rows, pitch, c, r, f32, swz, depth, (uint64_t)rows * pitch))
      ok = false;
    return m;
  }
  // ... in the boxes of the epilogue
  CUtensorMap boxes(const void* ptr, int depth, int rows, int cols, int pitch) {
    return map(ptr, depth, rows, cols, pitch, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  }
  OrthoGemm gemm(int M, int N, int K) {
    OrthoGemm g;
    std::memset(&g, 0, sizeof(g));
    g.M = M;
    g.N = N;
    g.kblocks = (K + 63) / 64;
    g.terms = g.d_terms = w.terms;
    g.batch = p->batch;
    g.status = status;
    g.timeout_ns = wait_limit_ns();
    g.debug_flags = g_debug_flags.load();
    return g;
  }
  int run(OrthoGemm& g, OrthoKind kind, int tag) {
    if (!ok) return MLP_ERR_CUDA;
    const bool sym = kind == ORTHO_SYM;
    g.chunk = chunk_of(g.M, sym);
    g.backwards = backwards;
    backwards = !backwards;
    if (sym && share_pairs(g)) {
      g.tiles_m = g.tiles_n = (g.M + 255) / 256;
      g.units = g.tiles_m * (g.tiles_m + 1) / 2 * g.batch;
      return traced(tag, stream, [&] { return launch_ortho_pairs(g, stream); });
    }
    const int cg = pick(g, sym), tile = 128 * cg;
    g.tiles_m = (g.M + tile - 1) / tile;
    g.tiles_n = (g.N + tile - 1) / tile;
    g.units = (sym ? g.tiles_m * (g.tiles_m + 1) / 2 : g.tiles_m * g.tiles_n) * g.batch;
    const int share =
        cg == 1 && g_tile_policy.load() != 1 ? pick_share(g.units, g.kblocks, g.terms == 2 ? 3 : 1)
                                           : 1;
    if (share > 1 && g.chunk > 4) g.chunk = 4;  // (a CTA's slice is short)
    return traced(tag, stream, [&] {
      return share > 1 ? launch_ortho_split(g, share, kind, stream)
                       : launch_ortho_gemm(g, cg, kind, stream);
    });
  }
};

}  // namespace

extern "C" {

size_t mlp_ortho_workspace_size(const mlp_ortho_t* p) {
  return check_ortho(p) == MLP_OK ? layout(p).total : 0;
}

int mlp_orthogonalize(const mlp_ortho_t* p, const void* G, void* out, void* ws, size_t ws_bytes,
                      void* stream) {
  MLP_TRY(check_ortho(p));
  MLP_TRY(need(G));
  MLP_TRY(need(out));
  if (out == G && p->type != p->out_type) return MLP_ERR_INVALID_ARG;
  if (!ws) return MLP_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return MLP_ERR_ALIGNMENT;
  const Layout w = layout(p);
  if (ws_bytes < w.total) return MLP_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* at = static_cast<char*>(ws);
  float* part = reinterpret_cast<float*>(at + w.part);
  const bool bf16 = p->type == MLP_ORTHO_BF16;
  if (const int width = small_width(p, w)) {
    const OrthoSmall g{G,
                       out,
                       w.m,
                       w.n,
                       p->batch,
                       p->steps,
                       w.terms,
                       p->rows > p->cols,
                       bf16,
                       p->out_type == MLP_ORTHO_BF16,
                       p->coeff[0],
                       p->coeff[1],
                       p->coeff[2],
                       p->eps,
                       p->scale,
                       static_cast<int*>(ws),
                       wait_limit_ns(),
                       g_debug_flags.load()};
    return traced(MLP_KERNEL_ORTHO_STEP, s, [&] { return launch_ortho_small(g, width, s); });
  }
  MLP_TRY(traced(MLP_KERNEL_ORTHO_SCALE, s, [&] {
    return launch_ortho_norm(G, bf16, (long long)w.m * w.n, p->batch, part,
                             static_cast<int*>(ws), s);
  }));
  MLP_TRY(traced(MLP_KERNEL_ORTHO_SCALE, s, [&] {
    return launch_ortho_scale(G, bf16, p->rows, p->cols, p->batch, w.np, part, p->eps,
                              at + w.x[0], s);
  }));
  Products run{p, w, s, static_cast<int*>(ws)};
  const int m = w.m, n = w.n;  // and the depths of X, A and P:
  const int xs = 2 * p->batch, as = w.terms * p->batch, ps = w.p_terms * p->batch;
  char *A = at + w.a, *P = at + w.poly;
  for (int i = 0; i < p->steps; ++i) {
    char *X = at + w.x[i & 1], *next = at + w.x[(i & 1) ^ 1];
    {
      OrthoGemm g = run.gemm(m, m, n);
      g.p = g.q = run.map(X, xs, m, n, w.np, 64, 128);
      g.in = g.d = run.boxes(A, as, m, m, w.mp);
      g.d_ptr = A;
      g.ld_d = w.mp;
      g.beta = ORTHO_A / (ORTHO_X * ORTHO_X);
      MLP_TRY(run.run(g, ORTHO_SYM, MLP_KERNEL_ORTHO_GRAM));
    }
    {
      OrthoGemm g = run.gemm(m, m, m);
      g.p = g.q = run.map(A, as, m, m, w.mp, 64, 128);
      g.in = run.boxes(A, as, m, m, w.mp);
      g.d = run.boxes(P, ps, m, m, w.mp);
      g.d_terms = w.p_terms;
      g.in_ptr = A;
      g.d_ptr = P;
      g.ld_in = g.ld_d = w.mp;
      g.alpha = p->coeff[1];
      g.beta = p->coeff[2] / ORTHO_A;
      MLP_TRY(run.run(g, ORTHO_SYM, MLP_KERNEL_ORTHO_POLY));
    }
    OrthoGemm g = run.gemm(m, n, m);
    g.terms = w.p_terms;
    g.p = run.map(P, ps, m, m, w.mp, 64, 128);
    g.q = run.map(X, xs, m, n, w.np, 64, 64);
    g.in = run.boxes(X, xs, m, n, w.np);
    g.in_ptr = X;
    g.d_ptr = i + 1 < p->steps ? next : out;
    g.ld_in = w.np;
    g.ld_d = i + 1 < p->steps ? w.np : p->cols;
    g.alpha = p->coeff[0];
    g.beta = 1.f / ORTHO_A;
    if (i + 1 < p->steps) {
      g.d = run.boxes(next, xs, m, n, w.np);
      MLP_TRY(run.run(g, ORTHO_STEP, MLP_KERNEL_ORTHO_STEP));
      continue;
    }
    const float scale = p->scale / ORTHO_X;
    g.alpha *= scale;
    g.beta *= scale;
    g.out_bf16 = p->out_type == MLP_ORTHO_BF16;
    g.transposed = p->rows > p->cols;
    g.d = g.out_bf16 ? run.boxes(out, p->batch, p->rows, p->cols, p->cols)
                     : run.map(out, p->batch, p->rows, p->cols, p->cols, 32, 32,
                               CU_TENSOR_MAP_SWIZZLE_128B, 1);
    MLP_TRY(run.run(g, ORTHO_LAST, MLP_KERNEL_ORTHO_STEP));
  }
  return MLP_OK;
}

}  // extern "C"
