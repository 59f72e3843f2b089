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
// in two terms twice, and A and P = b A + c A A in one term or two.
struct Layout {
  int m, n, terms;
  size_t part, x[2], a, poly, total;
};
Layout layout(const mlp_ortho_t* p) {
  Layout w;
  w.m = p->rows < p->cols ? p->rows : p->cols;
  w.n = p->rows < p->cols ? p->cols : p->rows;
  w.terms = p->out_type == MLP_ORTHO_F32 ? 2 : 1;
  const size_t x = round256((size_t)p->batch * w.m * w.n * 4);
  const size_t a = round256((size_t)p->batch * w.m * w.m * 2 * w.terms);
  size_t at = CTRL_BYTES;
  w.part = at;
  at += round256((size_t)p->batch * ORTHO_PARTS * 4);
  w.x[0] = at;
  w.x[1] = at + x;
  w.a = at + 2 * x;
  w.poly = w.a + a;
  w.total = w.poly + a;
  return w;
}

// Products run on CTA pairs (256 x 256 tiles) where their tiles fill the pairs at least as
// well as the singles' 128 x 128.
int pick(const OrthoGemm& g) {
  const int pol = g_tile_policy.load();
  if (pol == 1 || pol == 2) return pol;
  auto waves = [&](int tile, int slots) {
    const long long tm = (g.M + tile - 1) / tile, tn = (g.N + tile - 1) / tile;
    const long long units = (g.sym ? tm * (tm + 1) / 2 : tm * tn) * g.batch;
    return (units + slots - 1) / slots;
  };
  return 2 * waves(256, 76) <= waves(128, 152) + 1 ? 2 : 1;
}

struct Products {
  const mlp_ortho_t* p;
  Layout w;
  cudaStream_t stream;
  int* status;
  bool ok = true;

  // A stack [terms x batch, rows, cols] in boxes {64, box}.
  CUtensorMap map(const void* ptr, int rows, int cols, int terms, int box) {
    CUtensorMap m;
    if (!make_map(&m, ptr, cols, rows, cols, 64, box, 0, CU_TENSOR_MAP_SWIZZLE_128B,
                  (uint64_t)terms * p->batch, (uint64_t)rows * cols))
      ok = false;
    return m;
  }
  OrthoGemm gemm(int M, int N, int K, bool sym) {
    OrthoGemm g;
    std::memset(&g, 0, sizeof(g));
    g.M = M;
    g.N = N;
    g.kblocks = (K + 63) / 64;
    g.terms = w.terms;
    g.batch = p->batch;
    g.sym = sym;
    g.status = status;
    g.timeout_ns = wait_limit_ns();
    g.debug_flags = g_debug_flags.load();
    return g;
  }
  int run(OrthoGemm& g, bool q_mn, int tag) {
    if (!ok) return MLP_ERR_CUDA;
    const int cg = pick(g), tile = 128 * cg;
    g.tiles_m = (g.M + tile - 1) / tile;
    g.tiles_n = (g.N + tile - 1) / tile;
    g.units = (g.sym ? g.tiles_m * (g.tiles_m + 1) / 2 : g.tiles_m * g.tiles_n) * g.batch;
    return traced(tag, stream, [&] { return launch_ortho_gemm(g, cg, q_mn, stream); });
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
  const size_t mn = (size_t)p->batch * w.m * w.n, mm = (size_t)p->batch * w.m * w.m;
  MLP_TRY(traced(MLP_KERNEL_ORTHO_SCALE, s, [&] {
    return launch_ortho_norm(G, bf16, (long long)w.m * w.n, p->batch, part,
                             static_cast<int*>(ws), s);
  }));
  MLP_TRY(traced(MLP_KERNEL_ORTHO_SCALE, s, [&] {
    return launch_ortho_scale(G, bf16, p->rows, p->cols, p->batch, part, p->eps, at + w.x[0], s);
  }));
  Products run{p, w, s, static_cast<int*>(ws)};
  auto second = [&](void* first, size_t n) {  // of two terms
    return w.terms == 2 ? static_cast<char*>(first) + 2 * n : nullptr;
  };
  char *A = at + w.a, *P = at + w.poly;
  for (int i = 0; i < p->steps; ++i) {
    char *X = at + w.x[i & 1], *next = at + w.x[(i & 1) ^ 1];
    {
      OrthoGemm g = run.gemm(w.m, w.m, w.n, true);
      g.p = g.q = run.map(X, w.m, w.n, 2, 128);
      g.beta = ORTHO_A / (ORTHO_X * ORTHO_X);
      g.hi = A;
      g.lo = second(A, mm);
      MLP_TRY(run.run(g, false, MLP_KERNEL_ORTHO_GRAM));
    }
    {
      OrthoGemm g = run.gemm(w.m, w.m, w.m, true);
      g.p = g.q = run.map(A, w.m, w.m, w.terms, 128);
      g.alpha = p->coeff[1];
      g.beta = p->coeff[2] / ORTHO_A;
      g.in_hi = A;
      g.in_lo = second(A, mm);
      g.hi = P;
      g.lo = second(P, mm);
      MLP_TRY(run.run(g, false, MLP_KERNEL_ORTHO_POLY));
    }
    OrthoGemm g = run.gemm(w.m, w.n, w.m, false);
    g.p = run.map(P, w.m, w.m, w.terms, 128);
    g.q = run.map(X, w.m, w.n, 2, 64);
    g.alpha = p->coeff[0];
    g.beta = 1.f / ORTHO_A;
    g.in_hi = X;
    g.in_lo = X + 2 * mn;
    if (i + 1 < p->steps) {
      g.hi = next;
      g.lo = next + 2 * mn;
    } else {
      const float scale = p->scale / ORTHO_X;
      g.alpha *= scale;
      g.beta *= scale;
      g.out = out;
      g.out_bf16 = p->out_type == MLP_ORTHO_BF16;
      g.transposed = p->rows > p->cols;
    }
    MLP_TRY(run.run(g, true, MLP_KERNEL_ORTHO_STEP));
  }
  return MLP_OK;
}

}  // extern "C"
