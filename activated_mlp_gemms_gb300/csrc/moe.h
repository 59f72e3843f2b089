// moe.h -- the sorted layout of the mixture-of-experts calls, and the
// launchers of its kernels.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mlpk {

constexpr int MOE_ALIGN = 16;          // MLP_MOE_ROW_ALIGN
constexpr int MOE_MAX_EXPERTS = 1024;  // MLP_MOE_MAX_EXPERTS
constexpr int MOE_FINE_SLOTS = 64;     // MLP_MOE_FINE_SLOTS

// What a row tile of the experts' GEMMs (128 or 256 rows) belongs to: its
// expert's rows [row, end), whose tiles begin at tile `first`.
struct MoeTile {
  int expert, row, end, first;
};

// Where the parts of the plan are, in int32 values.
struct MoePlan {
  long long n, rows;                  // slots, rows of the sorted layout
  long long offsets, counts, ntiles;  // [E + 1], [E], [2] (128- and 256-row tiles)
  long long tiles[2];                 // MoeTile lists: 128 rows, 256 rows
  long long tile_cap[2];
  long long pos, src;
  // up to MOE_FINE_SLOTS slots: whether y's fp32 rows are there, and the rows
  // [rows, H] (-1: no room for them)
  long long fine_flag, fine;
  long long ints;
};

// H = 0: without the fp32 rows of y.
inline MoePlan moe_plan(int T, int E, int top_k, int H) {
  MoePlan L;
  L.n = static_cast<long long>(T) * top_k;
  const long long used = L.n < E ? L.n : E;
  L.rows = (L.n + used * (MOE_ALIGN - 1)) / MOE_ALIGN * MOE_ALIGN;
  auto r4 = [](long long v) { return (v + 3) / 4 * 4; };  // 16-byte parts
  L.offsets = 0;
  L.counts = r4(E + 1);
  L.ntiles = L.counts + r4(E);
  long long at = L.ntiles + 4;
  for (int h = 0; h < 2; ++h) {
    // an expert's last tile may be partial: at most one a non-empty expert
    L.tiles[h] = at;
    L.tile_cap[h] = L.rows / (h == 0 ? 128 : 256) + used;
    at += 4 * L.tile_cap[h];
  }
  L.pos = at;
  L.src = L.pos + r4(L.n);
  L.ints = L.src + r4(L.rows);
  L.fine_flag = L.fine = -1;
  if (H > 0 && L.n <= MOE_FINE_SLOTS) {
    L.fine_flag = L.ints;
    L.fine = L.ints + 4;
    L.ints = L.fine + L.rows * H;  // (rows are a multiple of 16)
  }
  return L;
}

cudaError_t launch_moe_sort(const int* ids, int* plan, const MoePlan& L, int E, cudaStream_t stream,
                            bool pdl);
cudaError_t launch_moe_dispatch(const void* x, const int* plan, const MoePlan& L, int T, int top_k,
                                int H, void* xs, cudaStream_t stream, bool pdl);
// w_bf16: the routing weights are bf16, else fp32; weights == nullptr: ones (the gradient of the dispatch); y32: y is fp32, with weights
cudaError_t launch_moe_combine(const void* y, bool y32, const int* plan, const MoePlan& L, int T,
                               int top_k, int H, const void* weights, bool w_bf16,
                               const void* residual, void* out, cudaStream_t stream, bool pdl);
cudaError_t launch_moe_combine_bwd(const void* dout, const void* y, const int* plan,
                                   const MoePlan& L, int T, int top_k, int H, const void* weights,
                                   bool w_bf16, void* dy, void* dweights, cudaStream_t stream,
                                   bool pdl);

// y[r] = bf16(fp32 row r of the plan) for the rows in use, and the plan's flag.
cudaError_t launch_moe_fine_rows(int* plan, const MoePlan& L, int E, int H, void* y,
                                 cudaStream_t stream, bool pdl);

// Up to eight tokens (and 128 slots): the touched experts' weights streamed,
// straight from the tokens and ids: h[slot] bf16 [n, I] (the slots that use an
// expert first for their token), then out[t] = residual[t] + sum of weighted
// down projections.  Clears *status.
constexpr int MOE_DECODE_MAX_T = 8;
constexpr int MOE_DECODE_MAX_SLOTS = 128;
cudaError_t launch_moe_decode_act(const void* x, const int* ids, const void* Wg, const void* Wu,
                                  const void* Wd, void* h, int T, int top_k, int E, int H, int I,
                                  int act, bool gated, float s, cudaStream_t stream, bool pdl,
                                  int* status);
cudaError_t launch_moe_decode_down(const void* h, const int* ids, const void* weights, bool w_bf16,
                                   const void* Wd, const void* residual, void* out, int T,
                                   int top_k, int E, int H, int I, cudaStream_t stream, bool pdl);

}  // namespace mlpk
