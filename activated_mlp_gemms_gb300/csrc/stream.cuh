// stream.cuh -- the weight stream on the warp-level MMA that the few-token
// kernels share: 16- or 32-byte loads of weights and tokens that are MMA
// fragments as they come (k_decode_mma.cu explains the layout).
#pragma once
#include "ptx.cuh"

namespace mlpk {

constexpr int MD_KG = 64;    // k per load group (two k-steps of 32)

__device__ __forceinline__ uint4 ld_weights_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void ld_weights_v8(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z),
                 "=r"(b.w)
               : "l"(p));
}

__device__ __forceinline__ uint4 ld_tokens_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// d += A (16 x 16, row-major fragment a0..a3) * B (16 x 8, column-major
// fragment b0, b1), bf16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Rows of K values at p begin at multiples of 32 bytes.
__device__ __forceinline__ bool wide_rows(const void* p, int K) {
  return K % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 31u) == 0;
}

// A load group: 64 k of NMAT weight matrices (RT 16-row tiles each) and of NT
// tokens, and its MMAs.  WIDE: a lane's two k-steps are 32 contiguous bytes of a
// row, one load where rows are wide_rows, so that a warp's load takes whole 128-byte
// lines (the experts' stream of 4 tokens of 4 x 44 MB 118 -> 110 us, of one token
// 33.2 -> 32.7; the linear layer's was 20.4 without, 21.1 with).
template <int NMAT_, int NT, int RT, bool WIDE = false>
struct MdGroup {
  // k from lane to lane, and from step to step
  static constexpr int KL = WIDE ? 16 : 8, KS = WIDE ? 8 : 32;
  static constexpr int NMAT = NMAT_;
  static constexpr int NTB = NT / 8;  // 8-token blocks
  uint4 w[NMAT][RT][2][2];            // [matrix][16-row tile][row g, g + 8][k-step]
  uint4 t[NTB][2];                    // [token block][k-step]

  // the weights of the group starting at k0 (zeros past the rows or K)
  __device__ __forceinline__ void load_w(const __nv_bfloat16* const (&W)[2], int row0, int R,
                                         int K, int k0, int lane) {
    const int g = lane >> 2, q = lane & 3;
    if constexpr (WIDE) {
      if (wide_rows(W[0], K) && (NMAT == 1 || wide_rows(W[1], K))) {
        const int k = k0 + 16 * q;
#pragma unroll
        for (int a = 0; a < NMAT; ++a)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = row0 + 16 * rt + g + 8 * h;
              if (k < K && r < R)
                ld_weights_v8(W[a] + static_cast<size_t>(r) * K + k, w[a][rt][h][0],
                              w[a][rt][h][1]);
              else w[a][rt][h][0] = w[a][rt][h][1] = make_uint4(0, 0, 0, 0);
            }
        return;
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = k0 + KS * s + KL * q;
#pragma unroll
      for (int a = 0; a < NMAT; ++a)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = row0 + 16 * rt + g + 8 * h;
            w[a][rt][h][s] = (k < K && r < R)
                                 ? ld_weights_v4(W[a] + static_cast<size_t>(r) * K + k)
                                 : make_uint4(0, 0, 0, 0);
          }
    }
  }

  // the token chunks of the group (zeros past the M tokens or K)
  __device__ __forceinline__ void load_t(const __nv_bfloat16* T, int M, int K, int k0, int lane) {
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = k0 + KS * s + KL * q;
#pragma unroll
      for (int b = 0; b < NTB; ++b) {
        const int m = 8 * b + g;
        t[b][s] = (k < K && m < M) ? ld_tokens_v4(T + static_cast<size_t>(m) * K + k)
                                   : make_uint4(0, 0, 0, 0);
      }
    }
  }

  // the same with a row address per token block of this lane (nullptr: zeros)
  __device__ __forceinline__ void load_t_rows(const __nv_bfloat16* const (&rows)[NTB], int K,
                                              int k0, int lane) {
    const int q = lane & 3;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = k0 + KS * s + KL * q;
#pragma unroll
      for (int b = 0; b < NTB; ++b)
        t[b][s] = (k < K && rows[b] != nullptr) ? ld_tokens_v4(rows[b] + k)
                                                : make_uint4(0, 0, 0, 0);
    }
  }

  // acc[a][rt][b] += the group's part of rows (g, g + 8) of tile rt of
  // matrix a times tokens of block b
  __device__ __forceinline__ void mma(float (&acc)[NMAT][RT][NTB][4]) const {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int a = 0; a < NMAT; ++a)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int b = 0; b < NTB; ++b) {
            const uint4(&x)[2][2] = w[a][rt];
            mma_16816(acc[a][rt][b], x[0][s].x, x[1][s].x, x[0][s].y, x[1][s].y, t[b][s].x,
                      t[b][s].y);
            mma_16816(acc[a][rt][b], x[0][s].z, x[1][s].z, x[0][s].w, x[1][s].w, t[b][s].z,
                      t[b][s].w);
          }
  }
};

}  // namespace mlpk
