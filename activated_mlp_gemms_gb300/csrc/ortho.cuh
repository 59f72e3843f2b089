// ortho.cuh -- what the orthogonalised update's kernels share on the device.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace mlpk {

namespace {

constexpr int O_TIMEOUT = -6;  // MLP_ERR_TIMEOUT

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// Part j (16 bytes) of row r of the 128 x 128 fp32 sums: the parts of a row swapped by the row,
// so that a row a thread and a row a warp both pass without bank conflicts.
__device__ __forceinline__ uint32_t sum_part(uint32_t at, int r, int j) {
  return at + static_cast<uint32_t>(r * 512 + ((j ^ (r & 31)) << 4));
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));  // (no clobber: all of a row's are on their way together)
  return v;
}
// The sum of eight columns of a row over the shared memories of the first N CTAs of the cluster,
// in their order; x, y: the parts' addresses in each.
template <int N>
__device__ __forceinline__ void cluster_sums(uint32_t x, uint32_t y, float (&f)[8]) {
  float4 u[N], v[N];
#pragma unroll
  for (int s = 0; s < N; ++s) {
    u[s] = ld_cluster_f4(mapa_shared(x, s));
    v[s] = ld_cluster_f4(mapa_shared(y, s));
  }
#pragma unroll
  for (int s = 0; s < N; ++s) {
    f[0] += u[s].x, f[1] += u[s].y, f[2] += u[s].z, f[3] += u[s].w;
    f[4] += v[s].x, f[5] += v[s].y, f[6] += v[s].z, f[7] += v[s].w;
  }
}

// Eight values of G.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 v = ld_global_v4(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack_bf16x2(w[i]);
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  } else {
    const uint4 a = ld_global_v4(p), b = ld_global_v4(p + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  }
}

}  // namespace

}  // namespace mlpk
