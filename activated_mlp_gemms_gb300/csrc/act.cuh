// act.cuh -- the MLP activations and their derivatives in fp32, as used by
// the fused epilogues.
//   silu(z)  = z * sigmoid(z)            silu'(z)  = s (1 + z (1 - s)),  s = sigmoid(z)
//   relu2(z) = max(z,0)^2                relu2'(z) = 2 max(z,0)
//   gelu_tanh(z) = 0.5 z (1 + t),  t = tanh(c (z + 0.044715 z^3)),  c = sqrt(2/pi)
//   gelu_tanh'(z) = 0.5 (1 + t) + 0.5 z (1 - t^2) c (1 + 3*0.044715 z^2)
//   relu(z)  = max(z,0)                  relu'(z)  = 1 for z > 0, else 0
//   sigmoid(z) = 1 / (1 + e^-z)          sigmoid'(z) = s (1 - s)
// (tanh approximation of GELU: Hendrycks & Gimpel, 2016).  The sigmoid is
// taken from the hardware tanh, sigmoid(z) = (1 + tanh(z/2)) / 2, one
// tanh.approx.f32 instead of an exponential and a reciprocal (measured on a
// GB300 over z in [-20, 20]: at most 4e-6 from the fp64 sigmoid, 1e-5 for
// silu and silu'; the epilogues' arithmetic is bound by instruction issue,
// and this takes SwiGLU's fused epilogues from two special-function
// instructions per element to one).  The GELU's tanh is CUDA's tanhf, in the
// dense MLP.
// The _EXP forms keep the relative error small where the result is (for z below
// -3 an absolute error of 4e-6 in the sigmoid is percents of it, and 1 + tanh
// cancels): sigmoid(z) = 1 / (1 + e^-z) with the hardware's exponential and
// reciprocal, and gelu_tanh(z) = z sigmoid(2u), u = c (z + 0.044715 z^3), since
// (1 + tanh(u)) / 2 = sigmoid(2u).  The linear layer, whose result the activation
// is, takes all three; the experts take the GELU's.
#pragma once
#include "gemm_params.h"

namespace mlpk {

__device__ __forceinline__ float tanh_hw(float x) {
  float y;
  asm("tanh.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float sigmoid_f(float z) {
  return fmaf(0.5f, tanh_hw(0.5f * z), 0.5f);
}

// sigmoid(x) = 1 / (1 + 2^-t), t = x log2(e)
__device__ __forceinline__ float sigmoid_exp2(float t) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-t));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}
constexpr float LOG2_E = 1.4426950408889634f;

// max(z, 0), NaN where z is
__device__ __forceinline__ float relu_f(float z) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(z));
  return r;
}

template <int ACT>
__device__ __forceinline__ float act_f(float z) {
  if constexpr (ACT == ACT_NONE) {
    return z;
  } else if constexpr (ACT == ACT_SILU) {
    return z * sigmoid_f(z);
  } else if constexpr (ACT == ACT_RELU_SQ) {
    float r = relu_f(z);
    return r * r;
  } else if constexpr (ACT == ACT_RELU) {
    return relu_f(z);
  } else if constexpr (ACT == ACT_SIGMOID) {
    return sigmoid_f(z);
  } else if constexpr (ACT == ACT_SILU_EXP) {
    return z * sigmoid_exp2(LOG2_E * z);
  } else if constexpr (ACT == ACT_SIGMOID_EXP) {
    return sigmoid_exp2(LOG2_E * z);
  } else if constexpr (ACT == ACT_GELU_EXP) {
    const float c2 = 2.0f * 0.7978845608028654f;  // 2 sqrt(2/pi)
    return z * sigmoid_exp2(LOG2_E * c2 * fmaf(0.044715f * z, z * z, z));
  } else {
    const float c = 0.7978845608028654f;  // sqrt(2/pi)
    float t = tanhf(c * fmaf(0.044715f * z, z * z, z));
    return 0.5f * z * (1.0f + t);
  }
}

// act(z) and act'(z) together.
template <int ACT>
__device__ __forceinline__ void act_and_grad(float z, float& a, float& da) {
  if constexpr (ACT == ACT_NONE) {
    a = z;
    da = 1.0f;
  } else if constexpr (ACT == ACT_SILU) {
    float s = sigmoid_f(z);
    a = z * s;
    da = s * fmaf(z, 1.0f - s, 1.0f);
  } else if constexpr (ACT == ACT_RELU_SQ) {
    float r = relu_f(z);
    a = r * r;
    da = 2.0f * r;
  } else if constexpr (ACT == ACT_RELU) {
    a = relu_f(z);
    da = z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == ACT_SIGMOID) {
    const float s = sigmoid_f(z);
    a = s;
    da = s * (1.0f - s);
  } else if constexpr (ACT == ACT_SILU_EXP) {
    const float s = sigmoid_exp2(LOG2_E * z);
    a = z * s;
    da = s * fmaf(z, 1.0f - s, 1.0f);
  } else if constexpr (ACT == ACT_SIGMOID_EXP) {
    const float s = sigmoid_exp2(LOG2_E * z);
    a = s;
    da = s * (1.0f - s);
  } else if constexpr (ACT == ACT_GELU_EXP) {
    // with s = sigmoid(2u): s + z s (1 - s) 2u',  u' = c (1 + 3 * 0.044715 z^2)
    const float c2 = 2.0f * 0.7978845608028654f;
    const float k = 0.044715f;
    const float z2 = z * z;
    const float s = sigmoid_exp2(LOG2_E * c2 * fmaf(k * z, z2, z));
    a = z * s;
    da = fmaf(a * (1.0f - s), fmaf(3.0f * k * c2, z2, c2), s);
  } else {
    const float c = 0.7978845608028654f;
    const float k = 0.044715f;
    float z2 = z * z;
    float t = tanhf(c * fmaf(k * z, z2, z));
    a = 0.5f * z * (1.0f + t);
    da = 0.5f * (1.0f + t) + 0.5f * z * (1.0f - t * t) * c * fmaf(3.0f * k, z2, 1.0f);
  }
}

}  // namespace mlpk
