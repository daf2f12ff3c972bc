// act.cuh — the activations and their slopes, in fp32.
//
// They are evaluated for every entry of a result, in epilogues that have few warps to hide
// them, so the forms are the cheapest that keep fp32 accuracy: one ex2.approx (the exponential is
// then off by about 1.2 |x| + 2 units in its last place), one rcp.approx (1 unit), both with
// subnormal numbers taken as zero, and no difference of nearly equal terms. With expf, erff, tanhf
// and IEEE division a tall layer (1,000,000 x 32, 32 outputs, silu) spent half of its time here.
//   gelu       the complementary error function q of |z| / sqrt(2) by Abramowitz and Stegun 7.1.26
//              (absolute error 1.5e-7): z (1 - q / 2) for z >= 0, z q / 2 below; its
//              exponential exp(-z^2 / 2) is the slope's too
//   gelu_tanh  z sigmoid(2 u), which is 0.5 z (1 + tanh(u)); with s = sigmoid(2 u) its slope is
//              s + z s (1 - s) 2 u'
#pragma once

#include <type_traits>

#include "layers.h"

namespace fxtx {

constexpr float kRootHalf = 0.70710678118654752440f;   // 1 / sqrt(2)
constexpr float kRootTwoPi = 0.39894228040143267794f;  // 1 / sqrt(2 pi)
constexpr float kTanh0 = 1.59576912160573071176f;      // 2 sqrt(2 / pi)
constexpr float kTanh1 = 0.044715f;

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sigmoid(float z) { return rcp(1.f + ex2(-kLog2e * z)); }

// erfc(|z| / sqrt(2)) and exp(-z^2 / 2).
__device__ __forceinline__ float erfc_half(float z, float& gauss) {
  const float t = rcp(fmaf(0.3275911f * kRootHalf, fabsf(z), 1.f));
  gauss = ex2(-0.5f * kLog2e * z * z);
  float p = fmaf(1.061405429f, t, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  return p * t * gauss;
}

// A NaN stays a NaN in each.
template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (ACT == FXTX_ACT_RELU) return z < 0.f ? 0.f : z;
  if constexpr (ACT == FXTX_ACT_GELU) {
    float gauss;
    const float q = 0.5f * erfc_half(z, gauss);
    return z * (z < 0.f ? q : 1.f - q);
  }
  if constexpr (ACT == FXTX_ACT_GELU_TANH) return z * sigmoid(kTanh0 * z * fmaf(kTanh1 * z, z, 1.f));
  if constexpr (ACT == FXTX_ACT_SILU) return z * sigmoid(z);
  if constexpr (ACT == FXTX_ACT_SIGMOID) return sigmoid(z);
  return z;
}

template <int ACT>
__device__ __forceinline__ float slope_of(float z) {
  if constexpr (ACT == FXTX_ACT_RELU) return z <= 0.f ? 0.f : 1.f;
  if constexpr (ACT == FXTX_ACT_GELU) {
    float gauss;
    const float q = 0.5f * erfc_half(z, gauss);
    return fmaf(z * kRootTwoPi, gauss, z < 0.f ? q : 1.f - q);
  }
  if constexpr (ACT == FXTX_ACT_GELU_TANH) {
    const float z2 = kTanh1 * z * z, s = sigmoid(kTanh0 * z * (1.f + z2));
    return fmaf(z * s * (1.f - s) * kTanh0, fmaf(3.f, z2, 1.f), s);
  }
  if constexpr (ACT == FXTX_ACT_SILU) {
    const float s = sigmoid(z);
    return s * fmaf(z, 1.f - s, 1.f);
  }
  if constexpr (ACT == FXTX_ACT_SIGMOID) {
    const float s = sigmoid(z);
    return s * (1.f - s);
  }
  return 1.f;
}

// f(std::integral_constant<int, ACT>) for the activation chosen at run time.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case FXTX_ACT_RELU: f(std::integral_constant<int, FXTX_ACT_RELU>{}); break;
    case FXTX_ACT_GELU: f(std::integral_constant<int, FXTX_ACT_GELU>{}); break;
    case FXTX_ACT_GELU_TANH: f(std::integral_constant<int, FXTX_ACT_GELU_TANH>{}); break;
    case FXTX_ACT_SILU: f(std::integral_constant<int, FXTX_ACT_SILU>{}); break;
    case FXTX_ACT_SIGMOID: f(std::integral_constant<int, FXTX_ACT_SIGMOID>{}); break;
    default: f(std::integral_constant<int, FXTX_ACT_NONE>{}); break;
  }
}

}  // namespace fxtx
