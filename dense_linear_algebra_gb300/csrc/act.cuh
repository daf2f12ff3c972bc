// act.cuh — the activations and their slopes, in fp32.
#pragma once

#include <type_traits>

#include "layers.h"

namespace fxtx {

constexpr float kRootHalf = 0.70710678118654752440f;   // 1 / sqrt(2)
constexpr float kRootTwoPi = 0.39894228040143267794f;  // 1 / sqrt(2 pi)
constexpr float kTanh0 = 0.79788456080286535588f;      // sqrt(2 / pi)
constexpr float kTanh1 = 0.044715f;

// A NaN stays a NaN in each.
template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (ACT == FXTX_ACT_RELU) return z < 0.f ? 0.f : z;
  if constexpr (ACT == FXTX_ACT_GELU) return 0.5f * z * (1.f + erff(z * kRootHalf));
  if constexpr (ACT == FXTX_ACT_GELU_TANH) return 0.5f * z * (1.f + tanhf(kTanh0 * (z + kTanh1 * z * z * z)));
  if constexpr (ACT == FXTX_ACT_SILU) return z / (1.f + expf(-z));
  if constexpr (ACT == FXTX_ACT_SIGMOID) return 1.f / (1.f + expf(-z));
  return z;
}

template <int ACT>
__device__ __forceinline__ float slope_of(float z) {
  if constexpr (ACT == FXTX_ACT_RELU) return z <= 0.f ? 0.f : 1.f;
  if constexpr (ACT == FXTX_ACT_GELU)
    return 0.5f * (1.f + erff(z * kRootHalf)) + z * expf(-0.5f * z * z) * kRootTwoPi;
  if constexpr (ACT == FXTX_ACT_GELU_TANH) {
    const float t = tanhf(kTanh0 * (z + kTanh1 * z * z * z));
    return 0.5f * (1.f + t) + 0.5f * z * (1.f - t * t) * kTanh0 * (1.f + 3.f * kTanh1 * z * z);
  }
  if constexpr (ACT == FXTX_ACT_SILU) {
    const float s = 1.f / (1.f + expf(-z));
    return s * (1.f + z * (1.f - s));
  }
  if constexpr (ACT == FXTX_ACT_SIGMOID) {
    const float s = 1.f / (1.f + expf(-z));
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
