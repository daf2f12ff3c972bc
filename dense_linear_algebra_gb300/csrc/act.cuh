// act.cuh — the activations and their slopes, in fp32.
//
// They are evaluated for every entry of a result, in epilogues that have few warps to hide
// them: with expf, erff, tanhf and IEEE division a tall layer (1,000,000 x 32, 32 outputs, silu) spent half
// of its time here. One exponential and one rcp.approx (1 unit in the last place, subnormal
// results zero) each; the exponential is expf for float32 layers (gelu: ex2.approx of an exponent in two
// parts), and plain ex2.approx, off by about 1.2 |x| + 2 units and zero where subnormal, for results that are
// rounded to 16 bits. With v the sigmoid's argument:
//   gelu       q = erfc(|z| / sqrt(2)) as exp(-z^2 / 2) times a polynomial in t = 1 / (1 + c |z| / sqrt(2)), the form of Abramowitz
//              and Stegun 7.1.26 with the relative error made small instead of the absolute one, up to
//              |z| = 13.5 (coefficients by iterated weighted least squares; c = 0.5: 4.3e-8, c = 0.3725 and two
//              fewer of them for 16 bits: 5.7e-7): z (1 - q / 2) for z >= 0, z q / 2 below, so that the tail
//              keeps its digits; the exponential is the slope's too
//   sigmoid    s and 1 - s both from e = exp(-|v|), as 1 / (1 + e) and e / (1 + e): the slopes use both,
//              and 1 - s as a difference would leave nothing of a slope beyond v = 17
//   gelu_tanh  z sigmoid(v), v = 2 u, which is 0.5 z (1 + tanh(u)); its slope is s + z s (1 - s) v'
// The slopes of gelu, gelu_tanh and silu cross zero below z = 0, as a difference of two terms; they are accurate
// to a few units of the larger one. The rounding of v itself leaves about 3 |v| units in gelu_tanh's tail.
#pragma once

#include <type_traits>

#include "layers.h"

namespace fxtx {

constexpr float kRootHalf = 0.70710678118654752440f;   // 1 / sqrt(2)
constexpr float kRootTwoPi = 0.39894228040143267794f;  // 1 / sqrt(2 pi)
constexpr float kTanh0 = 1.59576912160573071176f;      // 2 sqrt(2 / pi)
constexpr float kTanh1 = 0.044715f;

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kHalfLog2e = -0.5f * kLog2e;  // and what a float of it leaves out
constexpr float kHalfLog2eRest = (float)(-0.5 * 1.44269504088896340736 - (double)kHalfLog2e);

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

// The exponential for layers of type T.
template <typename T>
__device__ __forceinline__ float exp_of(float x) {
  if constexpr (sizeof(T) == 4) return expf(x);
  return ex2(kLog2e * x);
}

template <typename T>
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + exp_of<T>(-v)); }

// sigmoid(v), with 1 - sigmoid(v) beside it.
template <typename T>
__device__ __forceinline__ float sigmoid(float v, float& rest) {
  const float e = exp_of<T>(-fabsf(v)), r = rcp(1.f + e), x = e * r;
  rest = v < 0.f ? r : x;
  return v < 0.f ? x : r;
}

// A polynomial in t, its highest coefficient first.
__device__ __forceinline__ float horner(float, float p) { return p; }
template <typename... C>
__device__ __forceinline__ float horner(float t, float p, float c, C... rest) {
  return horner(t, fmaf(p, t, c), rest...);
}

// erfc(|z| / sqrt(2)) and exp(-z^2 / 2).
template <typename T>
__device__ __forceinline__ float erfc_half(float z, float& gauss) {
  if constexpr (sizeof(T) == 4) {
    // the exponent -z^2 log2(e) / 2 with what its roundings leave out (beyond 16 the exponential is zero)
    const float a = fminf(fabsf(z), 16.f), h = a * a, x = kHalfLog2e * h;
    float rest = fmaf(kHalfLog2e, h, -x);
    rest = fmaf(kHalfLog2eRest, h, rest);
    rest = fmaf(kHalfLog2e, fmaf(a, a, -h), rest);
    gauss = ex2(x);
    gauss = fmaf(gauss, kLn2 * rest, gauss);
    const float t = rcp(fmaf(0.5f * kRootHalf, fabsf(z), 1.f));
    return t * gauss *
           horner(t, -0.05890960971f, 0.2837944093f, -0.4855764104f, 0.2762003024f, -0.0253320584f, 0.2021358148f,
                  0.2432441336f, 0.282355836f, 0.2820875401f);
  } else {
    gauss = ex2(kHalfLog2e * z * z);
    const float t = rcp(fmaf(0.3725f * kRootHalf, fabsf(z), 1.f));
    return t * gauss *
           horner(t, -0.1396021335f, 0.4141580827f, -0.161081597f, 0.3023959233f, 0.1588338403f, 0.2154489112f,
                  0.2098469368f);
  }
}

// A NaN stays a NaN in each. T: the layer's type.
template <int ACT, typename T>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (ACT == FXTX_ACT_RELU) return z < 0.f ? 0.f : z;
  if constexpr (ACT == FXTX_ACT_GELU) {
    float gauss;
    const float q = 0.5f * erfc_half<T>(z, gauss);
    return z * (z < 0.f ? q : 1.f - q);
  }
  if constexpr (ACT == FXTX_ACT_GELU_TANH) return z * sigmoid<T>(kTanh0 * z * fmaf(kTanh1 * z, z, 1.f));
  if constexpr (ACT == FXTX_ACT_SILU) return z * sigmoid<T>(z);
  if constexpr (ACT == FXTX_ACT_SIGMOID) return sigmoid<T>(z);
  return z;
}

template <int ACT, typename T>
__device__ __forceinline__ float slope_of(float z) {
  if constexpr (ACT == FXTX_ACT_RELU) return z <= 0.f ? 0.f : 1.f;
  if constexpr (ACT == FXTX_ACT_GELU) {
    float gauss;
    const float q = 0.5f * erfc_half<T>(z, gauss);
    return fmaf(z * kRootTwoPi, gauss, z < 0.f ? q : 1.f - q);
  }
  if constexpr (ACT == FXTX_ACT_GELU_TANH) {
    const float z2 = kTanh1 * z * z;
    float rest;
    const float s = sigmoid<T>(kTanh0 * z * (1.f + z2), rest);
    const float slope = fmaf(z * s * rest * kTanh0, fmaf(3.f, z2, 1.f), s);
    // s is 0 or 1 long before, and from 1e19 on z2 is an infinity
    return fabsf(z) > 16.f ? (z < 0.f ? 0.f : 1.f) : slope;
  }
  if constexpr (ACT == FXTX_ACT_SILU) {
    float rest;
    const float s = sigmoid<T>(z, rest);
    return s * fmaf(z, rest, 1.f);
  }
  if constexpr (ACT == FXTX_ACT_SIGMOID) {
    float rest;
    const float s = sigmoid<T>(z, rest);
    return s * rest;
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
