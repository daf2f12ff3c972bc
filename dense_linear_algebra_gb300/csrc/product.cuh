// product.cuh — the epilogue of a product's entries: out = act(c + bias_j) + R_ij, c + bias_j to Z.
#pragma once

#include <type_traits>

#include "act.cuh"
#include "common.cuh"
#include "linear.h"

namespace fxtx {

template <typename T>
struct Finish {
  const Epilogue e;
  const int64_t rows, cols;
  bool wide_out, wide_z, wide_r, wide_b;

  __device__ static bool wide(const void* p, int64_t ld) {
    return p != nullptr && ((uintptr_t)p & 15u) == 0 && (ld * (int64_t)sizeof(T)) % 16 == 0;
  }
  __device__ Finish(const Epilogue& ep, int64_t m, int64_t n) : e(ep), rows(m), cols(n) {
    wide_out = wide(e.out, e.ldo);
    wide_z = wide(e.Z, e.ldz);
    wide_r = wide(e.R, e.ldr);
    wide_b = wide(e.bias, 0);
  }

  // NV entries in accesses of 16 bytes, or of 8 (NV = 4 of a 16-bit type).
  template <int NV>
  using Word = typename std::conditional<NV * sizeof(T) % 16 == 0, uint4, uint2>::type;
  template <int NV>
  __device__ __forceinline__ static void load(const T* p, int n, bool w, float* x) {
    if (w && n == NV) {
      constexpr int V = NV * sizeof(T) / sizeof(Word<NV>);
      Word<NV> v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = reinterpret_cast<const Word<NV>*>(p)[i];
      const T* t = reinterpret_cast<const T*>(v);
#pragma unroll
      for (int i = 0; i < NV; ++i) x[i] = to_f32(t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) x[i] = i < n ? to_f32(p[i]) : 0.f;
    }
  }
  template <int NV>
  __device__ __forceinline__ static void store(T* p, int n, bool w, const float* x) {
    if (w && n == NV) {
      constexpr int V = NV * sizeof(T) / sizeof(Word<NV>);
      Word<NV> v[V];
      T* t = reinterpret_cast<T*>(v);
#pragma unroll
      for (int i = 0; i < NV; ++i) t[i] = from_f32<T>(x[i]);
#pragma unroll
      for (int i = 0; i < V; ++i) reinterpret_cast<Word<NV>*>(p)[i] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i < n) p[i] = from_f32<T>(x[i]);
    }
  }

  // NV (4, 8 or 16) entries of row i from column j on, j a multiple of NV.
  template <int NV>
  __device__ __forceinline__ void row(int64_t i, int64_t j, const float* acc) const {
    if (i >= rows || j >= cols) return;
    const int n = cols - j >= NV ? NV : (int)(cols - j);
    float c[NV], x[NV];
#pragma unroll
    for (int q = 0; q < NV; ++q) c[q] = acc[q];
    if (e.bias) {
      load<NV>(static_cast<const T*>(e.bias) + j, n, wide_b, x);
#pragma unroll
      for (int q = 0; q < NV; ++q) c[q] += x[q];
    }
    if (e.Z) store<NV>(static_cast<T*>(e.Z) + i * e.ldz + j, n, wide_z, c);
    with_act(e.act, [&](auto act) {
#pragma unroll
      for (int q = 0; q < NV; ++q) c[q] = act_of<decltype(act)::value>(c[q]);
    });
    if (e.R) {
      load<NV>(static_cast<const T*>(e.R) + i * e.ldr + j, n, wide_r, x);
#pragma unroll
      for (int q = 0; q < NV; ++q) c[q] += x[q];
    }
    store<NV>(static_cast<T*>(e.out) + i * e.ldo + j, n, wide_out, c);
  }
};

// The same entries as partial sums.
__device__ __forceinline__ void part_row(float* part, int64_t rows, int64_t cols, int64_t i, int64_t j, const float* c) {
  if (i >= rows) return;
  float* p = part + i * cols + j;
  if (cols % 4 == 0 && j + 16 <= cols) {
#pragma unroll
    for (int q = 0; q < 16; q += 4) *reinterpret_cast<float4*>(p + q) = make_float4(c[q], c[q + 1], c[q + 2], c[q + 3]);
  } else {
#pragma unroll
    for (int q = 0; q < 16; ++q)
      if (j + q < cols) p[q] = c[q];
  }
}

}  // namespace fxtx
