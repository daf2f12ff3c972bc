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

  // One entry.
  __device__ __forceinline__ void one(int64_t i, int64_t j, float c) const {
    if (i >= rows || j >= cols) return;
    if (e.bias) c += to_f32(static_cast<const T*>(e.bias)[j]);
    if (e.Z) static_cast<T*>(e.Z)[i * e.ldz + j] = from_f32<T>(c);
    with_act(e.act, [&](auto act) { c = act_of<decltype(act)::value, T>(c); });
    if (e.R) c += to_f32(static_cast<const T*>(e.R)[i * e.ldr + j]);
    static_cast<T*>(e.out)[i * e.ldo + j] = from_f32<T>(c);
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
      for (int q = 0; q < NV; ++q) c[q] = act_of<decltype(act)::value, T>(c[q]);
    });
    if (e.R) {
      load<NV>(static_cast<const T*>(e.R) + i * e.ldr + j, n, wide_r, x);
#pragma unroll
      for (int q = 0; q < NV; ++q) c[q] += x[q];
    }
    store<NV>(static_cast<T*>(e.out) + i * e.ldo + j, n, wide_out, c);
  }
};

// A warp's 32 rows x 64 bytes (2 KB) on their way between the lanes, a row each, and memory, where
// 16-byte accesses of neighbouring lanes cover neighbouring bytes: row r's 16-byte chunk c lies at chunk
// c ^ (r / 2 % 4) of its 64 bytes, so that both sides' accesses fall into distinct banks.
template <typename T>
struct Tile32 {
  static constexpr int BYTES = 32 * 64;
  // W: entries a row, at most one a lane
  static constexpr int W = 64 / sizeof(T), EPC = 16 / sizeof(T), CH = 4, ROWS = 8;  // entries a row and a chunk, chunks a row, rows an access
  __device__ __forceinline__ static uint4* at(unsigned char* buf, int r, int c) {
    return reinterpret_cast<uint4*>(buf + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  }
  // 16 entries of the lane's own row from column x on
  __device__ __forceinline__ static void put(unsigned char* buf, int x, const float* v) {
    const int r = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < 16 / EPC; ++c) {
      uint4 w;
      T* t = reinterpret_cast<T*>(&w);
#pragma unroll
      for (int q = 0; q < EPC; ++q) t[q] = from_f32<T>(v[c * EPC + q]);
      *at(buf, r, x / EPC + c) = w;
    }
  }
  __device__ __forceinline__ static void add(unsigned char* buf, int x, float* v) {
    const int r = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < 16 / EPC; ++c) {
      const uint4 w = *at(buf, r, x / EPC + c);
      const T* t = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int q = 0; q < EPC; ++q) v[c * EPC + q] += to_f32(t[q]);
    }
  }
  // rows i0 .. i0 + 31 and columns j0 .. j0 + W - 1 of a matrix of rows x cols, held by the lanes on their way in
  __device__ __forceinline__ static void fetch(uint4 (&v)[CH], const T* p, int64_t ld, bool wide, int64_t i0, int64_t rows,
                                               int64_t j0, int64_t cols) {
    const int lane = threadIdx.x & 31;
    const int64_t j = j0 + lane % CH * EPC;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int64_t i = i0 + k * ROWS + lane / CH;
      const T* g = p + i * ld + j;
      if (i < rows && wide && j + EPC <= cols) {
        v[k] = *reinterpret_cast<const uint4*>(g);
      } else {
        T* t = reinterpret_cast<T*>(&v[k]);
#pragma unroll
        for (int q = 0; q < EPC; ++q) t[q] = i < rows && j + q < cols ? g[q] : from_f32<T>(0.f);
      }
    }
  }
  __device__ __forceinline__ static void place(unsigned char* buf, const uint4 (&v)[CH]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < CH; ++k) *at(buf, k * ROWS + lane / CH, lane % CH) = v[k];
  }
  // the tile's part of such a matrix to memory
  __device__ __forceinline__ static void drain(unsigned char* buf, T* p, int64_t ld, bool wide, int64_t i0, int64_t rows,
                                               int64_t j0, int64_t cols) {
    const int lane = threadIdx.x & 31;
    if (wide && j0 + W <= cols) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int r = k * ROWS + lane / CH, c = lane % CH;
        if (i0 + r < rows) *reinterpret_cast<uint4*>(p + (i0 + r) * ld + j0 + c * EPC) = *at(buf, r, c);
      }
    } else {
      const int n = cols - j0 < W ? (int)(cols - j0) : W, m = rows - i0 < 32 ? (int)(rows - i0) : 32;
      for (int r = 0; r < m; ++r)
        if (lane < n) p[(i0 + r) * ld + j0 + lane] = reinterpret_cast<const T*>(at(buf, r, lane / EPC))[lane % EPC];
    }
  }
};

}  // namespace fxtx
