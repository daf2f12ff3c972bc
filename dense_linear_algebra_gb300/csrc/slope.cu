// slope.cu — D = G * act'(Z), the gradient at a linear layer's pre-activations, and db, its
// column sums, in one pass over G and Z.
//
// Bound: HBM (G and Z read once, D written once). A thread takes 8 neighbouring columns, a
// CTA 256 / CX rows at a time of CX such column groups; each CTA's column sums go to a
// workspace and a second kernel adds them in order, so db is the same on every call. D is
// rounded to the layer's type (the products that follow take it as an operand); db is summed
// from the unrounded values. Of float32, D is written as the three bfloat16 planes that the
// products take. The same stores serve a plain copy into an aligned pitch (launch_pack).
#include <algorithm>
#include <type_traits>

#include "act.cuh"
#include "common.cuh"
#include "kernels.h"
#include "linear.h"

namespace fxtx {
namespace {

template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, bool wide, float* x) {
  if (wide) {
    if constexpr (sizeof(T) == 4) {
      const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      const T* e = reinterpret_cast<const T*>(&a);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = to_f32(e[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}

// 8 values as T, or of float32 as their three bfloat16 planes.
template <typename T>
__device__ __forceinline__ void store8(void* dst, int64_t at, int64_t plane_stride, int n, bool wide, const float* x) {
  using S = typename std::conditional<sizeof(T) == 4, __nv_bfloat16, T>::type;
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int plane = 0; plane < (sizeof(T) == 4 ? 3 : 1); ++plane) {
    S* p = static_cast<S*>(dst) + plane * plane_stride + at;
    uint4 a;
    S* e = reinterpret_cast<S*>(&a);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e[i] = from_f32<S>(r[i]);
      if constexpr (sizeof(T) == 4) r[i] -= to_f32(e[i]);  // exact
    }
    if (wide) {
      *reinterpret_cast<uint4*>(p) = a;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = e[i];
    }
  }
}

__host__ __device__ inline bool rows_aligned(const void* p, int64_t ld, int size) {
  return ((uintptr_t)p & 15u) == 0 && (ld * size) % 16 == 0;
}

// cx: column groups of 8 a CTA takes, a power of two up to 32
template <typename T>
__global__ void __launch_bounds__(256) slope_kernel(const SlopeArgs a, const int cx, const int64_t rows_per_cta) {
  after_previous();
  const int gx = threadIdx.x & (cx - 1), gy = threadIdx.x / cx, step = 256 / cx;
  const int64_t col = ((int64_t)blockIdx.x * cx + gx) * 8;
  const int64_t r1 = min(a.m, (int64_t)(blockIdx.y + 1) * rows_per_cta);
  const int n = a.k - col >= 8 ? 8 : (a.k > col ? (int)(a.k - col) : 0);
  const bool wg = n == 8 && rows_aligned(a.G, a.ldg, sizeof(T));
  const bool wz = n == 8 && rows_aligned(a.Z, a.ldz, sizeof(T));
  const bool wd = n == 8 && rows_aligned(a.D, a.ldd, 2) && a.d_planes % 8 == 0;
  const T *G = static_cast<const T*>(a.G) + col, *Z = static_cast<const T*>(a.Z) + col;
  float sum[8] = {};
  if (n > 0)
    with_act(a.act, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      for (int64_t r = (int64_t)blockIdx.y * rows_per_cta + gy; r < r1; r += step) {
        float g[8];
        load8(G + r * a.ldg, n, wg, g);
        if constexpr (ACT != FXTX_ACT_NONE) {
          float z[8];
          load8(Z + r * a.ldz, n, wz, z);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] *= slope_of<ACT>(z[i]);
        }
        if (a.D != nullptr) store8<T>(a.D, r * a.ldd + col, a.d_planes, n, wd, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += g[i];
      }
    });
  if (a.db == nullptr) return;
  __shared__ float part[256 * 8];
#pragma unroll
  for (int i = 0; i < 8; ++i) part[(gy * cx + gx) * 8 + i] = sum[i];
  __syncthreads();
  for (int c = threadIdx.x; c < cx * 8; c += 256) {
    const int64_t j = (int64_t)blockIdx.x * cx * 8 + c;
    if (j >= a.k) continue;
    float s = 0.f;
    for (int y = 0; y < step; ++y) s += part[y * cx * 8 + c];
    a.ws[(int64_t)blockIdx.y * a.k + j] = s;
  }
}

// db_j = the sum of `parts` rows of ws: 32 columns a CTA, 8 threads a column.
template <typename T>
__global__ void __launch_bounds__(256) sums_kernel(const float* ws, int64_t parts, int64_t k, T* db) {
  __shared__ float part[8][32];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t j = (int64_t)blockIdx.x * 32 + x;
  float s = 0.f;
  after_previous();
  if (j < k)
    for (int64_t r = y; r < parts; r += 8) s += ws[r * k + j];
  part[y][x] = s;
  __syncthreads();
  if (y == 0 && j < k) {
    for (int i = 1; i < 8; ++i) s += part[i][x];
    db[j] = from_f32<T>(s);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) pack_kernel(const PackArgs a) {
  const int64_t groups = (a.cols + 7) / 8, stride = (int64_t)gridDim.x * 256;
  after_previous();
  const bool aligned = rows_aligned(a.src, a.ld, sizeof(T));
  for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < a.rows * groups; x += stride) {
    const int64_t i = x / groups, j = x % groups * 8;
    const int n = a.cols - j >= 8 ? 8 : (int)(a.cols - j);
    float v[8];
    load8(static_cast<const T*>(a.src) + i * a.ld + j, n, aligned && n == 8, v);
    store8<T>(a.dst, i * a.pitch + j, a.plane_stride, n, n == 8, v);
  }
}

struct SlopeGrid {
  int cx;
  int64_t gx, gy, rows;
};
SlopeGrid slope_grid(int64_t m, int64_t k, int sm_count) {
  SlopeGrid g;
  const int64_t groups = (k + 7) / 8;
  g.cx = 1;
  while (g.cx < 32 && g.cx < groups) g.cx *= 2;
  g.gx = (groups + g.cx - 1) / g.cx;
  // about 6 CTAs a SM, each of at least one step of rows
  const int64_t step = 256 / g.cx, want = std::max<int64_t>(1, (int64_t)sm_count * 6 / g.gx);
  const int64_t steps = (m + step - 1) / step, per = std::max<int64_t>(1, (steps + want - 1) / want);
  g.rows = per * step;
  g.gy = std::max<int64_t>(1, (m + g.rows - 1) / g.rows);
  // the grid's second dimension ends at 65,535
  while (g.gy > 65535) {
    g.rows *= 2;
    g.gy = (m + g.rows - 1) / g.rows;
  }
  return g;
}

template <typename T>
cudaError_t launch_t(const SlopeArgs& a, int sm_count, cudaStream_t st) {
  const SlopeGrid g = slope_grid(a.m, a.k, sm_count);
  const cudaError_t e = launch_kernel(slope_kernel<T>, dim3((unsigned)g.gx, (unsigned)g.gy), 256, 0, st, a, g.cx, g.rows);
  if (e != cudaSuccess || a.db == nullptr) return e;
  return launch_kernel(sums_kernel<T>, dim3((unsigned)((a.k + 31) / 32)), 256, 0, st, a.ws, g.gy, a.k, static_cast<T*>(a.db));
}

}  // namespace

cudaError_t launch_pack(const PackArgs& a, int sm_count, cudaStream_t st) {
  const int64_t blocks = std::min<int64_t>((a.rows * ((a.cols + 7) / 8) + 255) / 256, (int64_t)sm_count * 16);
  if (blocks == 0) return cudaSuccess;
  switch (a.type) {
    case FXTX_F32: return launch_kernel(pack_kernel<float>, dim3((unsigned)blocks), 256, 0, st, a);
    case FXTX_BF16: return launch_kernel(pack_kernel<__nv_bfloat16>, dim3((unsigned)blocks), 256, 0, st, a);
    default: return launch_kernel(pack_kernel<__half>, dim3((unsigned)blocks), 256, 0, st, a);
  }
}

size_t slope_ws_bytes(int64_t m, int64_t k, int sm_count) {
  return (size_t)slope_grid(m, k, sm_count).gy * (size_t)k * 4;
}

cudaError_t launch_slope(const SlopeArgs& a, int sm_count, cudaStream_t st) {
  switch (a.type) {
    case FXTX_F32: return launch_t<float>(a, sm_count, st);
    case FXTX_BF16: return launch_t<__nv_bfloat16>(a, sm_count, st);
    default: return launch_t<__half>(a, sm_count, st);
  }
}

}  // namespace fxtx
