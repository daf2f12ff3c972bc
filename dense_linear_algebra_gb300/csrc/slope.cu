// slope.cu — D = G * act'(Z), the gradient at a linear layer's pre-activations, and db, its
// column sums, in one pass over G and Z.
//
// Bound: HBM (G and Z read once, D written once). A thread takes 8 neighbouring columns, a
// CTA 256 / CX rows at a time of CX such column groups; each CTA's column sums go to a
// workspace and a second kernel adds them in order, so db is the same on every call (few rows:
// a CTA takes all of them and writes db itself). D is
// rounded to the layer's type (the products that follow take it as an operand); db is summed
// from the unrounded values. Of float32, D is written as the three bfloat16 planes that the
// products take. The same stores copy a matrix into an aligned pitch, or split it into planes; a
// gradient's slope and copies are one launch. 8192 x 16384 bfloat16 with gelu: 153 us, 5.3 TB/s.
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

struct SlopeGrid {
  int cx;           // column groups of 8 a CTA takes, a power of two up to 32
  int64_t gx, gy;   // CTAs over the columns and over the rows
  int64_t rows;     // rows a CTA takes
};

template <typename T>
__device__ __forceinline__ void slope(const SlopeArgs& a, const SlopeGrid& grid, int64_t bx, int64_t by) {
  const int cx = grid.cx, gx = threadIdx.x & (cx - 1), gy = threadIdx.x / cx, step = 256 / cx;
  const int64_t col = (bx * cx + gx) * 8;
  const int64_t r1 = min(a.m, (by + 1) * grid.rows);
  const int n = a.k - col >= 8 ? 8 : (a.k > col ? (int)(a.k - col) : 0);
  const bool wg = n == 8 && rows_aligned(a.G, a.ldg, sizeof(T));
  const bool wz = n == 8 && rows_aligned(a.Z, a.ldz, sizeof(T));
  const bool wd = n == 8 && rows_aligned(a.D, a.ldd, 2) && a.d_planes % 8 == 0;
  const T *G = static_cast<const T*>(a.G) + col, *Z = static_cast<const T*>(a.Z) + col;
  float sum[8] = {};
  if (n > 0)
    with_act(a.act, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      for (int64_t r = by * grid.rows + gy; r < r1; r += step) {
        float g[8];
        load8(G + r * a.ldg, n, wg, g);
        if constexpr (ACT != FXTX_ACT_NONE) {
          float z[8];
          load8(Z + r * a.ldz, n, wz, z);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] *= slope_of<ACT, T>(z[i]);
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
    const int64_t j = bx * cx * 8 + c;
    if (j >= a.k) continue;
    float s = 0.f;
    for (int y = 0; y < step; ++y) s += part[y * cx * 8 + c];
    if (grid.gy == 1) static_cast<T*>(a.db)[j] = from_f32<T>(s);
    else a.ws[by * a.k + j] = s;
  }
}

template <typename T>
__device__ __forceinline__ void pack(const PackArgs& a, int64_t b, int64_t ctas) {
  const int64_t groups = (a.cols + 7) / 8, stride = ctas * 256;
  const bool aligned = rows_aligned(a.src, a.ld, sizeof(T));
  for (int64_t x = b * 256 + threadIdx.x; x < a.rows * groups; x += stride) {
    const int64_t i = x / groups, j = x % groups * 8;
    const int n = a.cols - j >= 8 ? 8 : (int)(a.cols - j);
    float v[8];
    load8(static_cast<const T*>(a.src) + i * a.ld + j, n, aligned && n == 8, v);
    store8<T>(a.dst, i * a.pitch + j, a.plane_stride, n, n == 8, v);
  }
}

struct PrepareArgs {
  SlopeArgs slope;
  SlopeGrid grid;
  PackArgs pack[2];
  int64_t ctas[3];  // the slope's, and each copy's
};

template <typename T>
__global__ void __launch_bounds__(256) prepare_kernel(const __grid_constant__ PrepareArgs a) {
  after_previous();
  int64_t b = blockIdx.x;
  if (b < a.ctas[0]) {
    slope<T>(a.slope, a.grid, b % a.grid.gx, b / a.grid.gx);
  } else if ((b -= a.ctas[0]) < a.ctas[1]) {
    pack<T>(a.pack[0], b, a.ctas[1]);
  } else {
    pack<T>(a.pack[1], b - a.ctas[1], a.ctas[2]);
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

SlopeGrid slope_grid(int64_t m, int64_t k, int sm_count) {
  SlopeGrid g;
  const int64_t groups = (k + 7) / 8;
  g.cx = 1;
  if (m <= 2048) {  // a CTA takes all rows, of as many columns as leave no SM without work
    while (g.cx < 32 && g.cx < groups && (groups + 2 * g.cx - 1) / (2 * g.cx) >= sm_count) g.cx *= 2;
    if (g.cx < 2 && groups > 1) g.cx = 2;  // whole 32-byte sectors
    g.gx = (groups + g.cx - 1) / g.cx;
    g.gy = 1;
    g.rows = m;
    return g;
  }
  while (g.cx < 32 && g.cx < groups) g.cx *= 2;
  g.gx = (groups + g.cx - 1) / g.cx;
  // one wave, 4 CTAs a SM at 64 registers, each of at least one step of rows; 6 a SM leave half of
  // a second wave idle (4096 x 4096 gelu: its gradient 92 us, 84 with one wave), 24 a SM make more
  // sums to join (20,000 x 100: 53 us, 39)
  const int64_t step = 256 / g.cx, want = std::max<int64_t>(1, (int64_t)sm_count * 4 / g.gx);
  const int64_t steps = (m + step - 1) / step, per = std::max<int64_t>(1, (steps + want - 1) / want);
  g.rows = per * step;
  g.gy = (m + g.rows - 1) / g.rows;
  return g;
}

template <typename T>
cudaError_t launch_t(const SlopeArgs* s, const PackArgs* packs, int count, int sm_count, cudaStream_t st) {
  PrepareArgs a;
  a.ctas[0] = a.ctas[1] = a.ctas[2] = 0;
  if (s) {
    a.slope = *s;
    a.grid = slope_grid(s->m, s->k, sm_count);
    a.ctas[0] = a.grid.gx * a.grid.gy;
  }
  for (int i = 0; i < count; ++i) {
    a.pack[i] = packs[i];
    a.ctas[1 + i] = std::min<int64_t>((packs[i].rows * ((packs[i].cols + 7) / 8) + 255) / 256, (int64_t)sm_count * 16);
  }
  const int64_t ctas = a.ctas[0] + a.ctas[1] + a.ctas[2];
  if (ctas == 0) return cudaSuccess;
  const cudaError_t e = launch_kernel(prepare_kernel<T>, dim3((unsigned)ctas), 256, 0, st, a);
  if (e != cudaSuccess || !s || s->db == nullptr || a.grid.gy == 1) return e;
  return launch_kernel(sums_kernel<T>, dim3((unsigned)((s->k + 31) / 32)), 256, 0, st, s->ws, a.grid.gy, s->k,
                       static_cast<T*>(s->db));
}

}  // namespace

size_t slope_ws_bytes(int64_t m, int64_t k, int sm_count) {
  const SlopeGrid g = slope_grid(m, k, sm_count);
  return g.gy == 1 ? 0 : (size_t)g.gy * (size_t)k * 4;
}

cudaError_t launch_prepare(fxtx_type_t type, const SlopeArgs* slope, const PackArgs* packs, int count, int sm_count,
                           cudaStream_t st) {
  switch (type) {
    case FXTX_F32: return launch_t<float>(slope, packs, count, sm_count, st);
    case FXTX_BF16: return launch_t<__nv_bfloat16>(slope, packs, count, sm_count, st);
    default: return launch_t<__half>(slope, packs, count, sm_count, st);
  }
}

}  // namespace fxtx
