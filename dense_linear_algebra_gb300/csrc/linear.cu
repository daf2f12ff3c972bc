// linear.cu — the product behind the linear layer and its gradient,
//     C_ij = sum_kk A(i, kk) B(j, kk),   out = act(C + bias_j) + R_ij,
// on the CUDA cores: 64 x 64 tiles, 4 x 4 entries a thread, operands staged in shared memory
// 16 of kk at a time, fp32 sums. Long sums are split over the grid's third dimension into
// fp32 partials of at most 4,096 terms that a second kernel adds in order.
#include <algorithm>
#include <type_traits>

#include "act.cuh"
#include "common.cuh"
#include "host.h"
#include "kernels.h"
#include "linear.h"

namespace fxtx {
namespace {

constexpr int TM = 64, TK = 16;

template <typename T>
__device__ __forceinline__ void finish(const Epilogue& e, int64_t i, int64_t j, float c) {
  if (e.bias) c += to_f32(static_cast<const T*>(e.bias)[j]);
  if (e.Z) static_cast<T*>(e.Z)[i * e.ldz + j] = from_f32<T>(c);
  with_act(e.act, [&](auto act) { c = act_of<decltype(act)::value>(c); });
  if (e.R) c += to_f32(static_cast<const T*>(e.R)[i * e.ldr + j]);
  static_cast<T*>(e.out)[i * e.ldo + j] = from_f32<T>(c);
}

template <typename T>
__device__ __forceinline__ void stage(float (*s)[TM + 1], const Operand& o, int64_t i0, int64_t rows, int64_t k0,
                                      int64_t k1) {
  for (int e = threadIdx.x; e < TM * TK; e += 256) {
    const int i = o.mn_major ? e % TM : e / TK, kk = o.mn_major ? e / TM : e % TK;
    const int64_t r = i0 + i, c = k0 + kk;
    float x = 0.f;
    if (r < rows && c < k1) x = to_f32(static_cast<const T*>(o.p)[o.mn_major ? c * o.ld + r : r * o.ld + c]);
    s[kk][i] = x;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) product_kernel(const Product p, const int64_t per_split, float* part) {
  __shared__ float as[TK][TM + 1], bs[TK][TM + 1];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t i0 = (int64_t)blockIdx.x * TM, j0 = (int64_t)blockIdx.y * TM;
  const int64_t k0 = (int64_t)blockIdx.z * per_split, k1 = min(p.K, k0 + per_split);
  float c[4][4] = {};
  for (int64_t k = k0; k < k1; k += TK) {
    stage<T>(as, p.A, i0, p.M, k, k1);
    stage<T>(bs, p.B, j0, p.N, k, k1);
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < TK; ++kk) {
      float x[4], y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        x[q] = as[kk][ty + 16 * q];
        y[q] = bs[kk][tx + 16 * q];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) c[u][v] = fmaf(x[u], y[v], c[u][v]);
    }
    __syncthreads();
  }
  for (int u = 0; u < 4; ++u)
    for (int v = 0; v < 4; ++v) {
      const int64_t i = i0 + ty + 16 * u, j = j0 + tx + 16 * v;
      if (i >= p.M || j >= p.N) continue;
      if (part) part[((int64_t)blockIdx.z * p.M + i) * p.N + j] = c[u][v];
      else finish<T>(p.e, i, j, c[u][v]);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) join_kernel(const Epilogue e, int64_t M, int64_t N, int splits, const float* part) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < M * N; x += stride) {
    float c = 0.f;
    for (int s = 0; s < splits; ++s) c += part[(int64_t)s * M * N + x];
    finish<T>(e, x / N, x % N, c);
  }
}

template <typename T>
fxtx_status_t run_t(const Product& p, const DeviceInfo& dev, cudaStream_t st) {
  const int64_t tm = (p.M + TM - 1) / TM, tn = (p.N + TM - 1) / TM;
  if (tn > 65535) return FXTX_ERR_UNSUPPORTED;
  int64_t splits = 1;
  if (p.K > 4096) splits = std::max<int64_t>(1, std::min<int64_t>((p.K + 4095) / 4096, (int64_t)dev.sm_count * 8 / (tm * tn)));
  int64_t per = ((p.K + splits - 1) / splits + TK - 1) / TK * TK;
  splits = p.K > 0 ? (p.K + per - 1) / per : 1;
  float* part = nullptr;
  if (splits > 1) {
    const fxtx_status_t s = alloc_ws(reinterpret_cast<void**>(&part), (size_t)splits * p.M * p.N * 4, st);
    if (s != FXTX_OK) return s;
  }
  product_kernel<T><<<dim3((unsigned)tm, (unsigned)tn, (unsigned)splits), 256, 0, st>>>(p, per, part);
  cudaError_t e = cudaGetLastError();
  if (part) {
    if (e == cudaSuccess) {
      const int64_t blocks = std::min<int64_t>((p.M * p.N + 255) / 256, (int64_t)dev.sm_count * 8);
      join_kernel<T><<<(unsigned)blocks, 256, 0, st>>>(p.e, p.M, p.N, (int)splits, part);
      e = cudaGetLastError();
    }
    cudaFreeAsync(part, st);
  }
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

}  // namespace

fxtx_status_t run_product(const Product& p, const DeviceInfo& dev, cudaStream_t st) {
  switch (p.type) {
    case FXTX_F32: return run_t<float>(p, dev, st);
    case FXTX_BF16: return run_t<__nv_bfloat16>(p, dev, st);
    default: return run_t<__half>(p, dev, st);
  }
}

}  // namespace fxtx
