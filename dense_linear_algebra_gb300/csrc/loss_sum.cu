// loss_sum.cu — products whose sums go over pieces: out = down (C + what earlier pieces left), or that kept in fp32 for
// the next piece (mode 3 of product_tc.cuh).
#include "product_tc.cuh"

namespace fxtx {
namespace {

// The same from the parts of split sums, added in order: 4 neighbouring entries a thread.
template <typename T>
__global__ void __launch_bounds__(256) sum_join_kernel(const __grid_constant__ ModeArgs<3> x, void* out, int64_t ldo, int64_t rows,
                                                       int64_t cols, int splits, const float* part) {
  const int64_t groups = (cols + 3) / 4, stride = (int64_t)gridDim.x * 256;
  const bool whole = cols % 4 == 0, wide_out = Finish<T>::wide(out, ldo);
  after_previous();
  const float down = x.scales ? x.scales[1] : 1.f;
  for (int64_t y = (int64_t)blockIdx.x * 256 + threadIdx.x; y < rows * groups; y += stride) {
    const int64_t i = y / groups, j = (y - i * groups) * 4, at = i * cols + j;
    const int n = cols - j >= 4 ? 4 : (int)(cols - j);
    float c[4] = {0.f, 0.f, 0.f, 0.f}, v[4];
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      Finish<float>::load<4>(part + s * rows * cols + at, n, whole, v);
#pragma unroll
      for (int q = 0; q < 4; ++q) c[q] += v[q];
    }
    if (x.in) {
      Finish<float>::load<4>(x.in + at, n, whole, v);
#pragma unroll
      for (int q = 0; q < 4; ++q) c[q] += v[q];
    }
    if (x.keep) {
      Finish<float>::store<4>(x.keep + at, n, whole, c);
      continue;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) c[q] *= down;
    Finish<T>::template store<4>(static_cast<T*>(out) + i * ldo + j, n, wide_out, c);
  }
}

template <typename T>
cudaError_t join(const ModeArgs<3>& x, void* out, int64_t ldo, int64_t rows, int64_t cols, int64_t parts, const float* part,
                 const DeviceInfo& dev, cudaStream_t st) {
  const int64_t blocks = std::min<int64_t>((rows * ((cols + 3) / 4) + 255) / 256, (int64_t)dev.sm_count * 8);
  return launch_kernel(sum_join_kernel<T>, dim3((unsigned)blocks), 256, 0, st, x, out, ldo, rows, cols, (int)parts, part);
}

template <typename T>
fxtx_status_t run_t(const PlanesProduct& p, const ModeArgs<3>& x, const DeviceInfo& dev, cudaStream_t st) {
  const TcPlan plan =
      plan_persistent(p.M, p.N, p.K, std::is_same<T, float>::value ? 3 : 1, p.A.mn_major, p.B.mn_major, dev.sm_count, INT64_MAX);
  TcArgs a;
  CUtensorMap am, bm;
  fxtx_status_t s = prepare_product<T>(p, plan, a, am, bm);
  if (s != FXTX_OK) return s;
  if (a.splits > 1) {
    s = alloc_pooled(reinterpret_cast<void**>(&a.part), (size_t)a.splits * p.M * p.N * 4, st);
    if (s != FXTX_OK) return s;
  }
  cudaError_t e = launch_persistent<T, 3>(plan, am, bm, a, x, dev.sm_count, st);
  if (a.part) {
    if (e == cudaSuccess) e = join<T>(x, p.e.out, p.e.ldo, p.M, p.N, a.splits, a.part, dev, st);
    cudaFreeAsync(a.part, st);
  }
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

}  // namespace

int* sum_error_word() { return device_error_word(); }

fxtx_status_t join_sums(fxtx_type_t type, const ModeArgs<3>& x, void* out, int64_t ldo, int64_t rows, int64_t cols, int64_t parts,
                        const float* part, const DeviceInfo& dev, cudaStream_t st) {
  cudaError_t e;
  switch (type) {
    case FXTX_F32: e = join<float>(x, out, ldo, rows, cols, parts, part, dev, st); break;
    case FXTX_BF16: e = join<__nv_bfloat16>(x, out, ldo, rows, cols, parts, part, dev, st); break;
    default: e = join<__half>(x, out, ldo, rows, cols, parts, part, dev, st); break;
  }
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

fxtx_status_t run_sum(fxtx_type_t type, const PlanesProduct& p, const ModeArgs<3>& x, const DeviceInfo& dev, cudaStream_t st) {
  switch (type) {
    case FXTX_F32: return run_t<float>(p, x, dev, st);
    case FXTX_BF16: return run_t<__nv_bfloat16>(p, x, dev, st);
    default: return run_t<__half>(p, x, dev, st);
  }
}

}  // namespace fxtx
