// product_tc.cu — the products of the linear layer and its gradient on the tensor cores:
//     C_ij = sum_kk A(i, kk) B(j, kk),   out = act(C + bias_j) + R_ij.
//
// Roles of a CTA, linked by mbarriers only:
//   warp 0      one lane: tensor copies of A, 64 or 128 of kk a stage, 128-byte swizzle;
//   warp 3      the same of B;
//   warp 1      the products (tcgen05.mma, K = 16), one elected lane issuing; in a pair the
//               first CTA issues for both, each holding its 128 rows of A and half of B;
//   warps 4 on  the epilogue: a tile's sums from tensor memory (lane = row of the tile), two
//               or four warps a quarter of the lanes, each a part of the columns.
//
// Two kernels share them.
//   product_tc_kernel     many tiles: one persistent CTA a SM, or a pair of CTAs over two SMs
//                         (CG = 2, 256 x 256 tiles), takes tiles in turn; the sums live in two
//                         tensor-memory accumulators, so that the epilogue of one tile overlaps
//                         the products of the next. Few tiles with long sums: the sums are split
//                         and fp32 partials go to a workspace, which join_kernel adds in order.
//   product_split_kernel  few tiles: a cluster of up to 8 CTAs takes one tile, each a part of
//                         kk; every CTA sends each of the others its share of the partial sums
//                         (distributed shared memory) and finishes its own, adding in order: one
//                         launch, no workspace. Stages are few, so that two or more CTAs share a
//                         SM and all of the weights' stream is in flight at once.
//
// Operands may be K-major (kk contiguous) or MN-major: the box of a tensor copy, the descriptor
// and the instruction's major bits change, nothing is transposed. Rows, columns and kk beyond
// the matrices read as zero.
//
// SWAP: the tile's lanes run over the result's columns and its columns over the result's rows,
// for results of few rows: a tile is then 128 columns x BN rows, and the weights are read once
// with no row of the tile wasted.
//
// float32 (PL = 3): each operand comes as three bfloat16 planes (x = hi + mid + lo, exactly),
// and the six products of planes whose order is within 2^-18 of the first are summed; the rest
// is at most 2^-26 of a term. The tensor cores' sums are taken out every 128 of kk and added in
// fp32 registers, rounded to nearest, so that a long sum's error does not grow with its length:
// 2-norm error 6e-7 for 2048^3 normal inputs (8e-7 for the vendor library's fp32 product, which has 1e-7 to 4e-7 where ours has 5e-7 to 6e-7 on some other sizes), 1.5e-6 when taken out every 256
// (5 % faster), 1.3e-7 every 64 (19 % slower).
//
// 16 bits: the tensor cores' sums drop what lies below the accumulator's last bits, 6.3e-9 of a sum of terms of one
// sign for each of kk (measured: 1.0e-4 after 16,384). A sum over more than FOLD of kk is therefore formed in pieces: the
// first in one accumulator, the others in the second, which the epilogue warps add to the first in fp32 (rounded to
// nearest). What is left is 5e-5, a tenth of float16's rounding; 300,000 rows in one piece were 2.7e-4 off. The products
// wait for each addition: 1 to 3 % of sums of 16,384 to 65,536 (65,536 x 4096, 4096 outputs: dW 1,264 to 1,291 us).
// Such sums have kernels of their own (LONG): beside that code the others took 1 to 2 % longer (512 x 4096, 4096
// outputs: 17.9 us, 17.7).
#include "product_split.cuh"
#include "product_tc.cuh"

namespace fxtx {
namespace {

// out = the epilogue of the splits' sums, added in order: 4 neighbouring entries a thread.
template <typename T>
__global__ void __launch_bounds__(256) join_kernel(const Epilogue e, int64_t rows, int64_t cols, int splits,
                                                   const float* part) {
  const Finish<T> fin(e, rows, cols);
  const int64_t groups = (cols + 3) / 4, stride = (int64_t)gridDim.x * 256;
  const bool wide = cols % 4 == 0;
  after_previous();
  for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < rows * groups; x += stride) {
    const int64_t i = x / groups, j = (x - i * groups) * 4;
    const float* p = part + i * cols + j;
    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < splits; ++s, p += rows * cols) {
      if (wide) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        c[0] += v.x; c[1] += v.y; c[2] += v.z; c[3] += v.w;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (j + q < cols) c[q] += p[q];
      }
    }
    fin.template row<4>(i, j, c);
  }
}

}  // namespace

int* product_error_word() { return device_error_word(); }

template <typename T>
fxtx_status_t run_planes(const PlanesProduct& p, const DeviceInfo& dev, cudaStream_t st) {
  constexpr bool F32 = std::is_same<T, float>::value;
  constexpr int PL = F32 ? 3 : 1;
  const TcPlan plan = plan_product(p.M, p.N, p.K, PL, p.A.mn_major, p.B.mn_major, dev.sm_count);
  TcArgs a;
  CUtensorMap am, bm;
  {
    const fxtx_status_t s = prepare_product<T>(p, plan, a, am, bm);
    if (s != FXTX_OK) return s;
  }
  if (!plan.cluster && a.splits > 1) {
    const fxtx_status_t s = alloc_pooled(reinterpret_cast<void**>(&a.part), (size_t)a.splits * p.M * p.N * 4, st);
    if (s != FXTX_OK) return s;
  }
  cudaError_t e = plan.cluster ? launch_cluster<T, false>(plan, am, bm, a, st)
                               : launch_persistent<T, 0>(plan, am, bm, a, ModeArgs<0>{}, dev.sm_count, st);
  if (a.part) {
    if (e == cudaSuccess) {
      const int64_t blocks = std::min<int64_t>((p.M * ((p.N + 3) / 4) + 255) / 256, (int64_t)dev.sm_count * 8);
      e = launch_kernel(join_kernel<T>, dim3((unsigned)blocks), 256, 0, st, a.e, p.M, p.N, a.splits, a.part);
    }
    cudaFreeAsync(a.part, st);
  }
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

template fxtx_status_t run_planes<float>(const PlanesProduct&, const DeviceInfo&, cudaStream_t);
template fxtx_status_t run_planes<__nv_bfloat16>(const PlanesProduct&, const DeviceInfo&, cudaStream_t);
template fxtx_status_t run_planes<__half>(const PlanesProduct&, const DeviceInfo&, cudaStream_t);

}  // namespace fxtx
