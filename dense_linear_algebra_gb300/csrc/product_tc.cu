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
#include "product_tc.cuh"

namespace fxtx {
namespace {

constexpr int SPLIT_EPI = 8;      // epilogue warps of the split kernel
constexpr int SPLIT_THREADS = 32 * (4 + SPLIT_EPI);

// The split kernel's stages, and room for a tile's partial sums: two CTAs a SM for tiles of
// up to 64 columns of 16 bits, one of the others.
template <int BN, int PL>
struct SplitCfg : Cfg<1, BN, PL, 64, PL == 3 ? 150 : (BN == 128 ? 128 : 80)> {
  static constexpr int CTAS = PL == 1 && BN <= 64 ? 2 : 1;
  static constexpr int RED = 128 * (BN + 4) * 4;
  static constexpr size_t BYTES = SplitCfg::Cfg::BYTES + RED;
  static_assert(CTAS * (BYTES + 2048) <= 228 * 1024, "shared memory");
};

// One tile a cluster. The CTA of rank r of R finishes lanes r * 128 / R .. of the tile: every
// CTA stores its partial sums of those lanes to r's shared memory (after the stages, which r
// may still be reading), one cluster barrier, and r adds the R parts in order.
template <typename T, int BN, int PL, bool SWAP, bool LONG>
__global__ void __launch_bounds__(SPLIT_THREADS, SplitCfg<BN, PL>::CTAS)
    product_split_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                         const __grid_constant__ TcArgs a) {
  using C = SplitCfg<BN, PL>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[C::S], empty[C::S], tfull[2], tempty[2], fin_bar;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  volatile int* abort_word = &s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int R = a.splits;

  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < C::S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], SPLIT_EPI);
    }
    mbar_init(&fin_bar, 1);
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc<1>(&s_tmem, C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_arrive();  // waited for before the first store to another CTA
  const uint32_t tmem = s_tmem;
  after_previous();

  int l, c;
  place((int)(blockIdx.x / (unsigned)R), a.tiles_l, a.tiles_c, l, c);
  const int k0 = (int)rank * a.per_split, k1 = min(a.kblocks, k0 + a.per_split);
  bool ok = true;
  float sum[PL == 3 ? C::COLS : 1];

  if (warp == 0 || warp == 3) {
    if (elect_one()) {
      const uint32_t st0 = smem_addr(smem);
      Ring<C::S> ring;
      int it = 0;
      for (int kb = k0; kb < k1; ++kb, ++it, ring.next()) {
        if (!(ok = tc_wait(&empty[ring.s], ring.phase ^ 1u, abort_word))) break;
        const uint32_t st = st0 + ring.s * C::STAGE;
        if (warp == 0) {
          mbar_arrive_expect_tx(&full[ring.s], (uint32_t)C::STAGE);
          load_operand<1, PL, C::BK, 128>(&amap, a.a_mn, st, l * 128, kb * C::BK, smem_addr(&full[ring.s]));
        } else {
          load_operand<1, PL, C::BK, C::BROWS>(&bmap, a.b_mn, st + PL * C::A_BYTES, c * BN, kb * C::BK,
                                               smem_addr(&full[ring.s]));
        }
      }
      if (!ok)
        for (int j = it > C::S ? it - C::S : 0; j < it; ++j) mbar_wait_bounded(&full[j % C::S], (uint32_t)((j / C::S) & 1));
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      bool more = true;
      ok = issue_products<1, C, PL, LONG>(a, smem, full, empty, tfull, tempty, tmem, BN, abort_word, [&](int& f0, int& f1) {
        f0 = k0;
        f1 = k1;
        const bool m = more;
        more = false;
        return m;
      });
      mma_commit<1>(&fin_bar);
      mbar_wait_bounded(&fin_bar, 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // the sums into registers (float32), or up to their last product (16 bits)
    const int q = warp & 3, half = (warp - 4) >> 2;
    const bool mine = half * C::COLS < BN;
    if constexpr (PL == 3) {
      const uint32_t t = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(half * C::COLS);
#pragma unroll
      for (int x = 0; x < C::COLS; ++x) sum[x] = 0.f;
      int acc = 0;
      for (int kb = k0; kb < k1; kb += CHUNK, ++acc) {
        if (!(ok = warp_wait(&tfull[acc & 1], (uint32_t)((acc >> 1) & 1), abort_word))) break;
        tc_fence_after();
        if (mine) add_columns<C::COLS>(t + (uint32_t)((acc & 1) * BN), sum);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(smem_addr(&tempty[acc & 1]));
      }
    } else {
      ok = warp_wait(&tfull[0], 0, abort_word);
      tc_fence_after();
      if constexpr (LONG) {
        const uint32_t t = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(half * C::COLS);
        uint32_t phase = 0;
        for (int kb = k0 + a.fold; kb < k1 && ok; kb += a.fold, phase ^= 1u) {
          if (!(ok = warp_wait(&tfull[1], phase, abort_word))) break;
          tc_fence_after();
          auto taken = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(smem_addr(&tempty[1]));
          };
          if (mine) fold_columns<C::COLS>(t + (uint32_t)BN, t, taken);
          else taken();
        }
      }
    }
  }

  // the partial sums to the CTAs that finish them: [from][lane of R-th][column] (rows of the result
  // are lanes), or with SWAP [from][column][lane]
  __syncwarp();
  cluster_wait();
  const int share = 128 / R;  // lanes a CTA finishes
  const int pitch = SWAP ? share : BN + 4, block = SWAP ? BN * share : share * pitch;
  float* red = reinterpret_cast<float*>(smem + (size_t)C::S * C::STAGE);
  if (warp >= 4 && ok) {
    const int q = warp & 3, half = (warp - 4) >> 2, L = 32 * q + lane;
    if (half * C::COLS < BN) {
      const uint32_t t = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(half * C::COLS);
      const uint32_t to = cluster_addr(red, (uint32_t)(L / share)) + (uint32_t)((rank * block) * 4);
#pragma unroll
      for (int x = 0; x < C::COLS; x += 16) {
        float r[16];
        if constexpr (PL == 3) {
#pragma unroll
          for (int i = 0; i < 16; ++i) r[i] = sum[x + i];
        } else {
          tc_load16(t + (uint32_t)x, r);
          tc_wait_ld();
        }
        const int col = half * C::COLS + x;
        if constexpr (SWAP) {
#pragma unroll
          for (int i = 0; i < 16; ++i) st_cluster(to + (uint32_t)(((col + i) * share + L % share) * 4), r[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            st_cluster4(to + (uint32_t)(((L % share) * pitch + col + i) * 4), r[i], r[i + 1], r[i + 2], r[i + 3]);
        }
      }
    }
  }
  tc_fence_before();
  const bool failed = __syncthreads_or(!ok);
  cluster_sync();
  tc_fence_after();
  if (warp == 2) tmem_free<1>(tmem, C::TMEM_COLS);
  if (failed) return;  // FXTX_ERR_TIMEOUT is raised

  const Finish<T> fin(a.e, a.rows, a.cols);
  const int groups = SWAP ? share / 4 : BN / 4, units = SWAP ? BN * groups : share * groups;
  for (int u = tid; u < units; u += SPLIT_THREADS) {
    const int y = u / groups, x = u % groups * 4;
    const int64_t i = SWAP ? (int64_t)c * BN + y : (int64_t)l * 128 + rank * share + y;
    const int64_t j = SWAP ? (int64_t)l * 128 + rank * share + x : (int64_t)c * BN + x;
    if (i >= a.rows || j >= a.cols) continue;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < R; ++s) {
      const float4 p = *reinterpret_cast<const float4*>(red + s * block + y * pitch + x);
      v[0] += p.x; v[1] += p.y; v[2] += p.z; v[3] += p.w;
    }
    fin.template row<4>(i, j, v);
  }
}

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

template <typename T, int BN, int PL, bool SWAP>
cudaError_t launch_split(const CUtensorMap& am, const CUtensorMap& bm, const TcArgs& a, cudaStream_t st) {
  const void* k = PL == 1 && a.fold ? (const void*)product_split_kernel<T, BN, PL, SWAP, PL == 1>
                                    : (const void*)product_split_kernel<T, BN, PL, SWAP, false>;
  return launch_clustered(k, SplitCfg<BN, PL>::BYTES,
                          (unsigned)(a.tiles_l * a.tiles_c * a.splits), SPLIT_THREADS, a.splits, am, bm, a, st);
}

}  // namespace

int take_product_device_error() { return take_device_error(); }

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
  cudaError_t e = cudaErrorInvalidConfiguration;
  if (plan.swap) {
    switch (plan.bn) {
      case 16: e = launch_split<T, 16, PL, true>(am, bm, a, st); break;
      case 32: e = launch_split<T, 32, PL, true>(am, bm, a, st); break;
      case 64: e = launch_split<T, 64, PL, true>(am, bm, a, st); break;
      case 128:
        if constexpr (!F32) e = launch_split<T, 128, PL, true>(am, bm, a, st);
        break;
    }
  } else if (plan.cluster) {
    switch (plan.bn) {
      case 64: e = launch_split<T, 64, PL, false>(am, bm, a, st); break;
      case 128:
        if constexpr (!F32) e = launch_split<T, 128, PL, false>(am, bm, a, st);
        break;
    }
  } else {
    e = launch_persistent<T, 0>(plan, am, bm, a, ModeArgs<0>{}, dev.sm_count, st);
  }
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
