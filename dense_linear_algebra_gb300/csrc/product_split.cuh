// product_split.cuh — the product kernel of few tiles, a cluster each; product_tc.cu says how it works. Each file that includes
// this has kernels of its own (internal linkage).
#pragma once

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

// RAW: the sums go to a.part in fp32, as they are.
// One tile a cluster. The CTA of rank r of R finishes lanes r * 128 / R .. of the tile: every
// CTA stores its partial sums of those lanes to r's shared memory (after the stages, which r
// may still be reading), one cluster barrier, and r adds the R parts in order.
template <typename T, int BN, int PL, bool SWAP, bool LONG, bool RAW>
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
      ok = issue_products<1, C, PL, LONG, PL == 3, CHUNK<0>>(a, smem, full, empty, tfull, tempty, tmem, BN, abort_word, [&](int& f0, int& f1) {
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
      for (int kb = k0; kb < k1; kb += CHUNK<0>, ++acc) {
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
    if constexpr (RAW) {
      Finish<float>::template store<4>(a.part + i * a.cols + j, a.cols - j >= 4 ? 4 : (int)(a.cols - j), a.cols % 4 == 0, v);
    } else {
      fin.template row<4>(i, j, v);
    }
  }
}

template <typename T, int BN, int PL, bool SWAP, bool RAW>
cudaError_t launch_split(const CUtensorMap& am, const CUtensorMap& bm, const TcArgs& a, cudaStream_t st) {
  const void* k = PL == 1 && a.fold ? (const void*)product_split_kernel<T, BN, PL, SWAP, PL == 1, RAW>
                                    : (const void*)product_split_kernel<T, BN, PL, SWAP, false, RAW>;
  return launch_clustered(k, SplitCfg<BN, PL>::BYTES,
                          (unsigned)(a.tiles_l * a.tiles_c * a.splits), SPLIT_THREADS, a.splits, am, bm, a, st);
}

// The split kernel that the plan names.
template <typename T, bool RAW>
cudaError_t launch_cluster(const TcPlan& plan, const CUtensorMap& am, const CUtensorMap& bm, const TcArgs& a, cudaStream_t st) {
  constexpr int PL = std::is_same<T, float>::value ? 3 : 1;
  if (plan.swap) {
    switch (plan.bn) {
      case 16: return launch_split<T, 16, PL, true, RAW>(am, bm, a, st);
      case 32: return launch_split<T, 32, PL, true, RAW>(am, bm, a, st);
      case 64: return launch_split<T, 64, PL, true, RAW>(am, bm, a, st);
      case 128:
        if constexpr (PL == 1) return launch_split<T, 128, PL, true, RAW>(am, bm, a, st);
        break;
    }
  } else {
    switch (plan.bn) {
      case 64: return launch_split<T, 64, PL, false, RAW>(am, bm, a, st);
      case 128:
        if constexpr (PL == 1) return launch_split<T, 128, PL, false, RAW>(am, bm, a, st);
        break;
    }
  }
  return cudaErrorInvalidConfiguration;
}

}  // namespace
}  // namespace fxtx
