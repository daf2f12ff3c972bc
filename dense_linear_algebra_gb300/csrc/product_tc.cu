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
#include <cuda.h>

#include <algorithm>
#include <cstdio>
#include <cstring>
#include <type_traits>

#include "act.cuh"
#include "common.cuh"
#include "host.h"
#include "kernels.h"
#include "linear.h"
#include "product.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace fxtx {
namespace {

constexpr int BX = 64;            // kk of a box of a K-major operand: 128 bytes
constexpr int SPLIT_EPI = 8;      // epilogue warps of the split kernel
constexpr int SPLIT_THREADS = 32 * (4 + SPLIT_EPI);
constexpr int CHUNK = 2;          // stages a sum stays in tensor memory (float32)
constexpr int FOLD = 8192;        // of kk that a piece of a sum covers (16 bits)

// BK: kk a stage; KB: kilobytes the stages may take.
template <int CG, int BN, int PL, int BK_, int KB>
struct Cfg {
  static constexpr int BK = BK_;
  static constexpr int BROWS = BN / CG;            // B's entries a CTA holds
  static constexpr int A_BYTES = 128 * BK * 2;     // one plane of A in a stage
  static constexpr int B_BYTES = BROWS * BK * 2;
  static constexpr int STAGE = PL * (A_BYTES + B_BYTES);
  static constexpr int S = std::min(8, KB * 1024 / STAGE);
  static constexpr size_t BYTES = (size_t)S * STAGE + 1024;
  static constexpr int TMEM_COLS = std::max(32, 2 * BN);
  static constexpr int COLS = BN / 2 >= 16 ? BN / 2 : 16;  // columns an epilogue thread of the split kernel takes
  static_assert(S >= 2 && BYTES <= 227 * 1024 && TMEM_COLS <= 512, "shared and tensor memory");
};

// The persistent kernel's stages, and the epilogue warps' rows. A 16-bit stage is 128 of kk: a turn
// of the copying and of the issuing thread costs 300 to 400 cycles whatever it moves, more
// than the 256 of a 64-wide stage's products.
template <int CG, int BN, int PL>
struct TileCfg : Cfg<CG, BN, PL, PL == 3 ? 64 : 128, 192> {
  // Epilogue warps: few are slow to finish a tile, for the latencies of the exponentials and of the stores (a
  // 128 x 128 tile with silu took 7,600 cycles with eight); 256 columns leave the memory for eight, the sums of
  // float32 the registers.
  static constexpr int EPI = BN == 256 || PL == 3 ? 8 : 16, THREADS = 32 * (4 + EPI);
  static constexpr int COLS = std::max(32, BN / (EPI / 4));  // columns a thread takes
  static constexpr size_t BYTES = TileCfg::Cfg::BYTES + EPI * Tile32<float>::BYTES;
  static_assert(BYTES + 2 * BN * 4 + 512 <= 227 * 1024, "shared memory");
};

// The split kernel's stages, and room for a tile's partial sums: two CTAs a SM for tiles of
// up to 64 columns of 16 bits, one of the others.
template <int BN, int PL>
struct SplitCfg : Cfg<1, BN, PL, 64, PL == 3 ? 150 : (BN == 128 ? 128 : 80)> {
  static constexpr int CTAS = PL == 1 && BN <= 64 ? 2 : 1;
  static constexpr int RED = 128 * (BN + 4) * 4;
  static constexpr size_t BYTES = SplitCfg::Cfg::BYTES + RED;
  static_assert(CTAS * (BYTES + 2048) <= 228 * 1024, "shared memory");
};

// A warp's 32 lanes of COLS tensor-memory columns added to `sum`, 32 on their way at a time.
template <int COLS>
__device__ __forceinline__ void add_columns(uint32_t t, float* sum) {
  constexpr int STEP = COLS < 32 ? COLS : 32;
#pragma unroll
  for (int x = 0; x < COLS; x += STEP) {
    float r[STEP];
#pragma unroll
    for (int y = 0; y < STEP; y += 16) tc_load16(t + (uint32_t)(x + y), r + y);
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < STEP; ++i) sum[x + i] += r[i];
  }
}

// A warp's 32 lanes of COLS tensor-memory columns at `from` added to those at `to`; `taken` is called once the last
// of them have been read.
template <int COLS, typename F>
__device__ __forceinline__ void fold_columns(uint32_t from, uint32_t to, F taken) {
  constexpr int STEP = COLS < 32 ? COLS : 32;
#pragma unroll 1
  for (int x = 0; x < COLS; x += STEP) {
    float r[STEP], s[STEP];
#pragma unroll
    for (int y = 0; y < STEP; y += 16) {
      tc_load16(from + (uint32_t)(x + y), r + y);
      tc_load16(to + (uint32_t)(x + y), s + y);
    }
    tc_wait_ld();
    if (x + STEP == COLS) taken();
#pragma unroll
    for (int i = 0; i < STEP; ++i) s[i] += r[i];
#pragma unroll
    for (int y = 0; y < STEP; y += 16) tc_store16(to + (uint32_t)(x + y), s + y);
  }
  tc_wait_st();
}

struct TcArgs {
  int64_t rows = 0, cols = 0;   // the result's
  int tiles_l = 0, tiles_c = 0;  // tiles along the lanes (A) and the columns (B) of a tile
  int kblocks = 0, splits = 1, per_split = 0;  // stages of kk
  int ksteps = 0;                              // 16 of kk
  int fold = 0;                                // stages a piece of a long 16-bit sum covers; 0: sums in one piece
  bool a_mn = false, b_mn = false;
  uint32_t idesc = 0;
  Epilogue e;
  float* part = nullptr;  // [splits][rows][cols] when splits > 1
};

// Tile `t`'s place: 8 tiles along the lanes at a time, then along the columns, so that the
// tiles in flight share their operands in L2.
__device__ __forceinline__ void place(int t, int tl, int tc, int& l, int& c) {
  const int group = 8 * tc, g = t / group, first = g * 8, size = min(8, tl - first), r = t - g * group;
  l = first + r % size;
  c = r / size;
}

// The tensor copies of one operand of a stage at `d`: kk from k on of its ROWS entries from r on. A
// K-major operand lies in boxes of 64 of kk (ROWS rows of 128 bytes), an MN-major one in boxes of 64
// entries (BK rows of 128 bytes).
template <int CG, int PL, int BK, int ROWS>
__device__ __forceinline__ void load_operand(const CUtensorMap* map, bool mn, uint32_t d, int r, int k, uint32_t bar) {
#pragma unroll
  for (int p = 0; p < PL; ++p, d += ROWS * BK * 2) {
    if (mn) {
#pragma unroll
      for (int x = 0; x < ROWS / 64; ++x) tma_load_3d<CG>(d + x * BK * 128, map, r + 64 * x, k, p, bar);
    } else {
#pragma unroll
      for (int x = 0; x < BK / BX; ++x) tma_load_3d<CG>(d + x * ROWS * 128, map, k + BX * x, r, p, bar);
    }
  }
}

// The products of one stage into the accumulator at `d`; `fresh`: the first of a sum; STEPS: the 16 of kk
// that are inside the matrices, up to all of the stage's.
template <int CG, class C, int PL, int STEPS>
__device__ __forceinline__ void mma_steps(uint32_t d, uint64_t ad, uint64_t bd, const TcArgs& a, bool fresh) {
  // K = 16 further: 32 bytes along a K-major row and the next box after 64, 16 rows of an MN-major
  // operand (in 16-byte units)
  const uint32_t as = a.a_mn ? 128 : 2, bs = a.b_mn ? 128 : 2;
  const uint32_t ax = a.a_mn ? 512 : 128 * 8, bx = a.b_mn ? 512 : C::BROWS * 8;
  // the planes' products, the smallest first
  constexpr int N = PL == 3 ? 6 : 1, PA[6] = {PL == 3 ? 2 : 0, 0, 1, 1, 0, 0}, PB[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
  for (int x = 0; x < N; ++x)
#pragma unroll
    for (int q = 0; q < STEPS; ++q)
      mma_f16<CG>(d, ad + PA[x] * (C::A_BYTES >> 4) + (q % 4) * as + (q / 4) * ax,
                  bd + PB[x] * (C::B_BYTES >> 4) + (q % 4) * bs + (q / 4) * bx, a.idesc, !fresh || x > 0 || q > 0);
}
template <int CG, class C, int PL>
__device__ __forceinline__ void mma_stage(uint32_t d, uint64_t ad, uint64_t bd, const TcArgs& a, bool fresh, int steps) {
  constexpr int Q = C::BK / 16;
  if (steps > Q / 2) mma_steps<CG, C, PL, Q>(d, ad, bd, a, fresh);
  else if (steps > Q / 4) mma_steps<CG, C, PL, Q / 2>(d, ad, bd, a, fresh);
  else mma_steps<CG, C, PL, Q / 4>(d, ad, bd, a, fresh);
}

// The two accumulators as the products take them and the epilogue gives them back: in turn, or (HOME) the first piece of a
// sum in one, the others in the second, and the next sum's first piece in the second too.
template <bool HOME>
struct Turns {
  uint32_t s = 0, phase = 0;  // the accumulator in turn; its barriers' phase (HOME: both's, a bit each)
  uint32_t home = 0;
  __device__ __forceinline__ uint32_t parity() const { return HOME ? phase >> s & 1u : phase; }
  // after a piece of a sum, the `last` or not
  __device__ __forceinline__ void next(bool last) {
    if constexpr (HOME) {
      phase ^= 1u << s;
      s = home ^ 1u;
      if (last) home = s;
    } else {
      s ^= 1u;
      if (s == 0) phase ^= 1u;
    }
  }
};

// The loop of a CTA's products over a ring of stages: one lane's. `tile(k0, k1)` gives the next range of
// stages of kk, false after the last.
template <int CG, class C, int PL, bool LONG, typename F>
__device__ __forceinline__ bool issue_products(const TcArgs& a, unsigned char* smem, uint64_t* full, uint64_t* empty,
                                               uint64_t* tfull, uint64_t* tempty, uint32_t tmem, int bn,
                                               volatile int* abort_word, F tile) {
  const uint64_t ad0 = swizzled_desc(smem_addr(smem), C::BK * 128, 1024);
  const uint64_t bd0 = swizzled_desc(smem_addr(smem + PL * C::A_BYTES), C::BK * 128, 1024);
  Ring<C::S> ring;
  Turns<PL == 3 || LONG> acc;
  bool ready = false;  // the stage in turn was seen full while the last one's products were issued
  int k0, k1;
  while (tile(k0, k1)) {
    int left = 0;  // stages of the piece in hand
    for (int kb = k0; kb < k1; ++kb) {
      const bool fresh = left == 0;
      if (fresh) {
        left = PL == 3 ? min(CHUNK, k1 - kb) : LONG ? min(a.fold, k1 - kb) : k1 - kb;
        if (!tc_wait(&tempty[acc.s], acc.parity() ^ 1u, abort_word)) return false;
      }
      if (!tc_wait(&full[ring.s], ring.phase, abort_word, ready)) return false;
      const uint32_t s = ring.s;
      ring.next();
      ready = mbar_test(&full[ring.s], ring.phase);
      tc_fence_after();
      mma_stage<CG, C, PL>(tmem + acc.s * bn, ad0 + s * (uint32_t)(C::STAGE >> 4), bd0 + s * (uint32_t)(C::STAGE >> 4), a,
                           fresh, a.ksteps - kb * (C::BK / 16));
      mma_commit<CG>(&empty[s]);
      if (--left == 0) {
        mma_commit<CG>(&tfull[acc.s]);
        acc.next(PL == 3 || kb + 1 == k1);
      }
    }
  }
  return true;
}

template <typename T, int CG, int BN, int PL, bool LONG>
__global__ void __launch_bounds__(TileCfg<CG, BN, PL>::THREADS, 1)
    product_tc_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                      const __grid_constant__ TcArgs a) {
  using C = TileCfg<CG, BN, PL>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[C::S], empty[C::S], tfull[2], tempty[2], fin_bar;
  __shared__ __align__(16) float s_bias[2][BN];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  volatile int* abort_word = &s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;

  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < C::S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], C::EPI * CG);
    }
    mbar_init(&fin_bar, 1);
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc<CG>(&s_tmem, C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  after_previous();

  const int tiles = a.tiles_l * a.tiles_c, work = tiles * a.splits;
  const int first = blockIdx.x / CG, step = gridDim.x / CG;
  // the stages of kk a piece of work covers
  auto range = [&](int w, int& k0, int& k1) {
    const int s = w % a.splits;
    k0 = s * a.per_split;
    k1 = min(a.kblocks, k0 + a.per_split);
  };

  if (warp == 0 || warp == 3) {
    // warp 0 copies A, warp 3 B: one lane's turn takes longer than a narrow tile's products
    if (elect_one()) {
      Ring<C::S> ring;
      int it = 0;
      bool ok = true;
      // a pair's copies all complete on its first CTA's barriers
      const uint32_t full0 = CG == 2 ? cluster_addr(&full[0], 0) : smem_addr(&full[0]);
      const uint32_t st0 = smem_addr(smem);
      for (int w = first; w < work && ok; w += step) {
        int l, c, k0, k1;
        place(w / a.splits, a.tiles_l, a.tiles_c, l, c);
        range(w, k0, k1);
        const int ar = l * 128 * CG + (int)rank * 128, br = c * BN + (int)rank * C::BROWS;
        for (int kb = k0; kb < k1; ++kb, ++it, ring.next()) {
          // (the barriers start as if the stages had been emptied once)
          if (!(ok = tc_wait(&empty[ring.s], ring.phase ^ 1u, abort_word))) break;
          const uint32_t st = st0 + ring.s * C::STAGE;
          if (warp == 0) {
            if (rank == 0) mbar_arrive_expect_tx(&full[ring.s], (uint32_t)(CG * C::STAGE));
            load_operand<CG, PL, C::BK, 128>(&amap, a.a_mn, st, ar, kb * C::BK, full0 + ring.s * 8);
          } else {
            load_operand<CG, PL, C::BK, C::BROWS>(&bmap, a.b_mn, st + PL * C::A_BYTES, br, kb * C::BK, full0 + ring.s * 8);
          }
        }
      }
      // copies still in flight after an abort land before the CTA leaves
      if (!ok && rank == 0)
        for (int j = it > C::S ? it - C::S : 0; j < it; ++j) mbar_wait_bounded(&full[j % C::S], (uint32_t)((j / C::S) & 1));
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      int w = first;
      issue_products<CG, C, PL, LONG>(a, smem, full, empty, tfull, tempty, tmem, BN, abort_word, [&](int& k0, int& k1) {
        if (w >= work) return false;
        range(w, k0, k1);
        w += step;
        return true;
      });
      // every product has completed before the CTA leaves, after an abort too
      mma_commit<CG>(&fin_bar);
      mbar_wait_bounded(&fin_bar, 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int q = warp & 3, group = (warp - 4) >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(group * C::COLS);
    const uint32_t te0 = CG == 2 ? cluster_addr(&tempty[0], 0) : smem_addr(&tempty[0]);
    unsigned char* buf = smem + (size_t)C::S * C::STAGE + (warp - 4) * Tile32<T>::BYTES;
    bool ok = true;
    const bool wide_out = Finish<T>::wide(a.e.out, a.e.ldo), wide_z = Finish<T>::wide(a.e.Z, a.e.ldz),
               wide_r = Finish<T>::wide(a.e.R, a.e.ldr);
    int turn = 0;
    Turns<PL == 3 || LONG> acc;
    // whether the products of the accumulator in turn are there
    auto wait_full = [&]() {
      if (!(ok = warp_wait(&tfull[acc.s], acc.parity(), abort_word))) return false;
      tc_fence_after();
      return true;
    };
    // accumulator x may be taken again
    auto release = [&](uint32_t x) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(te0 + x * 8);
    };
    // (after an abort a warp goes on to meet the others at each tile's barrier, and does nothing else)
    for (int w = first; w < work; w += step, ++turn) {
      int l, c, k0, k1;
      place(w / a.splits, a.tiles_l, a.tiles_c, l, c);
      range(w, k0, k1);
      const int64_t i0 = (int64_t)l * 128 * CG + rank * 128 + 32 * q;  // the warp's first row of the result
      const int64_t j0 = (int64_t)c * BN + group * C::COLS;            // and its first column
      float* part = a.splits > 1 ? a.part + (int64_t)(w % a.splits) * a.rows * a.cols : nullptr;
      // the tile's biases, read while its products run (the buffers alternate, and all epilogue warps
      // meet here once a tile)
      float* bias = s_bias[turn & 1];
      for (int e = tid - 128; e < BN; e += 32 * C::EPI)
        bias[e] = a.e.bias && !part && (int64_t)c * BN + e < a.cols ? to_f32(static_cast<const T*>(a.e.bias)[c * (int64_t)BN + e]) : 0.f;
      asm volatile("bar.sync 1, %0;" ::"n"(32 * C::EPI) : "memory");
      if (!ok) continue;
      if (group * C::COLS >= BN) {  // a narrow tile's spare warps only give its accumulators back
        for (int kb = k0; kb < k1;) {
          if (!wait_full()) break;
          release(acc.s);
          kb += PL == 3 ? CHUNK : LONG ? a.fold : k1 - k0;
          acc.next(PL == 3 || kb >= k1);
        }
        continue;
      }
      bias += group * C::COLS;
      using Tile = Tile32<T>;
      const T* R = static_cast<const T*>(a.e.R);
      // the residual's first rows are on their way while the products run
      uint4 next[Tile::CH];
      if (R && !part) Tile::fetch(next, R, a.e.ldr, wide_r, i0, a.rows, j0, a.cols);

      uint32_t held = acc.s;  // the accumulator with the whole sum
      uint32_t t = lane_base + held * BN;
      if constexpr (PL == 1) {
        if (!wait_full()) continue;
        acc.next(!LONG || k0 + a.fold >= k1);
        if constexpr (LONG) {
          for (int kb = k0 + a.fold; kb < k1; kb += a.fold) {
            if (!wait_full()) break;
            const uint32_t x = acc.s;
            fold_columns<C::COLS>(lane_base + x * BN, t, [&] { release(x); });
            acc.next(kb + a.fold >= k1);
          }
          if (!ok) continue;
        }
      } else {
        float sum[C::COLS];
#pragma unroll
        for (int x = 0; x < C::COLS; ++x) sum[x] = 0.f;
        for (int kb = k0; kb < k1; kb += CHUNK) {
          if (kb > k0) release(held);
          held = acc.s;
          t = lane_base + held * BN;
          if (!wait_full()) break;
          acc.next(true);
          add_columns<C::COLS>(t, sum);
        }
        if (!ok) continue;
        // the sums go back to where the last of them came from: what follows reads them 16 columns at a time
        // in a loop (unrolled over registers its code would not fit the instruction cache)
#pragma unroll
        for (int x = 0; x < C::COLS; x += 16) tc_store16(t + (uint32_t)x, sum + x);
        tc_wait_st();
      }
      // 16 sums of the lane's row from column x on, with their biases
      auto get = [&](int x, float* v) {
        tc_load16(t + (uint32_t)x, v);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 b = *reinterpret_cast<const float4*>(bias + x + i);
          v[i] += b.x; v[i + 1] += b.y; v[i + 2] += b.z; v[i + 3] += b.w;
        }
      };
      if (part) {
#pragma unroll 1
        for (int x = 0; x < C::COLS; x += 16) {
          float v[16];
          get(x, v);
          Tile32<float>::put(buf, 0, v);
          __syncwarp();
          Tile32<float>::drain(buf, part, a.cols, a.cols % 4 == 0, i0, a.rows, j0 + x, a.cols);
          __syncwarp();
        }
        release(held);
        continue;
      }
#pragma unroll 1
      for (int x = 0; x < C::COLS; x += Tile::W) {
        if (a.e.Z) {
#pragma unroll 1
          for (int y = 0; y < Tile::W; y += 16) {
            float v[16];
            get(x + y, v);
            Tile::put(buf, y, v);
          }
          __syncwarp();
          Tile::drain(buf, static_cast<T*>(a.e.Z), a.e.ldz, wide_z, i0, a.rows, j0 + x, a.cols);
          __syncwarp();
        }
        if (R) {
          Tile::place(buf, next);
          if (x + Tile::W < C::COLS) Tile::fetch(next, R, a.e.ldr, wide_r, i0, a.rows, j0 + x + Tile::W, a.cols);
          __syncwarp();
        }
#pragma unroll 1
        for (int y = 0; y < Tile::W; y += 16) {
          float v[16];
          get(x + y, v);
          with_act(a.e.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = act_of<decltype(act)::value, T>(v[i]);
          });
          if (R) Tile::add(buf, y, v);
          Tile::put(buf, y, v);
        }
        __syncwarp();
        Tile::drain(buf, static_cast<T*>(a.e.out), a.e.ldo, wide_out, i0, a.rows, j0 + x, a.cols);
        __syncwarp();
      }
      release(held);
    }
  }

  // tensor memory is released, and a pair's shared memory given up, when all roles are done
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) {
    // the pair's second CTA receives the first one's commits too: the last of them has landed
    if (rank == 1 && warp == 1) mbar_wait_bounded(&fin_bar, 0);
    __syncthreads();
    cluster_sync();
  }
  tc_fence_after();
  if (warp == 2) tmem_free<CG>(tmem, C::TMEM_COLS);
}

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

cudaError_t launch_clustered(const void* k, size_t smem, unsigned grid, int threads, int cluster, const CUtensorMap& am,
                             const CUtensorMap& bm, const TcArgs& a, cudaStream_t st) {
  cudaError_t e = ensure_smem(k, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // (see after_previous)
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  void* args[] = {const_cast<CUtensorMap*>(&am), const_cast<CUtensorMap*>(&bm), const_cast<TcArgs*>(&a)};
  return cudaLaunchKernelExC(&cfg, k, args);
}

template <typename T, int CG, int BN, int PL>
cudaError_t launch(const CUtensorMap& am, const CUtensorMap& bm, const TcArgs& a, int sm_count, cudaStream_t st) {
  const int64_t work = (int64_t)a.tiles_l * a.tiles_c * a.splits;
  const void* k = PL == 1 && a.fold ? (const void*)product_tc_kernel<T, CG, BN, PL, PL == 1>
                                    : (const void*)product_tc_kernel<T, CG, BN, PL, false>;
  return launch_clustered(k, TileCfg<CG, BN, PL>::BYTES,
                          (unsigned)(std::min<int64_t>(work, sm_count / CG) * CG), TileCfg<CG, BN, PL>::THREADS, CG, am, bm, a, st);
}

template <typename T, int BN, int PL, bool SWAP>
cudaError_t launch_split(const CUtensorMap& am, const CUtensorMap& bm, const TcArgs& a, cudaStream_t st) {
  const void* k = PL == 1 && a.fold ? (const void*)product_split_kernel<T, BN, PL, SWAP, PL == 1>
                                    : (const void*)product_split_kernel<T, BN, PL, SWAP, false>;
  return launch_clustered(k, SplitCfg<BN, PL>::BYTES,
                          (unsigned)(a.tiles_l * a.tiles_c * a.splits), SPLIT_THREADS, a.splits, am, bm, a, st);
}

// The map of an operand for boxes of 128 bytes x its tile's rows (or a stage's kk of them, MN-major).
bool operand_map(CUtensorMap* map, const Planes& o, bool bf16, int box_rows, int bk) {
  return encode_planes_map(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, o.p, o.planes,
                           o.rows, o.cols, o.pitch * 2, o.plane_stride * 2, o.mn_major ? bk : box_rows);
}

int stage_of(const TcPlan& plan, int planes) { return planes == 1 && !plan.cluster ? 128 : 64; }

}  // namespace

int take_product_device_error() { return take_device_error(); }

template <typename T>
fxtx_status_t run_planes(const PlanesProduct& p, const DeviceInfo& dev, cudaStream_t st) {
  constexpr bool F32 = std::is_same<T, float>::value;
  constexpr int PL = F32 ? 3 : 1;
  const bool bf16 = !std::is_same<T, __half>::value;
  const TcPlan plan = plan_product(p.M, p.N, p.K, PL, p.A.mn_major, p.B.mn_major, dev.sm_count);
  if (log_enabled())
    fprintf(stderr, "[fxtx] product M=%lld N=%lld K=%lld planes=%d %s%s cg=%d bn=%d splits=%d\n", (long long)p.M,
            (long long)p.N, (long long)p.K, PL, plan.swap ? "swap " : "", plan.cluster ? "cluster" : "persistent", plan.cg,
            plan.bn, plan.splits);
  const Planes &A = plan.swap ? p.B : p.A, &B = plan.swap ? p.A : p.B;
  TcArgs a;
  a.rows = p.M;
  a.cols = p.N;
  const int64_t L = plan.swap ? p.N : p.M, Cn = plan.swap ? p.M : p.N;
  a.tiles_l = (int)((L + 128 * plan.cg - 1) / (128 * plan.cg));
  a.tiles_c = (int)((Cn + plan.bn - 1) / plan.bn);
  const int bk = stage_of(plan, PL);
  a.kblocks = (int)((p.K + bk - 1) / bk);
  a.ksteps = (int)((p.K + 15) / 16);
  a.per_split = (a.kblocks + plan.splits - 1) / plan.splits;
  a.splits = (a.kblocks + a.per_split - 1) / a.per_split;  // none of them empty
  if (PL == 1 && (int64_t)a.per_split * bk > FOLD) a.fold = FOLD / bk;
  // a cluster's CTAs share the tile's 128 lanes out evenly, and each has work
  if (plan.cluster && (a.splits != plan.splits || 128 % a.splits != 0 || a.splits > 8)) return FXTX_ERR_UNSUPPORTED;
  a.a_mn = A.mn_major;
  a.b_mn = B.mn_major;
  a.idesc = mma_desc(bf16, A.mn_major, B.mn_major, 128 * plan.cg, plan.bn);
  a.e = p.e;
  CUtensorMap am, bm;
  memset(&am, 0, sizeof am);
  memset(&bm, 0, sizeof bm);
  if (!operand_map(&am, A, bf16, 128, bk) || !operand_map(&bm, B, bf16, plan.bn / plan.cg, bk)) return FXTX_ERR_CUDA;
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
  } else if (plan.cg == 2) {
    switch (plan.bn) {
      case 128: e = launch<T, 2, 128, PL>(am, bm, a, dev.sm_count, st); break;
      case 256:
        if constexpr (!F32) e = launch<T, 2, 256, PL>(am, bm, a, dev.sm_count, st);
        break;
    }
  } else {
    switch (plan.bn) {
      case 64: e = launch<T, 1, 64, PL>(am, bm, a, dev.sm_count, st); break;
      case 128: e = launch<T, 1, 128, PL>(am, bm, a, dev.sm_count, st); break;
    }
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
