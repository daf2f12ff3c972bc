// product_tc.cuh — the persistent product kernel on the tensor cores and its launch; product_tc.cu says how it works. What is
// done with a tile's sums is its MODE:
//   0  the layer's epilogue: out = act(C + bias_j) + R_ij
//   1  softmax statistics: of each row, over the columns that a thread takes, the largest C + bias_j and the sum of
//      exp(C + bias_j - that), and the entry of the row's label
//   2  the gradient of softmax cross entropy at C + bias: g_i (exp(C + bias_j - lse_i) - [j = label_i]), stored as an operand
//      of the products that follow, and its column sums
//   3  sums over pieces: out = scale (C + what earlier pieces left), or C + that kept in fp32 for the next piece
//   4  C in fp32 (in any mode, the parts of split sums are stored so)
// Each file that includes this has kernels of its own (internal linkage).
#pragma once

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
#include "loss.h"
#include "product.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace fxtx {
namespace {

constexpr int BX = 64;            // kk of a box of a K-major operand: 128 bytes
// Stages of 64 of kk that a float32 sum stays in tensor memory: two, one for logits that an epilogue takes, whose error is that of
// their exponentials (2-norm error of 2048^3: 6e-7, 1.3e-7 and 19 % more time). The logits of few rows that are written out are a
// layer's: two.
template <int MODE>
constexpr int CHUNK = MODE == 1 || MODE == 2 ? 1 : 2;
constexpr int FOLD = 8192;        // of kk that a piece of a sum covers (16 bits)
constexpr int LOGIT_FOLD = 1024;  // of logits, which are not rounded to 16 bits

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

// A warp's 32 lanes of COLS tensor-memory columns added to `sum`, 32 on their way at a time (16 where the sums themselves fill
// the registers).
template <int COLS>
__device__ __forceinline__ void add_columns(uint32_t t, float* sum) {
  constexpr int STEP = COLS < 32 ? COLS : COLS > 64 ? 16 : 32;
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
  float* part = nullptr;  // [splits][rows][cols] where the sums are split, or wanted as they are
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

// z = v where `is` holds. (A chain of selections by an index is compiled into an array in local memory: D's epilogue took twice
// its time with one.)
__device__ __forceinline__ void take_if(float& z, float v, bool is) {
  asm("{\n.reg .pred p;\nsetp.ne.b32 p, %2, 0;\n@p mov.f32 %0, %1;\n}" : "+f"(z) : "f"(v), "r"((int)is));
}

// The sums over a warp's lanes of N (16 or 32) values of each, column y's to p[y] for y < left: each step, a lane gives half of
// its columns away, until one is left.
template <int N>
__device__ __forceinline__ void column_sums(const float* v, float* p, int64_t left, bool store) {
  const int lane = threadIdx.x & 31;
  float s[N];
#pragma unroll
  for (int y = 0; y < N; ++y) s[y] = v[y];
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1)
#pragma unroll
    for (int y = 0; y < o; ++y) {
      const bool upper = lane & o;
      const float give = upper ? s[y] : s[y + o];
      s[y] = (upper ? s[y + o] : s[y]) + shfl_xor(give, o);
    }
  if constexpr (N == 16) s[0] += shfl_xor(s[0], 16);
  if (store && lane < N && lane < left) p[lane] = s[0];
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
template <int CG, class C, int PL, bool LONG, bool REGS, int PIECE, typename F>
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
        left = PL == 3 ? min(PIECE, k1 - kb) : LONG ? min(a.fold, k1 - kb) : k1 - kb;
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
        acc.next(REGS || kb + 1 == k1);
      }
    }
  }
  return true;
}

template <typename T, int CG, int BN, int PL, bool LONG, int MODE>
__global__ void __launch_bounds__(TileCfg<CG, BN, PL>::THREADS, 1)
    product_tc_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                      const __grid_constant__ TcArgs a, const __grid_constant__ ModeArgs<MODE> mode) {
  using C = TileCfg<CG, BN, PL>;
  // the pieces of a sum are added up in registers, each freeing its accumulator: float32, and logits, whose pieces are short
  constexpr bool REGS = PL == 3 || ((MODE == 1 || MODE == 2) && LONG);
  // and taken from there too: D's epilogue is as long as the products of a piece, which waited for the accumulator that it held (D of
  // 8192 x 2048, 32,768 classes 648 us; from registers 593, in pieces of 8,192 features 579)
  constexpr bool FROM_REGS = MODE == 2 && PL == 1 && LONG;
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
      issue_products<CG, C, PL, LONG, REGS, CHUNK<MODE>>(a, smem, full, empty, tfull, tempty, tmem, BN, abort_word, [&](int& k0, int& k1) {
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
      float* part = a.part ? a.part + (int64_t)(w % a.splits) * a.rows * a.cols : nullptr;
      // the tile's biases, read while its products run (the buffers alternate, and all epilogue warps
      // meet here once a tile)
      float* bias = s_bias[turn & 1];
      for (int e = tid - 128; e < BN; e += 32 * C::EPI) {
        if constexpr (MODE == 1) {
          // columns beyond the last are no classes
          if ((int64_t)c * BN + e >= a.cols) {
            bias[e] = -INFINITY;
            continue;
          }
        }
        bias[e] = a.e.bias && !part && (int64_t)c * BN + e < a.cols ? to_f32(static_cast<const T*>(a.e.bias)[c * (int64_t)BN + e]) : 0.f;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * C::EPI) : "memory");
      if (!ok) continue;
      if (group * C::COLS >= BN) {  // a narrow tile's spare warps only give its accumulators back
        for (int kb = k0; kb < k1;) {
          if (!wait_full()) break;
          release(acc.s);
          kb += PL == 3 ? CHUNK<MODE> : LONG ? a.fold : k1 - k0;
          acc.next(REGS || kb >= k1);
        }
        continue;
      }
      bias += group * C::COLS;
      using Tile = Tile32<T>;
      const T* R = static_cast<const T*>(a.e.R);
      // the residual's first rows are on their way while the products run
      uint4 next[Tile::CH];
      if (MODE == 0 && R && !part) Tile::fetch(next, R, a.e.ldr, wide_r, i0, a.rows, j0, a.cols);

      float sum[REGS ? C::COLS : 1];
      uint32_t held = acc.s;  // the accumulator with the whole sum
      uint32_t t = lane_base + held * BN;
      if constexpr (!REGS) {
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
#pragma unroll
        for (int x = 0; x < C::COLS; ++x) sum[x] = 0.f;
        const int piece = PL == 3 ? CHUNK<MODE> : a.fold;
        for (int kb = k0; kb < k1; kb += piece) {
          if (kb > k0) release(held);
          held = acc.s;
          t = lane_base + held * BN;
          if (!wait_full()) break;
          acc.next(true);
          add_columns<C::COLS>(t, sum);
        }
        if (!ok) continue;
        if constexpr (FROM_REGS) {
          release(held);
        } else {
          // the sums go back to where the last of them came from: what follows reads them 16 columns at a time
          // in a loop (unrolled over registers its code would not fit the instruction cache)
#pragma unroll
          for (int x = 0; x < C::COLS; x += 16) tc_store16(t + (uint32_t)x, sum + x);
          tc_wait_st();
        }
      }
      // 16 sums of the lane's row from column x on, with their biases
      auto get = [&](int x, float* v) {
        if constexpr (FROM_REGS) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = sum[x + i];
        } else {
          tc_load16(t + (uint32_t)x, v);
          tc_wait_ld();
        }
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 b = *reinterpret_cast<const float4*>(bias + x + i);
          v[i] += b.x; v[i + 1] += b.y; v[i + 2] += b.z; v[i + 3] += b.w;
        }
      };
      if constexpr (!FROM_REGS) {  // (such sums are not split)
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
      }
      if constexpr (MODE == 0) {
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
      } else if constexpr (MODE == 1) {
        // the largest so far, and the sum of the exponentials from it; where there is only -inf, that is not subtracted
        const int64_t i = i0 + lane, label = i < a.rows ? label_at(mode.labels, mode.labels64, i, mode.count) - mode.col0 - j0 : -1;
        const int at = label >= 0 && label < C::COLS ? (int)label : -1;
        float top = -INFINITY, sum = 0.f;
#pragma unroll 1
        for (int x = 0; x < C::COLS; x += 16) {
          float v[16];
          get(x, v);
          float most = top;
#pragma unroll
          for (int y = 0; y < 16; ++y) most = fmaxf(most, v[y]);
          const float from = most == -INFINITY ? 0.f : most;
          sum *= exp_of<T>(top - from);
          top = most;
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int y = 0; y < 16; ++y) s4[y & 3] += exp_of<T>(v[y] - from);
          sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
          if (__any_sync(FULL_MASK, at >= x && at < x + 16)) {
            float z = 0.f;
#pragma unroll
            for (int y = 0; y < 16; ++y) take_if(z, v[y], at - x == y);
            if (at >= x && at < x + 16) mode.target[i] = z;
          }
        }
        if (i < a.rows) mode.stats[((int64_t)c * (BN / C::COLS) + group) * a.rows + i] = make_float2(top, sum);
      } else if constexpr (MODE == 2) {
        using S = typename std::conditional<PL == 3, __nv_bfloat16, T>::type;
        using Out = Tile32<S>;  // 32 columns
        const int64_t i = i0 + lane, own = i < a.rows ? label_at(mode.labels, mode.labels64, i, mode.count) : -1;
        const bool on = own >= 0;
        const int64_t label = own - mode.col0 - j0;
        const int at = on && label >= 0 && label < C::COLS ? (int)label : -1;
        const float lse = on ? mode.lse[i] : 0.f;
        float g = on ? mode.gain : 0.f;
        if (on && mode.g) g *= mode.g[i];
        if (mode.scales) g *= mode.scales[0];
        const bool wide = Finish<S>::wide(mode.D, mode.ldd) && mode.d_planes % 8 == 0;
        if constexpr (PL == 1) {
          auto columns = [&](int x) {  // 32
            auto half = [&](int y) {
              float v[16];
              get(x + y, v);
#pragma unroll
              for (int q = 0; q < 16; ++q) v[q] = on ? g * exp_of<T>(v[q] - lse) : 0.f;
              if (__any_sync(FULL_MASK, at >= x + y && at < x + y + 16)) {
#pragma unroll
                for (int q = 0; q < 16; ++q) v[q] -= at - x - y == q ? g : 0.f;
              }
              Out::put(buf, y, v);
              if (mode.sums) column_sums<16>(v, mode.sums + i0 / 32 * mode.sums_ld + j0 + x + y, a.cols - j0 - x - y, i0 < a.rows);
            };
            if constexpr (FROM_REGS) {
              half(0);
              half(16);
            } else {
#pragma unroll 1
              for (int y = 0; y < 32; y += 16) half(y);
            }
            __syncwarp();
            Out::drain(buf, static_cast<S*>(mode.D), mode.ldd, wide, i0, a.rows, j0 + x, a.cols);
            __syncwarp();
          };
          // (columns beyond the last: the whole warp's)
          if constexpr (FROM_REGS) {
#pragma unroll
            for (int x = 0; x < C::COLS; x += 32)
              if (j0 + x < a.cols) columns(x);
          } else {
#pragma unroll 1
            for (int x = 0; x < C::COLS && j0 + x < a.cols; x += 32) columns(x);
          }
        } else {
#pragma unroll 1
          for (int x = 0; x < C::COLS; x += 32) {
            if (j0 + x >= a.cols) break;
            float v[32];
#pragma unroll
            for (int y = 0; y < 32; y += 16) get(x + y, v + y);
#pragma unroll
            for (int y = 0; y < 32; ++y) v[y] = on ? g * exp_of<T>(v[y] - lse) : 0.f;
            if (__any_sync(FULL_MASK, at >= x && at < x + 32)) {
#pragma unroll
              for (int y = 0; y < 32; ++y) v[y] -= at - x == y ? g : 0.f;
            }
            if (mode.sums) column_sums<32>(v, mode.sums + i0 / 32 * mode.sums_ld + j0 + x, a.cols - j0 - x, i0 < a.rows);
#pragma unroll
            for (int p = 0; p < PL; ++p) {
#pragma unroll
              for (int y = 0; y < 32; y += 16) Out::put(buf, y, v + y);
              __syncwarp();
              Out::drain(buf, static_cast<S*>(mode.D) + p * mode.d_planes, mode.ldd, wide, i0, a.rows, j0 + x, a.cols);
              __syncwarp();
#pragma unroll
              for (int y = 0; y < 32; ++y) v[y] -= to_f32(from_f32<S>(v[y]));  // exact
            }
          }
        }
      } else if constexpr (MODE == 3) {
        const float down = mode.scales ? mode.scales[1] : 1.f;
        const bool wide_in = Finish<float>::wide(mode.in, a.cols), wide_keep = Finish<float>::wide(mode.keep, a.cols);
#pragma unroll 1
        for (int x = 0; x < C::COLS; x += Tile::W) {
          float v[Tile::W];
#pragma unroll
          for (int y = 0; y < Tile::W; y += 16) {
            get(x + y, v + y);
            if (mode.in) {
              uint4 r[Tile32<float>::CH];
              Tile32<float>::fetch(r, mode.in, a.cols, wide_in, i0, a.rows, j0 + x + y, a.cols);
              Tile32<float>::place(buf, r);
              __syncwarp();
              Tile32<float>::add(buf, 0, v + y);
              __syncwarp();
            }
            if (mode.keep) {
              Tile32<float>::put(buf, 0, v + y);
              __syncwarp();
              Tile32<float>::drain(buf, mode.keep, a.cols, wide_keep, i0, a.rows, j0 + x + y, a.cols);
              __syncwarp();
            }
          }
          if (mode.keep) continue;
#pragma unroll
          for (int y = 0; y < Tile::W; y += 16) {
#pragma unroll
            for (int q = 0; q < 16; ++q) v[y + q] *= down;
            Tile::put(buf, y, v + y);
          }
          __syncwarp();
          Tile::drain(buf, static_cast<T*>(a.e.out), a.e.ldo, wide_out, i0, a.rows, j0 + x, a.cols);
          __syncwarp();
        }
      }
      if constexpr (!FROM_REGS) release(held);
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

// (`mode`: the kernel's last argument, where it has one)
cudaError_t launch_clustered(const void* k, size_t smem, unsigned grid, int threads, int cluster, const CUtensorMap& am,
                             const CUtensorMap& bm, const TcArgs& a, cudaStream_t st, const void* mode = nullptr) {
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
  void* args[] = {const_cast<CUtensorMap*>(&am), const_cast<CUtensorMap*>(&bm), const_cast<TcArgs*>(&a), const_cast<void*>(mode)};
  return cudaLaunchKernelExC(&cfg, k, args);
}

template <typename T, int CG, int BN, int PL, int MODE>
cudaError_t launch(const CUtensorMap& am, const CUtensorMap& bm, const TcArgs& a, const ModeArgs<MODE>& mode, int sm_count,
                   cudaStream_t st) {
  const int64_t work = (int64_t)a.tiles_l * a.tiles_c * a.splits;
  const void* k = PL == 1 && a.fold ? (const void*)product_tc_kernel<T, CG, BN, PL, PL == 1, MODE>
                                    : (const void*)product_tc_kernel<T, CG, BN, PL, false, MODE>;
  return launch_clustered(k, TileCfg<CG, BN, PL>::BYTES, (unsigned)(std::min<int64_t>(work, sm_count / CG) * CG),
                          TileCfg<CG, BN, PL>::THREADS, CG, am, bm, a, st, &mode);
}

// The map of an operand for boxes of 128 bytes x its tile's rows (or a stage's kk of them, MN-major).
bool operand_map(CUtensorMap* map, const Planes& o, bool bf16, int box_rows, int bk) {
  return encode_planes_map(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, o.p, o.planes,
                           o.rows, o.cols, o.pitch * 2, o.plane_stride * 2, o.mn_major ? bk : box_rows);
}

int stage_of(const TcPlan& plan, int planes) { return planes == 1 && !plan.cluster ? 128 : 64; }

// A product's arguments and its operands' maps.
template <typename T>
fxtx_status_t prepare_product(const PlanesProduct& p, const TcPlan& plan, TcArgs& a, CUtensorMap& am, CUtensorMap& bm,
                              int fold = FOLD) {
  constexpr int PL = std::is_same<T, float>::value ? 3 : 1;
  const bool bf16 = !std::is_same<T, __half>::value;
  if (log_enabled())
    fprintf(stderr, "[fxtx] product M=%lld N=%lld K=%lld planes=%d %s%s cg=%d bn=%d splits=%d\n", (long long)p.M,
            (long long)p.N, (long long)p.K, PL, plan.swap ? "swap " : "", plan.cluster ? "cluster" : "persistent", plan.cg,
            plan.bn, plan.splits);
  const Planes &A = plan.swap ? p.B : p.A, &B = plan.swap ? p.A : p.B;
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
  if (PL == 1 && (int64_t)a.per_split * bk > fold) a.fold = fold / bk;
  // a cluster's CTAs share the tile's 128 lanes out evenly, and each has work
  if (plan.cluster && (a.splits != plan.splits || 128 % a.splits != 0 || a.splits > 8)) return FXTX_ERR_UNSUPPORTED;
  a.a_mn = A.mn_major;
  a.b_mn = B.mn_major;
  a.idesc = mma_desc(bf16, A.mn_major, B.mn_major, 128 * plan.cg, plan.bn);
  a.e = p.e;
  memset(&am, 0, sizeof am);
  memset(&bm, 0, sizeof bm);
  if (!operand_map(&am, A, bf16, 128, bk) || !operand_map(&bm, B, bf16, plan.bn / plan.cg, bk)) return FXTX_ERR_CUDA;
  return FXTX_OK;
}

// The persistent kernel that the plan names.
template <typename T, int MODE>
cudaError_t launch_persistent(const TcPlan& plan, const CUtensorMap& am, const CUtensorMap& bm, const TcArgs& a,
                              const ModeArgs<MODE>& mode, int sm_count, cudaStream_t st) {
  constexpr int PL = std::is_same<T, float>::value ? 3 : 1;
  if (plan.cg == 2) {
    switch (plan.bn) {
      case 128: return launch<T, 2, 128, PL, MODE>(am, bm, a, mode, sm_count, st);
      case 256:
        if constexpr (PL == 1) return launch<T, 2, 256, PL, MODE>(am, bm, a, mode, sm_count, st);
        break;
    }
  } else {
    switch (plan.bn) {
      case 64: return launch<T, 1, 64, PL, MODE>(am, bm, a, mode, sm_count, st);
      case 128: return launch<T, 1, 128, PL, MODE>(am, bm, a, mode, sm_count, st);
    }
  }
  return cudaErrorInvalidConfiguration;
}

// A product of logits (modes 1 and 2), whose kk is not split. Both modes take the same sums, since the gradient's exponentials are
// divided by the sum that the loss had of them: with pieces of FOLD in mode 2 alone, logits of 8,192 positive terms around 400 gave
// probabilities 1.2 (bfloat16) and 2.1 % (float16) too small. The gradient of 8192 x 2048, 65,536 classes takes 0.5 % longer for it.
template <typename T, int MODE>
fxtx_status_t run_mode(const PlanesProduct& p, const ModeArgs<MODE>& mode, const DeviceInfo& dev, cudaStream_t st) {
  const TcPlan plan = plan_persistent(p.M, p.N, p.K, std::is_same<T, float>::value ? 3 : 1, p.A.mn_major, p.B.mn_major, dev.sm_count, 1);
  TcArgs a;
  CUtensorMap am, bm;
  const fxtx_status_t s = prepare_product<T>(p, plan, a, am, bm, LOGIT_FOLD);
  if (s != FXTX_OK) return s;
  if (launch_persistent<T, MODE>(plan, am, bm, a, mode, dev.sm_count, st) == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

}  // namespace
}  // namespace fxtx
