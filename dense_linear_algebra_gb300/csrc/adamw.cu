// adamw.cu — one AdamW step over a list of tensors in one launch, the moments held in 32
// bits or in 8.
//
//     m' = b1 m + (1 - b1) g            v' = b2 v + (1 - b2) g^2
//     p' = p (1 - lr wd) - lr / (1 - b1^t) * m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
//
// (Loshchilov and Hutter, "Decoupled weight decay regularization", algorithm 2.) Every value
// is computed in fp32, each operation rounded on its own (no fused multiply-add), so that the
// result is a function of the formulas above and of nothing in the compiler's choices: an
// 8-bit code next to a rounding boundary comes out the same for everyone who follows them.
//
// 8-bit states. A tensor is cut into blocks of 256 elements, the last one short; a block has
// one fp32 scale per moment. The first moment is held as c in -127 .. 127, m = s c |c|,
// s = max |m'| / 127^2; the second as its root r = sqrt(v) in c in 0 .. 255, r = s c^2,
// s = max r' / 255^2, both rounded to nearest in c. Square-law codes are finer at the top of
// a block's range (a step is 2/c of the value) and reach down to 1/65025 of the largest root;
// a linear code of the same width would stop at 1/255, and Adam divides by r. For the same
// reason a root that is not zero is never held as zero. A block whose largest value is below
// 1e-30 is held as zeros, and one that holds an infinity or a NaN reads back as NaN.
//
// Bound: HBM. Each of p, g and the states is read once and p and the states are written once.
// One warp takes one block of 256 elements, 8 neighbouring elements a lane, so that every
// array moves in 16-byte (32-bit and 16-bit types) or 8-byte (codes) accesses and the block's
// maxima are one warp reduction. With 8-bit states the instructions bound it first (a square
// root and a division an element as IEEE rounds them, and two approximate roots for the codes, taken
// again as IEEE has them where they lie near the middle of two): products and sums go two
// elements at a time, codes become numbers by one conversion and numbers codes by one addition. 100 M fp32 weights
// with bfloat16 gradients and copy: 414 us, 6.76 TB/s. 250 M bfloat16 weights with 8-bit states: 758 us
// (368 at the copy rate), their moments read back 381 us. The tensor table travels as a kernel parameter (constant
// bank): no copy and no workspace before the launch, at most 448 tensors a launch.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "layers.h"

namespace fxtx {
namespace {

constexpr int BLOCK = FXTX_ADAMW_BLOCK;  // elements a block, one warp
constexpr int PER = BLOCK / 32;          // elements a lane
constexpr int WARPS = 8;
static_assert(PER == 8, "a lane holds 8 elements");

template <int N>
struct Table {
  fxtx_adamw_tensor_t t[N];
  uint32_t first[N];  // blocks before tensor i
  uint32_t blocks;    // blocks in all
  int count;
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const T* e = reinterpret_cast<const T*>(&a);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(e[i]);
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float* x) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint4 a;
    T* e = reinterpret_cast<T*>(&a);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(x[i]);
    *reinterpret_cast<uint4*>(p) = a;
  }
}

template <typename T>
__device__ __forceinline__ void load_n(const T* p, int n, float* x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = i < n ? to_f32(p[i]) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store_n(T* p, int n, const float* x) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = from_f32<T>(x[i]);
}

// Two products or sums in one instruction, each rounded on its own (the sum as a fused a * one + x,
// with a 1 that the assembler does not know: it would merge a product with the sum that follows it, and round once).
__device__ __forceinline__ void mul2(float& a, float& b, float x, float y) {
  asm("{\n.reg .b64 u, v;\nmov.b64 u, {%0, %1};\nmov.b64 v, {%2, %3};\nmul.rn.f32x2 u, u, v;\nmov.b64 {%0, %1}, u;\n}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}
__device__ __forceinline__ void add2(float& a, float& b, float x, float y, float one) {
  asm("{\n.reg .b64 u, v, w;\nmov.b64 u, {%0, %1};\nmov.b64 v, {%2, %3};\nmov.b64 w, {%4, %4};\nfma.rn.f32x2 u, u, w, v;\n"
      "mov.b64 {%0, %1}, u;\n}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y), "f"(one));
}

// The largest |x| of a block, NaN if one is a NaN (magnitudes order as their bits do).
__device__ __forceinline__ float block_max(const float* x) {
  float top = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < PER; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(x[i])));
  return __uint_as_float(__reduce_max_sync(FULL_MASK, __float_as_uint(top) & 0x7fffffffu));
}

constexpr float kRound = 12582912.f;  // 1.5 * 2^23: a sum with it ends in the other term rounded to an integer

// x_i becomes the integer rint(sqrt(x_i)), root and rounding as IEEE has them, for x_i up to 255.4^2. The
// approximate root is off by less than 1e-4 and settles the code, unless it lies that close to the middle
// of two: then the lane's roots are taken again.
__device__ __forceinline__ void code_roots(float* x, float one) {
  float off = 0.f, s[PER];
#pragma unroll
  for (int i = 0; i < PER; i += 2) {
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(s[i]) : "f"(x[i]));
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(s[i + 1]) : "f"(x[i + 1]));
    float a = s[i], b = s[i + 1], u, v;
    add2(a, b, kRound, kRound, one);
    add2(a, b, -kRound, -kRound, one);
    u = a;
    v = b;
    add2(a, b, -s[i], -s[i + 1], one);
    off = fmaxf(off, fmaxf(fabsf(a), fabsf(b)));
    s[i] = u;
    s[i + 1] = v;
  }
  if (off > 0.4999f) {
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = __fsub_rn(__fadd_rn(__fsqrt_rn(x[i]), kRound), kRound);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) x[i] = s[i];
}

// The scale of a block and the factor that takes its values to squares of codes; `square` is
// the largest code squared and `part` its reciprocal, rounded.
__device__ __forceinline__ float block_scale(float top, float square, float part, float& inv) {
  const bool held = !(top < 1e-30f);
  inv = held ? __fmul_rn(__frcp_rn(top), square) : 0.f;
  return held ? __fmul_rn(top, part) : 0.f;
}

template <typename P, typename G, int BITS, int N>
__global__ void __launch_bounds__(WARPS * 32) adamw_kernel(const __grid_constant__ Table<N> tab, const AdamwConst c,
                                                           const int copy_type, const int per_warp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  after_previous();
  int ti = -1;
  uint32_t lo = 0, hi = 0;  // the blocks of tensor ti
  for (int it = 0; it < per_warp; ++it) {
    const uint32_t b = (blockIdx.x * (uint32_t)per_warp + (uint32_t)it) * WARPS + (uint32_t)warp;
    if (b >= tab.blocks) return;
    if (ti < 0 || b >= hi) {  // the last tensor whose first block is at or before b
      int l = ti < 0 ? 0 : ti, h = tab.count;
      while (h - l > 1) {
        const int mid = (l + h) >> 1;
        if (tab.first[mid] <= b) l = mid; else h = mid;
      }
      ti = l;
      lo = tab.first[ti];
      hi = ti + 1 < tab.count ? tab.first[ti + 1] : tab.blocks;
    }
    const fxtx_adamw_tensor_t& t = tab.t[ti];
    const int64_t blk = (int64_t)(b - lo), at = blk * BLOCK + lane * PER;
    const int64_t left = t.n - at;
    const int n = left >= PER ? PER : (left > 0 ? (int)left : 0);
    P* pp = static_cast<P*>(t.p) + at;
    const G* gp = static_cast<const G*>(t.g) + at;
    const uintptr_t bits = (uintptr_t)t.p | (uintptr_t)t.g | (uintptr_t)t.copy | (BITS == 32 ? (uintptr_t)t.m | (uintptr_t)t.v : 0);
    // codes move 8 bytes a lane
    const bool wide = n == PER && (bits & 15u) == 0 && (BITS == 32 || (((uintptr_t)t.m | (uintptr_t)t.v) & 7u) == 0);

    float p[PER], g[PER], m[PER], v[PER];
    if (wide) {
      load8(pp, p);
      load8(gp, g);
    } else {
      load_n(pp, n, p);
      load_n(gp, n, g);
    }
    if constexpr (BITS == 32) {
      const float *mp = static_cast<const float*>(t.m) + at, *vp = static_cast<const float*>(t.v) + at;
      if (wide) {
        load8(mp, m);
        load8(vp, v);
      } else {
        load_n(mp, n, m);
        load_n(vp, n, v);
      }
    } else {
      const int8_t* mp = static_cast<const int8_t*>(t.m) + at;
      const uint8_t* vp = static_cast<const uint8_t*>(t.v) + at;
      int8_t mc[PER];
      uint8_t vc[PER];
      if (wide) {
        *reinterpret_cast<uint2*>(mc) = *reinterpret_cast<const uint2*>(mp);
        *reinterpret_cast<uint2*>(vc) = *reinterpret_cast<const uint2*>(vp);
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          mc[i] = i < n ? mp[i] : (int8_t)0;
          vc[i] = i < n ? vp[i] : (uint8_t)0;
        }
      }
      const float ms = t.m_scale[blk], vs = t.v_scale[blk];
#pragma unroll
      for (int i = 0; i < PER; i += 2) {
        m[i] = (float)mc[i];
        m[i + 1] = (float)mc[i + 1];
        mul2(m[i], m[i + 1], fabsf(m[i]), fabsf(m[i + 1]));  // exact
        mul2(m[i], m[i + 1], ms, ms);
        v[i] = (float)vc[i];
        v[i + 1] = (float)vc[i + 1];
        mul2(v[i], v[i + 1], v[i], v[i + 1]);  // exact
        mul2(v[i], v[i + 1], vs, vs);
        mul2(v[i], v[i + 1], v[i], v[i + 1]);
      }
    }

    float r[PER];
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
      float x = g[i], y = g[i + 1];
      mul2(x, y, x, y);
      mul2(x, y, c.c2, c.c2);
      mul2(v[i], v[i + 1], c.b2, c.b2);
      add2(v[i], v[i + 1], x, y, c.one);
      mul2(g[i], g[i + 1], c.c1, c.c1);
      mul2(m[i], m[i + 1], c.b1, c.b1);
      add2(m[i], m[i + 1], g[i], g[i + 1], c.one);
      x = r[i] = __fsqrt_rn(v[i]);
      y = r[i + 1] = __fsqrt_rn(v[i + 1]);
      mul2(x, y, c.root, c.root);
      add2(x, y, c.eps, c.eps, c.one);
      x = __fdiv_rn(m[i], x);
      y = __fdiv_rn(m[i + 1], y);
      mul2(x, y, -c.rate, -c.rate);
      mul2(p[i], p[i + 1], c.keep, c.keep);
      add2(p[i], p[i + 1], x, y, c.one);
    }

    if (wide) store8(pp, p);
    else store_n(pp, n, p);
    if (t.copy != nullptr) {
      if (copy_type == FXTX_BF16) {
        __nv_bfloat16* q = static_cast<__nv_bfloat16*>(t.copy) + at;
        if (wide) store8(q, p);
        else store_n(q, n, p);
      } else if (copy_type == FXTX_F16) {
        __half* q = static_cast<__half*>(t.copy) + at;
        if (wide) store8(q, p);
        else store_n(q, n, p);
      } else {
        float* q = static_cast<float*>(t.copy) + at;
        if (wide) store8(q, p);
        else store_n(q, n, p);
      }
    }
    if constexpr (BITS == 32) {
      float *mp = static_cast<float*>(t.m) + at, *vp = static_cast<float*>(t.v) + at;
      if (wide) {
        store8(mp, m);
        store8(vp, v);
      } else {
        store_n(mp, n, m);
        store_n(vp, n, v);
      }
    } else {
      float mi, vi;
      const float ms = block_scale(block_max(m), 16129.f, 1.f / 16129.f, mi);
      const float vs = block_scale(block_max(r), 65025.f, 1.f / 65025.f, vi);
      int8_t mc[PER];
      uint8_t vc[PER];
      float x[PER];
#pragma unroll
      for (int i = 0; i < PER; i += 2) {
        x[i] = fabsf(m[i]);
        x[i + 1] = fabsf(m[i + 1]);
        mul2(x[i], x[i + 1], mi, mi);
      }
      code_roots(x, c.one);
#pragma unroll
      for (int i = 0; i < PER; ++i) mc[i] = (int8_t)(__float_as_int(copysignf(x[i], m[i]) + kRound));
#pragma unroll
      for (int i = 0; i < PER; i += 2) {
        x[i] = r[i];
        x[i + 1] = r[i + 1];
        mul2(x[i], x[i + 1], vi, vi);
      }
      code_roots(x, c.one);
#pragma unroll
      for (int i = 0; i < PER; ++i) vc[i] = (uint8_t)(__float_as_int((r[i] > 0.f ? fmaxf(x[i], 1.f) : x[i]) + kRound));
      // an infinity or a NaN in the block: nothing has a code, and all reads back as NaN by its scale (0 times an
      // infinity, or a NaN; an infinite scale with codes above 0 would hold every weight of the block still for good)
      if (!(ms <= 3.4e38f)) {
#pragma unroll
        for (int i = 0; i < PER; ++i) mc[i] = 0;
      }
      if (!(vs <= 3.4e38f)) {
#pragma unroll
        for (int i = 0; i < PER; ++i) vc[i] = 0;
      }
      int8_t* mp = static_cast<int8_t*>(t.m) + at;
      uint8_t* vp = static_cast<uint8_t*>(t.v) + at;
      if (wide) {
        *reinterpret_cast<uint2*>(mp) = *reinterpret_cast<const uint2*>(mc);
        *reinterpret_cast<uint2*>(vp) = *reinterpret_cast<const uint2*>(vc);
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i < n) {
            mp[i] = mc[i];
            vp[i] = vc[i];
          }
      }
      if (lane == 0) {
        t.m_scale[blk] = ms;
        t.v_scale[blk] = vs;
      }
    }
  }
}

template <typename P, typename G, int BITS, int N>
cudaError_t launch_n(int64_t count, const fxtx_adamw_tensor_t* t, int copy_type, const AdamwConst& c, int sm_count,
                     cudaStream_t st) {
  Table<N> tab;
  int64_t i = 0;
  while (i < count) {
    tab.count = 0;
    uint64_t blocks = 0;
    // as many tensors as the table and 2^31 blocks hold; tensors without elements take no place
    for (; i < count && tab.count < N; ++i) {
      if (t[i].n == 0) continue;
      const uint64_t nb = (uint64_t)(t[i].n + BLOCK - 1) / BLOCK;
      if (tab.count > 0 && blocks + nb > 0x7fffffffu) break;
      tab.t[tab.count] = t[i];
      tab.first[tab.count++] = (uint32_t)blocks;
      blocks += nb;
    }
    if (tab.count == 0) break;
    tab.blocks = (uint32_t)blocks;
    // up to 4 blocks a warp in turn, fewer while that leaves SMs without work
    const int64_t units = ((int64_t)blocks + WARPS - 1) / WARPS;
    const int per_warp = (int)std::min<int64_t>(4, std::max<int64_t>(1, units / ((int64_t)sm_count * 8)));
    const unsigned grid = (unsigned)((units + per_warp - 1) / per_warp);
    const cudaError_t e = launch_kernel(adamw_kernel<P, G, BITS, N>, dim3(grid), WARPS * 32, 0, st, tab, c, copy_type, per_warp);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename P, typename G, int BITS>
cudaError_t launch_bits(int64_t count, const fxtx_adamw_tensor_t* t, int copy_type, const AdamwConst& c, int sm_count,
                        cudaStream_t st) {
  // the short table keeps a small network's launch parameters at 3.3 KB
  return count <= 48 ? launch_n<P, G, BITS, 48>(count, t, copy_type, c, sm_count, st)
                     : launch_n<P, G, BITS, 448>(count, t, copy_type, c, sm_count, st);
}

template <typename P, typename G>
cudaError_t launch_types(int64_t count, const fxtx_adamw_tensor_t* t, int copy_type, int bits, const AdamwConst& c,
                         int sm_count, cudaStream_t st) {
  return bits == 32 ? launch_bits<P, G, 32>(count, t, copy_type, c, sm_count, st)
                    : launch_bits<P, G, 8>(count, t, copy_type, c, sm_count, st);
}

template <typename P>
cudaError_t launch_param(int64_t count, const fxtx_adamw_tensor_t* t, int g_type, int copy_type, int bits,
                         const AdamwConst& c, int sm_count, cudaStream_t st) {
  switch (g_type) {
    case FXTX_F32: return launch_types<P, float>(count, t, copy_type, bits, c, sm_count, st);
    case FXTX_BF16: return launch_types<P, __nv_bfloat16>(count, t, copy_type, bits, c, sm_count, st);
    default: return launch_types<P, __half>(count, t, copy_type, bits, c, sm_count, st);
  }
}

// The values that 8-bit states stand for: 4 elements a thread, so that a warp's stores are whole lines.
__global__ void __launch_bounds__(256) moments_kernel(int64_t n, const int8_t* m, const float* ms, const uint8_t* r,
                                                      const float* rs, float* m_out, float* v_out) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  after_previous();
  if (at >= n) return;
  const float a = ms[at / BLOCK], b = rs[at / BLOCK];
  const bool wide = at + 4 <= n && (((uintptr_t)m | (uintptr_t)r) & 3u) == 0 &&
                    (((uintptr_t)m_out | (uintptr_t)v_out) & 15u) == 0;
  int8_t mc[4];
  uint8_t rc[4];
  if (wide) {
    *reinterpret_cast<uint32_t*>(mc) = *reinterpret_cast<const uint32_t*>(m + at);
    *reinterpret_cast<uint32_t*>(rc) = *reinterpret_cast<const uint32_t*>(r + at);
  } else {
    for (int i = 0; i < 4; ++i) {
      mc[i] = at + i < n ? m[at + i] : (int8_t)0;
      rc[i] = at + i < n ? r[at + i] : (uint8_t)0;
    }
  }
  float x[4], y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float p = (float)mc[i], q = (float)rc[i];
    x[i] = __fmul_rn(p * fabsf(p), a);
    const float root = __fmul_rn(q * q, b);
    y[i] = __fmul_rn(root, root);
  }
  if (wide) {
    *reinterpret_cast<float4*>(m_out + at) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(v_out + at) = make_float4(y[0], y[1], y[2], y[3]);
  } else {
    for (int i = 0; i < 4 && at + i < n; ++i) {
      m_out[at + i] = x[i];
      v_out[at + i] = y[i];
    }
  }
}

}  // namespace

cudaError_t launch_adamw(int64_t count, const fxtx_adamw_tensor_t* t, int p_type, int g_type, int copy_type, int bits,
                         const AdamwConst& c, int sm_count, cudaStream_t st) {
  switch (p_type) {
    case FXTX_F32: return launch_param<float>(count, t, g_type, copy_type, bits, c, sm_count, st);
    case FXTX_BF16: return launch_param<__nv_bfloat16>(count, t, g_type, copy_type, bits, c, sm_count, st);
    default: return launch_param<__half>(count, t, g_type, copy_type, bits, c, sm_count, st);
  }
}

cudaError_t launch_adamw_moments(int64_t n, const int8_t* m, const float* ms, const uint8_t* r, const float* rs,
                                 float* m_out, float* v_out, cudaStream_t st) {
  if (n <= 0) return cudaSuccess;
  return launch_kernel(moments_kernel, dim3((unsigned)((n + 1023) / 1024)), 256, 0, st, n, m, ms, r, rs, m_out, v_out);
}

}  // namespace fxtx
