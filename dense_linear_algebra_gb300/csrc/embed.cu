// embed.cu — the embedding lookup and its gradient:
//     out_i = scale E[ids_i],   dE_v = scale * the sum of the rows of G with id v (zeros where there is none).
//
// Bound: HBM; the lookup reads each row once and writes it (65,536 of 131,072 x 4096 bfloat16 115 us, 6.1 TB/s), the gradient
// reads G and writes dE once (65,536 x 2048 into 131,072 rows 170 us, 4.7 TB/s: 136 the sums and the zeroed rows, the sort and
// the long runs the rest).
//
// The gradient sorts the ids, so that every row of dE is summed in registers, in the order of the positions, and
// written once, with no atomic addition: the result is the same on every call. The sort is a stable radix sort of
// (id, position), up to 9 bits a pass: each CTA counts its ids' digits, a second kernel turns the counts into places,
// a third scatters, a warp ranking its 32 ids at a time by votes on the digits' bits; up to 16,384 ids take one launch of one
// cluster, whose CTAs exchange their counts.
//
// The sorted positions are then cut into chunks of 32. A worker adds a chunk's rows of G run by run; a run that goes over
// into the next chunk and ends there is finished by the worker that began it. Of a longer one the chunks' parts are written
// out in fp32, and a second kernel adds each such run's, so that a frequent id's thousands of rows are shared out evenly.
// The rows of dE without an id are zeroed by further CTAs of the first of these launches, which look their rows up among
// the sorted ids.
#include <algorithm>

#include "common.cuh"
#include "host.h"
#include "kernels.h"
#include "tc.cuh"
#include "train.h"

namespace fxtx {

int* embed_error_word() { return device_error_word(); }

namespace {

constexpr int THREADS = 256;
constexpr int MAX_BITS = 9, RADIX = 1 << MAX_BITS;
constexpr int ITEMS = 4, TILE = THREADS * ITEMS;         // ids a thread and a CTA of the sort take
constexpr int CLUSTER_ITEMS = 2, CLUSTER_THREADS = 1024, CLUSTER = 8;  // the same of the sort in one cluster, and its CTAs at most
constexpr int CHUNK = 32;                                // sorted ids a worker adds

constexpr uint32_t NONE = 0xffffffffu;  // the key of no id

// V neighbouring entries (of 16 bytes, or one; of float: V of them) from p on.
template <typename S, int V>
struct Piece {
  static constexpr int B = V * sizeof(S);
  static_assert(B % 16 == 0, "16 bytes");
  uint4 v[B / 16];
  __device__ __forceinline__ void load(const S* p) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float get(int i) const { return to_f32(reinterpret_cast<const S*>(v)[i]); }
  __device__ __forceinline__ void set(int i, float x) { reinterpret_cast<S*>(v)[i] = from_f32<S>(x); }
  __device__ __forceinline__ void store(S* p) const {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
  }
};
template <typename S>
struct Piece<S, 1> {
  S v;
  __device__ __forceinline__ void load(const S* p) { v = *p; }
  __device__ __forceinline__ void zero() { v = from_f32<S>(0.f); }
  __device__ __forceinline__ float get(int) const { return to_f32(v); }
  __device__ __forceinline__ void set(int, float x) { v = from_f32<S>(x); }
  __device__ __forceinline__ void store(S* p) const { *p = v; }
};

// The id at position i, `count` for one outside the table.
__device__ __forceinline__ uint32_t id_at(const void* ids, bool wide, int64_t i, int64_t count) {
  const int64_t v = wide ? static_cast<const int64_t*>(ids)[i] : (int64_t)static_cast<const int32_t*>(ids)[i];
  return (uint32_t)(v < 0 || v >= count ? count : v);
}

// How the accesses of a row lie over threads: `tpr` threads a slab of the row, `groups` slabs a CTA in work.
struct Shape {
  int tpr = 1, groups = 1;
  int64_t slabs = 1;
};

template <typename T, int V>
__global__ void __launch_bounds__(THREADS) embed_kernel(const __grid_constant__ EmbedArgs a, const Shape s) {
  constexpr int U = 4;
  const int group = threadIdx.x / s.tpr, t = threadIdx.x % s.tpr;
  const int64_t accesses = a.n / V, units = a.m * s.slabs;
  after_previous();
  for (int64_t w = (int64_t)blockIdx.x * s.groups + group; w < units; w += (int64_t)gridDim.x * s.groups) {
    const int64_t i = w / s.slabs, first = (w - i * s.slabs) * s.tpr * U + t;
    const uint32_t id = id_at(a.ids, a.ids64, i, a.count);
    const bool in = id < a.count;
    const T* p = static_cast<const T*>(a.src) + (int64_t)(in ? id : 0) * a.lds;
    T* o = static_cast<T*>(a.out) + i * a.ldo;
    Piece<T, V> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = first + u * s.tpr;
      if (in && c < accesses) x[u].load(p + c * V);
      else x[u].zero();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = first + u * s.tpr;
      if (c >= accesses) break;
#pragma unroll
      for (int q = 0; q < V; ++q)
        if (in) x[u].set(q, x[u].get(q) * a.scale);
      x[u].store(o + c * V);
    }
  }
}

// ------------------------------------------------------------------------------------------------ the sort
struct SortArgs {
  const void* ids;
  bool ids64;
  int64_t m, count;
  const uint2* from;  // (id, position); NULL: the ids themselves
  uint2* to;
  uint32_t *counts, *totals;  // [digit][CTA], [digit]
  uint32_t* clear;            // a word to be zeroed on the way
  int64_t ctas;
  int shift, bits;
};

__device__ __forceinline__ uint2 item(const SortArgs& a, int64_t i) {
  if (i >= a.m) return make_uint2(NONE, 0);
  return a.from ? a.from[i] : make_uint2(id_at(a.ids, a.ids64, i, a.count), (uint32_t)i);
}
__device__ __forceinline__ uint32_t digit_of(uint32_t key, int shift, int bits) { return (key >> shift) & ((1u << bits) - 1u); }

// The warp's items (32 at a time, in order) ranked among its own of the same digit; `hist` counts them.
template <int ITEMS>
__device__ __forceinline__ void rank_items(const uint2* x, int items, uint32_t* hist, int shift, int bits, uint32_t* rank) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    if (i >= items) break;
    const bool in = x[i].x != NONE;
    const uint32_t d = in ? digit_of(x[i].x, shift, bits) : 0;
    // the lanes with the same digit, by a vote a bit (match.any takes about 150 cycles where the digits differ)
    uint32_t same = __ballot_sync(FULL_MASK, in);
#pragma unroll
    for (int q = 0; q < MAX_BITS; ++q) {
      const uint32_t set = __ballot_sync(FULL_MASK, d >> q & 1u);
      same &= d >> q & 1u ? set : ~set;
    }
    const uint32_t before = __popc(same & ((1u << lane) - 1u)), had = hist[d];
    __syncwarp();
    if (in && before == 0) hist[d] = had + __popc(same);
    __syncwarp();
    rank[i] = had + before;
  }
}

// An exclusive scan of v[0 .. n - 1] in shared memory by the whole CTA (n at most 2 RADIX); `warps` holds 32 words.
__device__ __forceinline__ void scan(uint32_t* v, int n, uint32_t* warps) {
  const int tid = threadIdx.x, lane = tid & 31, per = (n + (int)blockDim.x - 1) / (int)blockDim.x;
  uint32_t own = 0;
  for (int i = 0; i < per; ++i)
    if (tid * per + i < n) own += v[tid * per + i];
  uint32_t upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(FULL_MASK, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) warps[tid >> 5] = upto;
  __syncthreads();
  uint32_t at = upto - own;
  for (int w = 0; w < tid >> 5; ++w) at += warps[w];
  for (int i = 0; i < per; ++i)
    if (tid * per + i < n) {
      const uint32_t y = v[tid * per + i];
      v[tid * per + i] = at;
      at += y;
    }
  __syncthreads();
}

__global__ void __launch_bounds__(THREADS) sort_count_kernel(const __grid_constant__ SortArgs a) {
  __shared__ uint32_t hist[RADIX];
  for (int d = threadIdx.x; d < 1 << a.bits; d += THREADS) hist[d] = 0;
  __syncthreads();
  after_previous();
  const int64_t base = (int64_t)blockIdx.x * TILE;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint2 x = item(a, base + i * THREADS + threadIdx.x);
    if (x.x != NONE) atomicAdd(&hist[digit_of(x.x, a.shift, a.bits)], 1u);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < 1 << a.bits; d += THREADS) a.counts[d * a.ctas + blockIdx.x] = hist[d];
}

// counts: over the CTAs before, a warp a digit; totals: over all of them.
__global__ void __launch_bounds__(THREADS) sort_places_kernel(const __grid_constant__ SortArgs a) {
  const int lane = threadIdx.x & 31, d = (int)(blockIdx.x * (THREADS / 32)) + (int)(threadIdx.x >> 5);
  after_previous();
  if (d >= 1 << a.bits) return;
  uint32_t* c = a.counts + d * a.ctas;
  uint32_t sum = 0;
  for (int64_t i = 0; i < a.ctas; i += 32) {
    const uint32_t own = i + lane < a.ctas ? c[i + lane] : 0;
    uint32_t upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(FULL_MASK, upto, o);
      if (lane >= o) upto += y;
    }
    if (i + lane < a.ctas) c[i + lane] = sum + upto - own;
    sum += __shfl_sync(FULL_MASK, upto, 31);
  }
  if (lane == 0) a.totals[d] = sum;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.clear = 0;
}

__global__ void __launch_bounds__(THREADS) sort_scatter_kernel(const __grid_constant__ SortArgs a) {
  constexpr int WARPS = THREADS / 32;
  __shared__ uint32_t hist[WARPS][RADIX], first[RADIX], warps[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, digits = 1 << a.bits;
  for (int d = tid; d < WARPS * RADIX; d += THREADS) (&hist[0][0])[d] = 0;
  after_previous();
  for (int d = tid; d < digits; d += THREADS) first[d] = a.totals[d];
  uint2 x[ITEMS];
  uint32_t rank[ITEMS];
  const int64_t base = (int64_t)blockIdx.x * TILE + warp * 32 * ITEMS + lane;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) x[i] = item(a, base + 32 * i);
  __syncthreads();
  rank_items<ITEMS>(x, ITEMS, hist[warp], a.shift, a.bits, rank);
  scan(first, digits, warps);
  // where each warp's ids of a digit begin
  for (int d = tid; d < digits; d += THREADS) {
    uint32_t at = first[d] + a.counts[d * a.ctas + blockIdx.x], y[WARPS];
#pragma unroll
    for (int w = 0; w < WARPS; ++w) y[w] = hist[w][d];
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      hist[w][d] = at;
      at += y[w];
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
    if (x[i].x != NONE) a.to[hist[warp][digit_of(x[i].x, a.shift, a.bits)] + rank[i]] = x[i];
}

// All passes in one cluster: each CTA takes `items` ids a thread, the CTAs' counts are exchanged through distributed shared
// memory, and the cluster's barriers make the ids that one CTA has written seen by the others in the next pass.
struct ClusterSort {
  SortArgs s;
  uint2* other;  // takes turns with s.to, which the last pass ends in
  int passes, items;
};

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(CLUSTER_THREADS) sort_cluster_kernel(const __grid_constant__ ClusterSort c) {
  constexpr int WARPS = CLUSTER_THREADS / 32;
  extern __shared__ __align__(16) uint32_t shared[];
  __shared__ uint32_t total[RADIX], first[RADIX], before[RADIX], warps[32];
  const SortArgs& a = c.s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, digits = 1 << a.bits;
  const int ctas = (int)gridDim.x, rank_here = (int)blockIdx.x;  // (one cluster)
  uint32_t* hist = shared;  // [WARPS][digits]
  const int64_t base = (int64_t)rank_here * CLUSTER_THREADS * c.items + warp * 32 * c.items + lane;
  uint2 x[CLUSTER_ITEMS];
  uint32_t rank[CLUSTER_ITEMS];
  after_previous();
  if (rank_here == 0 && tid == 0) *a.clear = 0;
  const uint2* from = nullptr;
  uint2* to = c.passes % 2 ? a.to : c.other;
  for (int p = 0; p < c.passes; ++p) {
    const int shift = p * a.bits;
#pragma unroll
    for (int i = 0; i < CLUSTER_ITEMS; ++i) {
      if (i >= c.items) break;
      const int64_t at = base + 32 * i;
      x[i] = at >= a.m ? make_uint2(NONE, 0) : from ? from[at] : item(a, at);
    }
    for (int d = tid; d < WARPS * digits; d += CLUSTER_THREADS) hist[d] = 0;
    __syncthreads();
    rank_items<CLUSTER_ITEMS>(x, c.items, hist + warp * digits, shift, a.bits, rank);
    __syncthreads();
    // over the warps before, and over all of them
    for (int d = tid; d < digits; d += CLUSTER_THREADS) {
      uint32_t at = 0;
#pragma unroll 1
      for (int w = 0; w < WARPS; w += 8) {
        uint32_t y[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) y[q] = hist[(w + q) * digits + d];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          hist[(w + q) * digits + d] = at;
          at += y[q];
        }
      }
      total[d] = at;
    }
    // over the CTAs before, and over all of them
    cluster_sync();
    for (int d = tid; d < digits; d += CLUSTER_THREADS) {
      uint32_t mine = 0, all = 0;
#pragma unroll 4
      for (int r = 0; r < ctas; ++r) {
        const uint32_t v = ld_cluster(cluster_addr(total + d, (uint32_t)r));
        all += v;
        mine += r < rank_here ? v : 0;
      }
      first[d] = all;
      before[d] = mine;
    }
    __syncthreads();
    scan(first, digits, warps);
#pragma unroll
    for (int i = 0; i < CLUSTER_ITEMS; ++i) {
      if (i >= c.items) break;
      if (x[i].x == NONE) continue;
      const uint32_t d = digit_of(x[i].x, shift, a.bits);
      to[first[d] + before[d] + hist[warp * digits + d] + rank[i]] = x[i];
    }
    // (the other CTAs have read this one's totals, and this pass's ids are seen by all)
    cluster_sync();
    from = to;
    to = to == a.to ? c.other : a.to;
  }
}

// ------------------------------------------------------------------------------------------------ the sums
struct ReduceArgs {
  int64_t m, n, count;
  const uint2* sorted;  // (id, row of G)
  const void* G;
  int64_t ldg;
  float scale;
  void* out;
  int64_t ldo;
  float* part;          // [2 a chunk][n]: what a chunk has of a long run that began before it, and of one that it begins
  uint32_t* longs;      // how many long runs there are, and the chunks that they begin in
  Shape shape;
  int64_t sum_ctas, ctas;  // CTAs of sums, spread among all; the others zero `zero_rows` rows each
  int zero_rows;
};

// How many of 0 .. n - 1 the predicate holds for, where it holds for the first ones and no others: a warp tries 32 at a time.
template <typename F>
__device__ __forceinline__ int64_t warp_bound(int64_t n, F holds) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0;
  while (n > 0) {
    const int64_t step = (n + 31) / 32, i = min(lo + n, lo + (lane + 1) * step) - 1;
    const int yes = __popc(__ballot_sync(FULL_MASK, holds(i)));
    if (yes == 32) return lo + n;
    lo += yes * step;
    n = min(n - yes * step, step) - 1;  // (the first that fails is known)
  }
  return lo;
}

// `bytes` from p on to zero, by the whole CTA: 16 at a time between the first and the last multiple of that. p and bytes are
// multiples of 2.
__device__ __forceinline__ void zero_bytes(void* p, int64_t bytes) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const int64_t head = min(bytes, (int64_t)(-at & 15u)), words = (bytes - head) / 16, tail = bytes - head - words * 16;
  char* base = static_cast<char*>(p);
  for (int64_t i = threadIdx.x; i < words; i += blockDim.x) reinterpret_cast<uint4*>(base + head)[i] = make_uint4(0, 0, 0, 0);
  const int i = (int)threadIdx.x;
  if (2 * i < head) *reinterpret_cast<uint16_t*>(base + 2 * i) = 0;
  if (2 * i < tail) *reinterpret_cast<uint16_t*>(base + head + words * 16 + 2 * i) = 0;
}

// Rows of dE without an id.
template <typename T>
__device__ __forceinline__ void zero_rows(const ReduceArgs& a, int64_t row0) {
  __shared__ uint32_t s_absent;
  if (threadIdx.x < 32) {
    const int64_t v = row0 + threadIdx.x;
    const bool mine = (int)threadIdx.x < a.zero_rows && v < a.count;
    // the first entry not below these rows; those from there on show which rows are there
    int64_t lo = warp_bound(a.m, [&](int64_t i) { return a.sorted[i].x < (uint32_t)row0; });
    uint32_t there = 0;
    bool all = false;
    for (int i = 0; i < 4 && !all; ++i) {
      const int64_t e = lo + 32 * i + threadIdx.x;
      const uint32_t at = (e < a.m ? a.sorted[e].x : NONE) - (uint32_t)row0;
      const bool in = at < (uint32_t)a.zero_rows;
      there |= __reduce_or_sync(FULL_MASK, in ? 1u << at : 0u);
      all = !__all_sync(FULL_MASK, in);
    }
    if (!all) {  // many entries to a row: a search a row
      int64_t hi = mine ? a.m : lo;
      while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (a.sorted[mid].x < (uint32_t)v) lo = mid + 1;
        else hi = mid;
      }
      there = __ballot_sync(FULL_MASK, mine && lo < a.m && a.sorted[lo].x == (uint32_t)v);
    }
    const uint32_t absent = __ballot_sync(FULL_MASK, mine) & ~there;
    if (threadIdx.x == 0) s_absent = absent;
  }
  __syncthreads();
  // neighbouring rows without a gap between them as one range
  const int64_t bytes = a.n * (int64_t)sizeof(T);
  for (uint32_t left = s_absent; left;) {
    const int first = __ffs(left) - 1, rows = a.ldo == a.n ? __ffs(~(left >> first)) - 1 : 1;  // (32 rows: ~ has no bit, 0 - 1)
    const int some = rows < 0 ? 32 : rows;
    zero_bytes(static_cast<T*>(a.out) + (row0 + first) * a.ldo, some * bytes);
    left = first + some < 32 ? left >> (first + some) << (first + some) : 0;
  }
}

// A chunk of 32 sorted ids and the runs that go over its ends. A run that begins in one chunk and ends in the next is the
// first one's as a whole; a longer one is cut at the chunks' ends, and its parts are added by the second kernel.
struct Chunk {
  int n;                    // its ids
  uint32_t left, right;     // the runs at the chunk's ends, NONE where none goes over them
  bool skip, part_left;     // the left one is the chunk before's; is long
  bool more, part_right;    // the right one goes on in the next chunk and ends there; is long
  bool begins_long;         // the right one is long and begins here
  // `k`: the sorted ids from the chunk's first on, those of BEFORE entries before it and of the next chunk among them
  __device__ __forceinline__ Chunk(const ReduceArgs& a, int64_t chunk, const uint2* k) {
    n = (int)min((int64_t)CHUNK, a.m - chunk * CHUNK);
    const uint32_t m33 = k[-CHUNK - 1].x, m32 = k[-CHUNK].x, m1 = k[-1].x, k0 = k[0].x, last = k[n - 1].x, next = k[n].x,
                   n31 = k[2 * CHUNK - 1].x, n32 = k[2 * CHUNK].x;
    left = m1 == k0 ? k0 : NONE;
    skip = left != NONE && !(m32 == left && m33 == left) && !(last == left && next == left);
    part_left = left != NONE && !skip;
    right = next == last ? last : NONE;
    const bool begins = !(k0 == right && m1 == right), ends = !(n31 == right && n32 == right);
    more = right != NONE && begins && ends;
    part_right = right != NONE && !more;
    begins_long = right != NONE && begins && !ends && right < a.count;
  }
};
constexpr int BEFORE = CHUNK + 1;

// The sorted ids of `chunks` chunks from one on, with those before and after them, to shared memory (NONE beyond the ends), by
// the whole CTA. Gives the place of the first chunk's.
__device__ __forceinline__ const uint2* load_ids(const ReduceArgs& a, int64_t chunk, int chunks, uint2* s) {
  const int64_t first = chunk * CHUNK - BEFORE;
  const int n = BEFORE + chunks * CHUNK + CHUNK + 1;
  for (int i = threadIdx.x; i < n; i += blockDim.x) s[i] = first + i >= 0 && first + i < a.m ? a.sorted[first + i] : make_uint2(NONE, 0);
  __syncthreads();
  return s + BEFORE;
}

// CH accesses of a row of dE, `step` apart: a chunk's sums, run by run.
template <typename T, int V, int CH>
struct RunSum {
  const ReduceArgs& a;
  const Chunk& k;
  const int64_t chunk, c, accesses;
  const int step;
  float acc[CH * V] = {};
  uint32_t run = NONE;
  __device__ __forceinline__ RunSum(const ReduceArgs& a_, const Chunk& k_, int64_t chunk_, int64_t c_, int step_)
      : a(a_), k(k_), chunk(chunk_), c(c_), accesses(a_.n / V), step(step_) {}
  __device__ __forceinline__ bool has(int h) const { return c + h * step < accesses; }
  __device__ __forceinline__ int64_t at(int h) const { return (c + h * step) * V; }
  __device__ __forceinline__ void add(uint32_t key, const Piece<T, V> (&x)[CH]) {
    if (key != run) {
      flush(false);
      run = key;
    }
#pragma unroll
    for (int h = 0; h < CH; ++h)
#pragma unroll
      for (int q = 0; q < V; ++q) acc[h * V + q] += x[h].get(q);
  }
  __device__ __forceinline__ void flush(bool part_right) {
    if (run < a.count) {
      const bool part_left = k.part_left && run == k.left;
#pragma unroll
      for (int h = 0; h < CH; ++h) {
        if (!has(h)) continue;
        if (!part_left && !part_right) {
          Piece<T, V> o;
#pragma unroll
          for (int q = 0; q < V; ++q) o.set(q, acc[h * V + q] * a.scale);
          o.store(static_cast<T*>(a.out) + (int64_t)run * a.ldo + at(h));
        } else {
          Piece<float, V> o;
#pragma unroll
          for (int q = 0; q < V; ++q) o.set(q, acc[h * V + q]);
          o.store(a.part + (2 * chunk + (part_left ? 0 : 1)) * a.n + at(h));
        }
      }
    }
#pragma unroll
    for (int q = 0; q < CH * V; ++q) acc[q] = 0.f;
  }
  // the rows of the first `n` of N ids, those other than `only` left out unless it is NONE
  template <int N>
  __device__ __forceinline__ void add_rows(const uint2* ids, int n, uint32_t only) {
    Piece<T, V> x[N][CH];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint2 y = ids[i < n ? i : 0];
      // (an id outside the table is `count`, sorted last; NONE is above it)
      const bool take = i < n && y.x < a.count && (only == NONE || y.x == only);
      const T* row = static_cast<const T*>(a.G) + (int64_t)y.y * a.ldg;
#pragma unroll
      for (int h = 0; h < CH; ++h) {
        if (take && has(h)) x[i][h].load(row + at(h));
        else x[i][h].zero();
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i >= n) break;
      const uint32_t key = ids[i].x;
      if (only == NONE || key == only) add(key, x[i]);
    }
  }
  // after the chunk's own entries: the rest of a run that ends in the next chunk
  template <int N>
  __device__ __forceinline__ void finish(const uint2* ids) {
    if (run == NONE) return;
    if (k.more)
#pragma unroll 1
      for (int i = CHUNK; i < 2 * CHUNK && ids[i].x == k.right; i += N) add_rows<N>(ids + i, 2 * CHUNK - i, k.right);
    flush(k.part_right);
  }
};

// Whether the CTA sums (its place among those that do), else its place among those that zero rows: they lie among one
// another, so that reading and writing go on together.
__device__ __forceinline__ bool sums_here(const ReduceArgs& a, int64_t& at) {
  const int64_t b = blockIdx.x, before = b * a.sum_ctas / a.ctas;
  const bool is = (b + 1) * a.sum_ctas / a.ctas != before;
  at = is ? before : b - before;
  return is;
}

__device__ __forceinline__ void note_long(const ReduceArgs& a, const Chunk& k, int64_t chunk) {
  if (k.begins_long) a.longs[1 + atomicAdd(a.longs, 1u)] = (uint32_t)chunk;  // (their order has no say in the result)
}

// Rows of at least 1 KB: a chunk's rows (1 KB of each) come by bulk copies to shared memory, all 32 on their way at once, a
// lane each.
constexpr int BULK_THREADS = 64, BULK_ROW = BULK_THREADS * 16;

template <typename T>
__global__ void __launch_bounds__(BULK_THREADS) embed_bulk_kernel(const __grid_constant__ ReduceArgs a) {
  constexpr int V = 16 / sizeof(T), PER = 8, BARS = CHUNK / PER;  // rows a barrier
  extern __shared__ __align__(128) unsigned char stage[];
  __shared__ __align__(8) uint64_t full[BARS];
  __shared__ uint2 s_ids[BEFORE + 2 * CHUNK + 1];
  if (threadIdx.x == 0) {
    for (int i = 0; i < BARS; ++i) mbar_init(&full[i], PER);
    fence_mbar_init();
  }
  __syncthreads();
  after_previous();
  int64_t at;
  if (!sums_here(a, at)) {
    zero_rows<T>(a, at * a.zero_rows);
    return;
  }
  const int64_t chunk = at / a.shape.slabs, slab = at % a.shape.slabs, accesses = a.n / V;
  const int64_t c0 = slab * BULK_THREADS, c = c0 + threadIdx.x;
  const uint32_t bytes = (uint32_t)min((int64_t)BULK_ROW, (accesses - c0) * 16);
  const uint2* ids = load_ids(a, chunk, 1, s_ids);
  const Chunk k(a, chunk, ids);
  // an id of the chunk's own, NONE where it is the chunk before's
  auto own = [&](int i) { return i >= k.n || (k.skip && ids[i].x == k.left) ? NONE : ids[i].x; };
  if (threadIdx.x < CHUNK) {
    const int lane = threadIdx.x;
    const bool copy = own(lane) < a.count;
    mbar_arrive_expect_tx(&full[lane / PER], copy ? bytes : 0);
    if (copy)
      bulk_g2s(stage + lane * BULK_ROW, static_cast<const T*>(a.G) + (int64_t)ids[lane].y * a.ldg + c0 * V, bytes, &full[lane / PER],
               policy_evict_first());
    if (lane == 0 && slab == 0) note_long(a, k, chunk);
  }
  RunSum<T, V, 1> sum(a, k, chunk, c, 0);
  bool ok = true;
#pragma unroll 1
  for (int i = 0; i < CHUNK; ++i) {
    if (i % PER == 0) ok = mbar_wait_bounded(&full[i / PER], 0) && ok;
    const uint32_t key = own(i);
    if (key == NONE || !ok) continue;
    Piece<T, V> x[1];
    if (key < a.count) x[0].load(reinterpret_cast<const T*>(stage + i * BULK_ROW + threadIdx.x * 16));
    else x[0].zero();
    sum.add(key, x);
  }
  if (ok) sum.template finish<4>(ids);
}

// Other rows: a worker is `tpr` threads, which hold several rows' accesses on their way. Many rows that go entry by entry (no 16-byte
// accesses) have 4 entries a thread, `tpr` apart.
constexpr int GROUPS = 16;  // workers a CTA has at most

// EACH: accesses a thread has.
template <typename T, int V, int EACH>
__global__ void __launch_bounds__(THREADS, V == 1 ? 4 : 2) embed_reduce_kernel(const __grid_constant__ ReduceArgs a) {
  __shared__ uint2 s_ids[BEFORE + (GROUPS + 1) * CHUNK + 1];
  after_previous();
  int64_t at;
  if (!sums_here(a, at)) {
    zero_rows<T>(a, at * a.zero_rows);
    return;
  }
  constexpr int N = V == 1 && EACH == 1 ? 16 : 8;
  const Shape& s = a.shape;
  const int group = threadIdx.x / s.tpr, t = threadIdx.x % s.tpr;
  const int64_t w = at * s.groups + group, chunk = w / s.slabs, c = (w - chunk * s.slabs) * s.tpr * EACH + t, first = at * s.groups / s.slabs;
  const uint2* ids = load_ids(a, first, s.groups, s_ids);
  if (group >= s.groups || chunk * CHUNK >= a.m) return;
  ids += (chunk - first) * CHUNK;
  const Chunk k(a, chunk, ids);
  if (c == 0) note_long(a, k, chunk);
  RunSum<T, V, EACH> sum(a, k, chunk, c, s.tpr);
  int i = 0;
  if (k.skip)
    while (ids[i].x == k.left) ++i;
#pragma unroll 1
  for (; i < k.n; i += N) sum.template add_rows<N>(ids + i, k.n - i, NONE);
  sum.template finish<N>(ids);
}

// The rows of dE of long runs, from the chunks' parts: TX accesses of a row a CTA, JOIN / TX threads an access, whose sums are
// added in order.
constexpr int JOIN = 256;

template <typename T, int V>
__global__ void __launch_bounds__(JOIN) embed_join_kernel(const __grid_constant__ ReduceArgs a, int tx, int64_t slabs) {
  __shared__ float sums[JOIN * V];
  after_previous();
  const int64_t chunks = (a.m + CHUNK - 1) / CHUNK, units = (int64_t)a.longs[0] * slabs;
  const int x = threadIdx.x % tx, y = threadIdx.x / tx, ty = JOIN / tx;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t chunk = a.longs[1 + u / slabs], e1 = (chunk + 1) * CHUNK, c = u % slabs * tx + x;
    const uint32_t run = a.sorted[e1].x;
    // the chunks that end in the run, and the next where it begins with it
    const int64_t after = chunks - chunk - 1;
    int64_t parts = warp_bound(after, [&](int64_t i) { return a.sorted[min(a.m, e1 + (i + 1) * CHUNK) - 1].x == run; });
    if (parts < after && a.sorted[e1 + parts * CHUNK].x == run) ++parts;
    ++parts;
    const bool mine = c < a.n / V;
    float acc[V] = {};
    constexpr int U = 4;
    for (int64_t p = y; p < parts; p += U * ty) {
      Piece<float, V> v[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t q = p + i * ty;
        if (mine && q < parts) v[i].load(a.part + (2 * (chunk + q) + (q == 0 ? 1 : 0)) * a.n + c * V);
        else v[i].zero();
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int q = 0; q < V; ++q) acc[q] += v[i].get(q);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < V; ++q) sums[q * JOIN + threadIdx.x] = acc[q];
    __syncthreads();
    if (y != 0 || !mine) continue;
    Piece<T, V> o;
#pragma unroll
    for (int q = 0; q < V; ++q) {
      float s = acc[q];
      for (int i = 1; i < ty; ++i) s += sums[q * JOIN + i * tx + x];
      o.set(q, s * a.scale);
    }
    o.store(static_cast<T*>(a.out) + (int64_t)run * a.ldo + c * V);
  }
}

// ------------------------------------------------------------------------------------------------ on the host
bool aligned(const void* p, int64_t ld, int size) { return ((uintptr_t)p & 15u) == 0 && ld * size % 16 == 0; }

// `per` accesses a thread.
Shape shape_of(int64_t accesses, int per) {
  Shape s;
  s.slabs = (accesses + (int64_t)THREADS * per - 1) / ((int64_t)THREADS * per);
  const int64_t need = (accesses + s.slabs * per - 1) / (s.slabs * per);
  if (need <= 32)
    while (s.tpr < need) s.tpr *= 2;
  else
    s.tpr = (int)((need + 31) / 32 * 32);
  s.groups = std::max(1, THREADS / s.tpr);
  return s;
}

template <typename T, int V>
cudaError_t lookup(const EmbedArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  const Shape s = shape_of(a.n / V, 4);
  const int64_t ctas = std::min<int64_t>((a.m * s.slabs + s.groups - 1) / s.groups, (int64_t)dev.sm_count * 64);
  return launch_kernel(embed_kernel<T, V>, dim3((unsigned)ctas), (unsigned)(s.tpr * s.groups), 0, st, a, s);
}

// The ids sorted into `to`, by way of `other`.
cudaError_t sort_ids(const EmbedArgs& a, uint2* to, uint2* other, uint32_t* counts, uint32_t* clear, int64_t ctas, cudaStream_t st) {
  SortArgs s = {};
  s.ids = a.ids;
  s.ids64 = a.ids64;
  s.m = a.m;
  s.count = a.count;
  s.counts = counts;
  s.clear = clear;
  s.totals = counts + RADIX * ctas;
  s.ctas = ctas;
  int bits = 1;
  while ((a.count >> bits) != 0) ++bits;  // of 0 .. count
  const int passes = (bits + MAX_BITS - 1) / MAX_BITS;
  s.bits = (bits + passes - 1) / passes;
  if (a.m <= (int64_t)CLUSTER * CLUSTER_THREADS * CLUSTER_ITEMS) {
    ClusterSort c;
    c.s = s;
    c.s.to = to;
    c.other = other;
    c.passes = passes;
    int ctas = 1;
    while (ctas < CLUSTER && a.m > (int64_t)ctas * CLUSTER_THREADS) ctas *= 2;
    c.items = (int)((a.m + (int64_t)ctas * CLUSTER_THREADS - 1) / (ctas * CLUSTER_THREADS));
    const size_t smem = (size_t)CLUSTER_THREADS / 32 * ((size_t)1 << s.bits) * 4;
    const cudaError_t e = ensure_smem((const void*)sort_cluster_kernel, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(CLUSTER_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // (see after_previous)
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sort_cluster_kernel, c);
  }
  // the last pass ends in `to`
  uint2* next = passes % 2 ? to : other;
  for (int p = 0; p < passes; ++p) {
    s.shift = p * s.bits;
    s.to = next;
    cudaError_t e = launch_kernel(sort_count_kernel, dim3((unsigned)ctas), THREADS, 0, st, s);
    if (e == cudaSuccess)
      e = launch_kernel(sort_places_kernel, dim3((unsigned)(((1 << s.bits) + THREADS / 32 - 1) / (THREADS / 32))), THREADS, 0, st, s);
    if (e == cudaSuccess) e = launch_kernel(sort_scatter_kernel, dim3((unsigned)ctas), THREADS, 0, st, s);
    if (e != cudaSuccess) return e;
    s.from = next;
    next = next == to ? other : to;
  }
  return cudaSuccess;
}

template <typename T, int V>
fxtx_status_t gradient(const EmbedArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  const int64_t tiles = (a.m + TILE - 1) / TILE, chunks = (a.m + CHUNK - 1) / CHUNK, accesses = a.n / V;
  const bool longs = chunks > 2;  // there may be runs over three chunks
  auto up = [](int64_t bytes) { return (size_t)((bytes + 255) / 256 * 256); };
  const size_t sort_bytes = up(a.m * 8), count_bytes = up((RADIX * tiles + RADIX) * 4), long_bytes = up((chunks + 1) * 4);
  const size_t part_bytes = longs ? up(2 * chunks * a.n * 4) : 0;
  char* ws = nullptr;
  const fxtx_status_t r = alloc_pooled(reinterpret_cast<void**>(&ws), 2 * sort_bytes + count_bytes + long_bytes + part_bytes, st);
  if (r != FXTX_OK) return r;
  ReduceArgs q = {};
  uint2* sorted = reinterpret_cast<uint2*>(ws);
  q.sorted = sorted;
  q.longs = reinterpret_cast<uint32_t*>(ws + 2 * sort_bytes + count_bytes);
  q.part = reinterpret_cast<float*>(ws + 2 * sort_bytes + count_bytes + long_bytes);
  cudaError_t e = cudaSuccess;
  if (a.m > 0)
    e = sort_ids(a, sorted, reinterpret_cast<uint2*>(ws + sort_bytes), reinterpret_cast<uint32_t*>(ws + 2 * sort_bytes), q.longs, tiles, st);
  q.m = a.m;
  q.n = a.n;
  q.count = a.count;
  q.G = a.src;
  q.ldg = a.lds;
  q.scale = a.scale;
  q.out = a.out;
  q.ldo = a.ldo;
  // CTAs that zero rows: 32 rows each, fewer where the table is small
  q.zero_rows = (int)std::max<int64_t>(1, std::min<int64_t>(32, a.count / (8 * (int64_t)dev.sm_count)));
  const int64_t zero_ctas = (a.count + q.zero_rows - 1) / q.zero_rows;
  if (V > 1 && accesses >= BULK_THREADS) {
    if constexpr (V > 1) {
      q.shape.slabs = (accesses + BULK_THREADS - 1) / BULK_THREADS;
      q.sum_ctas = chunks * q.shape.slabs;
      q.ctas = q.sum_ctas + zero_ctas;
      const size_t smem = CHUNK * BULK_ROW;
      if (e == cudaSuccess) e = ensure_smem((const void*)embed_bulk_kernel<T>, smem);
      if (e == cudaSuccess) e = launch_kernel(embed_bulk_kernel<T>, dim3((unsigned)q.ctas), BULK_THREADS, smem, st, q);
    }
  } else {
    // (entry by entry, four a thread where each SM has several CTAs all the same)
    const bool four = V == 1 && chunks * accesses >= (int64_t)dev.sm_count * THREADS * 4 * 8;
    q.shape = shape_of(accesses, four ? 4 : 1);
    q.shape.groups = std::min(q.shape.groups, GROUPS);
    q.sum_ctas = (chunks * q.shape.slabs + q.shape.groups - 1) / q.shape.groups;
    q.ctas = q.sum_ctas + zero_ctas;
    const unsigned threads = (unsigned)((q.shape.tpr * q.shape.groups + 31) / 32 * 32);
    if (e == cudaSuccess && !four) e = launch_kernel(embed_reduce_kernel<T, V, 1>, dim3((unsigned)q.ctas), threads, 0, st, q);
    if constexpr (V == 1) {
      if (e == cudaSuccess && four) e = launch_kernel(embed_reduce_kernel<T, V, 4>, dim3((unsigned)q.ctas), threads, 0, st, q);
    }
  }
  if (e == cudaSuccess && longs) {
    int tx = 1;
    while (tx < 32 && tx < accesses) tx *= 2;
    const int64_t slabs = (accesses + tx - 1) / tx, most = (chunks - 2) * slabs;
    e = launch_kernel(embed_join_kernel<T, V>, dim3((unsigned)std::min<int64_t>(most, (int64_t)dev.sm_count * 8)), JOIN, 0, st, q, tx, slabs);
  }
  cudaFreeAsync(ws, st);
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

template <typename T>
fxtx_status_t run_t(const EmbedArgs& a, bool backward, const DeviceInfo& dev, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T), S = sizeof(T);
  const bool wide = a.n % V == 0 && aligned(a.src, a.lds, S) && aligned(a.out, a.ldo, S);
  if (backward) return wide ? gradient<T, V>(a, dev, st) : gradient<T, 1>(a, dev, st);
  const cudaError_t e = wide ? lookup<T, V>(a, dev, st) : lookup<T, 1>(a, dev, st);
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

fxtx_status_t run(fxtx_type_t type, const EmbedArgs& a, bool backward, const DeviceInfo& dev, cudaStream_t st) {
  switch (type) {
    case FXTX_F32: return run_t<float>(a, backward, dev, st);
    case FXTX_BF16: return run_t<__nv_bfloat16>(a, backward, dev, st);
    default: return run_t<__half>(a, backward, dev, st);
  }
}

}  // namespace

fxtx_status_t run_embed(fxtx_type_t type, const EmbedArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  return run(type, a, false, dev, st);
}
fxtx_status_t run_embed_grad(fxtx_type_t type, const EmbedArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  return run(type, a, true, dev, st);
}

}  // namespace fxtx
