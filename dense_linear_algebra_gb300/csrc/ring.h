// ring.h — the turns of a ring of copies: a copying thread fills the stage of an item as soon as the one `stages` items before it has
// been read, and each fill completes a phase of its stage's barrier.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FXTX_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define FXTX_HOST_DEVICE inline
#endif

namespace fxtx {

struct RingTurn {
  int stages, s = 0;   // the stage in turn
  uint32_t phase = 0;  // the phase that its copies complete
  FXTX_HOST_DEVICE explicit RingTurn(int n) : stages(n) {}
  FXTX_HOST_DEVICE void next() {
    if (++s == stages) {
      s = 0;
      phase ^= 1u;
    }
  }
  // Of stage x: the turns until it is read, and the phase that its copies for that turn complete.
  FXTX_HOST_DEVICE int ahead(int x) const { return x < s ? x - s + stages : x - s; }
  FXTX_HOST_DEVICE uint32_t parity(int x) const { return x < s ? phase ^ 1u : phase; }
  // Whether those copies have been asked for when the copies of `item` are waited for: items are every step-th below `items`.
  template <typename I>
  FXTX_HOST_DEVICE bool asked(int x, I item, I items, I step) const {
    return item + ahead(x) * step < items;
  }
};

}  // namespace fxtx
