// host.h — what the C entry points share: the current device's properties, transient
// workspace on the caller's stream, and the FXTX_LOG switch (defined in api.cu).
#pragma once

#include <cstddef>
#include <cuda_runtime.h>

#include "fxtx.h"
#include "plan.h"

namespace fxtx {

// Properties of the current device; FXTX_ERR_UNSUPPORTED without a compute capability 10.3 device.
fxtx_status_t current_device(const DeviceInfo** out);

// `bytes` of device memory in stream order (freed with cudaFreeAsync on the same stream);
// FXTX_ERR_ALLOC if it cannot be had, *p = nullptr for 0 bytes.
fxtx_status_t alloc_ws(void** p, size_t bytes, cudaStream_t st);

// The same from a pool of the library's own that keeps up to 1 GB between calls, so that a
// call after a synchronisation does not map its workspace anew (a fifth of a millisecond).
fxtx_status_t alloc_pooled(void** p, size_t bytes, cudaStream_t st);

// True when the environment variable FXTX_LOG is set and not "0".
bool log_enabled();

}  // namespace fxtx
