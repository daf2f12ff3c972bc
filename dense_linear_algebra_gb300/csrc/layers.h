// layers.h — element types, activations and argument blocks of the layer operators
// (the fused linear layer, its gradient, the AdamW step).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fxtx.h"
#include "plan.h"

namespace fxtx {

inline int type_size(fxtx_type_t t) { return t == FXTX_F32 ? 4 : 2; }
inline bool type_ok(int t) { return t >= FXTX_F32 && t <= FXTX_F16; }
inline bool act_ok(int a) { return a >= FXTX_ACT_NONE && a <= FXTX_ACT_SIGMOID; }

// The layer operators' kernels are launched so that each may start while the one before it on
// the stream drains: its CTAs are set up as SMs come free, and wait in after_previous() until that
// kernel has completed and its writes are seen. Every such kernel calls it, in all threads, before
// its first access to global memory. A launch then costs what its work does, not also the two
// microseconds between kernels (measured on calls of a few microseconds).
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Widening is exact; narrowing rounds to nearest even, once.
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// One AdamW launch sequence over `count` tensors (host table).
struct AdamwConst {
  float b1, c1, b2, c2;  // beta1, 1 - beta1, beta2, 1 - beta2
  float root;            // 1 / sqrt(1 - beta2^t)
  float eps;
  float keep;            // 1 - lr * weight_decay
  float rate;            // lr / (1 - beta1^t)
  float one = 1.f;
};
cudaError_t launch_adamw(int64_t count, const fxtx_adamw_tensor_t* t, int p_type, int g_type, int copy_type, int bits,
                         const AdamwConst& c, int sm_count, cudaStream_t st);
cudaError_t launch_adamw_moments(int64_t n, const int8_t* m, const float* ms, const uint8_t* r, const float* rs,
                                 float* m_out, float* v_out, cudaStream_t st);

}  // namespace fxtx
