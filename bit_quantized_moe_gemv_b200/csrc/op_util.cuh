// Helpers shared by the row-sort and fp4 operators: element types, vector
// access and the argument checks their entry points have in common.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"
#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {

inline bool ptr_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The status word at the start of `ws`: what the operators without scratch
// need of a workspace.
inline moe_status status_ws_check(const void* ws, size_t ws_bytes) {
  if (ws == nullptr || !ptr_aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  return ws_bytes < size_t(MOE_STATUS_BYTES) ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

// Bytes of one element, 0 for an unknown type.
inline int dtype_size(int32_t dtype) {
  switch (dtype) {
    case MOE_DT_BF16:
    case MOE_DT_FP16: return 2;
    case MOE_DT_FP32: return 4;
    case MOE_DT_U8: return 1;
    default: return 0;
  }
}

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

// N elements that are loaded and stored together.
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T v[N];
};

}  // namespace moe
