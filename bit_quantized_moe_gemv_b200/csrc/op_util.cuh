// Helpers shared by the row-sort and fp4 operators: element types, vector
// access and the argument checks their entry points have in common.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

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

// The status of a call that ends with `e`. A failure also stays behind as the
// runtime's last error, which the next launch of another call would report as its own.
inline moe_status launched(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ERR_CUDA;
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

// Chained launches: the kernel may be started while its predecessor on the
// stream still runs, and touches no memory before chain_wait, which returns
// when the predecessor is done and its writes are seen. A predecessor of this
// kind lets it start at chain_go, any other at its end. What runs before the
// wait (barriers, TMEM, descriptors) and the launch itself then overlap the
// predecessor: two small calls in a row take 5.5 us instead of 8.2.
// Inputs are written while the kernel is already there, so they are not
// read-only for its lifetime: their pointers are not __restrict__ (that would
// allow loads which need not see the predecessor's writes), the outputs' are.
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void chain_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... Params, typename... Actual>
cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                           Actual... args) {
  cudaLaunchAttribute chained{};
  chained.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  chained.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &chained;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
  count_launches(1);
  return e;
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

// N consecutive elements of type T that are loaded and stored together, held
// as the words they are (16-bit elements taken apart only where they are used:
// held one to a register they cost twice the registers, and the loads in
// flight are what hides the latency).
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  using Word = typename std::conditional<sizeof(T) * N == 2, uint16_t, uint32_t>::type;
  static constexpr int kWords = int(sizeof(T) * N / sizeof(Word));
  Word w[kWords];

  __device__ __forceinline__ void get(float (&v)[N]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __uint_as_float(w[i]);
    } else if constexpr (N == 1) {
      v[0] = std::is_same<T, __half>::value ? f16_to_f32(w[0]) : bf16_to_f32(w[0]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if constexpr (std::is_same<T, __half>::value) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          v[2 * i] = f.x;
          v[2 * i + 1] = f.y;
        } else {
          v[2 * i] = __uint_as_float(uint32_t(w[i]) << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      }
    }
  }
  __device__ __forceinline__ void set(const float (&v)[N]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __float_as_uint(v[i]);
    } else if constexpr (N == 1) {
      const T t = from_f32<T>(v[0]);
      w[0] = *reinterpret_cast<const uint16_t*>(&t);
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if constexpr (std::is_same<T, __half>::value) {
          const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
    }
  }
};

}  // namespace moe
