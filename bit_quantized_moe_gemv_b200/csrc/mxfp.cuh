// What the microscaled fp4 kernels share: the scale layout and decoding.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

#include "moe.h"
#include "moe_common.cuh"

namespace moe {

constexpr int kMaxFpCols = 1 << 24;

// Bytes between the scale rows of a [*, cols] matrix: its blocks, rounded up
// to 16 so that every row starts aligned.
__host__ __device__ inline int scale_stride(bool nv, int cols) { return (cols / (nv ? 16 : 32) + 15) & ~15; }

template <bool kNv>
__device__ __forceinline__ float scale_value(uint8_t b) {
  if (kNv) return f16_to_f32(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3).x);
  if (b == 0xff) return __uint_as_float(0x7fc00000u);
  return __uint_as_float(b ? uint32_t(b) << 23 : 0x00400000u);  // 2^-127 is subnormal
}

}  // namespace moe
