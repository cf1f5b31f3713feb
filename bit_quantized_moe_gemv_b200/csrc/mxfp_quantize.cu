// Microscaled 4-bit floating point: rows to E2M1 codes with block scales, and
// back.
//   MOE_FP_MX  one E8M0 scale 2^(b-127) per 32 elements of a row,
//              b - 127 = floor(log2(amax)) - 2;
//   MOE_FP_NV  one E4M3 scale s per 16 elements and one fp32 scale g per
//              tensor, s = E4M3(amax / (6 g)).
// A code is the E2M1 value nearest to x / scale, ties to even, saturating
// at 6.
//
// Rounding is decided on the exact quotient, so that codes do not depend on
// how a division was rounded: MX scales by powers of two, which is exact; in
// the other cases the fp32 quotient is used unless it lies within kNear units
// in the last place of a rounding border, where the exact comparison of x
// with border * scale decides (an fma for plain NV, whose border * s fits 7
// bits; 64-bit arithmetic for the SwiGLU input, whose fp32 value carries a few
// units of error).
//
// HBM bound: 8 elements per thread by 16-byte loads, a block's 4 (MX) or 2
// (NV) lanes exchange their maxima by shuffles, codes leave as one 32-bit word
// per thread.
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "call_range.h"
#include "mxfp.cuh"
#include "op_util.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
// Largest error of a computed quotient, in units in the last place: expf 2,
// the sum 0.5 and the division 0.5 of silu, the product 0.5, the scale's
// product and reciprocal 1, the last product 0.5; taken three times.
constexpr uint32_t kNear = 16;

// Rows in chunks of 8 elements: chunk g is chunk (g % per_row) of row
// (g / per_row). For fewer than 2^31 chunks the quotient comes from one
// multiplication: m = floor(2^(31+l) / d) + 1 with 2^l >= d is exact there.
struct Split {
  long long total;
  uint32_t per_row, mul;
  int shift;
};
Split make_split(long long rows, int per_row) {
  Split s{rows * per_row, uint32_t(per_row), 0, 0};
  int l = 0;
  while ((1u << l) < s.per_row) ++l;
  s.mul = uint32_t(((1ull << (31 + l)) / s.per_row) + 1);
  s.shift = 31 + l;
  return s;
}
__device__ __forceinline__ void split_at(const Split& s, long long g, long long* row, uint32_t* chunk) {
  if (s.total <= 0x7fffffffLL) {
    const uint32_t n = uint32_t(g), q = uint32_t((uint64_t(n) * s.mul) >> s.shift);
    *row = q;
    *chunk = n - q * s.per_row;
  } else {
    *row = g / s.per_row;
    *chunk = uint32_t(g - *row * s.per_row);
  }
}

__device__ __forceinline__ long long rows_in_use(const int* rows_dev, long long rows) {
  if (!rows_dev) return rows;
  const long long n = *rows_dev;
  return n < 0 ? 0 : n < rows ? n : rows;
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  constexpr int kVecs = sizeof(T) / 2;  // 16-byte loads
  Vec<T, 8 / kVecs> q[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) q[i] = reinterpret_cast<const Vec<T, 8 / kVecs>*>(p)[i];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f32(q[i / (8 / kVecs)].v[i % (8 / kVecs)]);
}

__device__ __forceinline__ double swiglu_f64(float gate, float up) {
  return double(gate) / (1.0 + exp(-double(gate))) * double(up);
}

// The value with `keep` mantissa bits nearest to v, and whether v lies in the
// range [lo, hi) that has borders and so near to it that an error of kNear
// units may have moved v across.
__device__ __forceinline__ bool near_border(float v, int keep, float lo_v, float hi_v, float* border) {
  const uint32_t u = __float_as_uint(v), low = (1u << (23 - keep)) - 1;
  const uint32_t b = (u + (low >> 1) + 1) & ~low;
  *border = __uint_as_float(b);
  return u + kNear - b <= 2 * kNear && v >= lo_v && v < hi_v;
}
// v moved to the side of the border that `diff` (x minus border * scale) says.
__device__ __forceinline__ float beside(float border, double diff) {
  return __uint_as_float(__float_as_uint(border) + (diff > 0) - (diff < 0));
}

// Codes and the scale byte of one block whose lanes hold 8 elements each.
template <typename T, bool kNv, bool kSwiglu>
__device__ __forceinline__ void quantise8(const float (&x)[8], const float (&up)[8], float g, uint32_t* codes,
                                          uint32_t* scale) {
  constexpr int kLanes = kNv ? 2 : 4;
  float h[8];
  uint32_t top = 0;  // bits of |h| order like the values, NaN above infinity
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = kSwiglu ? silu_f32(x[i]) * up[i] : x[i];
    top = max(top, __float_as_uint(h[i]) & 0x7fffffffu);
  }
#pragma unroll
  for (int o = 1; o < kLanes; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool bad = top >= 0x7f800000u;

  // largest |h| in 64 bits, for the rare border cases of the scale
  auto top_f64 = [&]() {
    double t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = fmax(t, fabs(kSwiglu ? swiglu_f64(x[i], up[i]) : double(h[i])));
#pragma unroll
    for (int o = 1; o < kLanes; o *= 2) t = fmax(t, __shfl_xor_sync(0xffffffffu, t, o));
    return t;
  };

  float s, inv;  // block scale without g, and 1 / (s g)
  if (kNv) {
    float q = __uint_as_float(top) / (6.f * g), border;
    const bool near = !bad && near_border(q, 4, 0x1p-11f, 512.f, &border);
    if (__any_sync(0xffffffffu, near)) {
      const double t = top_f64();
      if (near) q = beside(border, t - double(border) * 6.0 * double(g));
    }
    const __nv_fp8_storage_t b = __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
    *scale = bad ? 0x7fu : b;
    s = f16_to_f32(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3).x);
    inv = s > 0.f ? 1.f / (s * g) : 0.f;
  } else {
    if (kSwiglu) {
      const uint32_t up_ = (top + kNear) & 0x7fffffu;  // small when top is about a power of two
      const bool near = !bad && up_ <= 2 * kNear && top > 0x01000000u;  // below, the scale byte is 0 either way
      if (__any_sync(0xffffffffu, near)) {
        const double t = top_f64();
        if (near) {
          const uint32_t b = (top + kNear) & 0xff800000u;  // the power of two
          top = t < double(__uint_as_float(b)) ? b - 1 : b;
        }
      }
    }
    const int e = int(top >> 23) - 2;  // biased floor(log2), less E2M1's largest exponent
    *scale = bad ? 0xffu : uint32_t(max(e, 0));
    s = 1.f;  // borders are compared in units of the scale below
    inv = __uint_as_float(uint32_t(254 - max(e, 0)) << 23);
  }

  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float v[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      v[c] = fabsf(h[i + c]) * inv;
      if (kNv || kSwiglu) {
        float border;
        if (near_border(v[c], 2, 0.125f, 8.f, &border)) {
          if (kSwiglu) {
            const double unit = kNv ? double(s) * double(g) : 1.0 / double(inv);
            v[c] = beside(border, fabs(swiglu_f64(x[i + c], up[i + c])) - double(border) * unit);
          } else {
            v[c] = beside(border, fmaf(-(border * s), g, fabsf(h[i + c])));
          }
        }
      }
      v[c] = copysignf(v[c], h[i + c]);
    }
    word |= uint32_t(__nv_cvt_float2_to_fp4x2(make_float2(v[0], v[1]), __NV_E2M1, cudaRoundNearest)) << (4 * i);
  }
  *codes = bad || (kNv && s == 0.f) ? 0u : word;
}

template <typename T, bool kNv, bool kSwiglu, int kUnroll>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const T* __restrict__ x, long long rows, Split sp, int scale_stride, const float* __restrict__ tscale,
                const int* __restrict__ rows_dev, uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr int kLanes = kNv ? 2 : 4;
  const float g = kNv && tscale ? *tscale : 1.f;
  const long long limit = rows_in_use(rows_dev, rows) * sp.per_row;
  const long long g0 = (long long)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  float v[kUnroll][8], u[kUnroll][8];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const long long n = g0 + i * kThreads;
#pragma unroll
    for (int q = 0; q < 8; ++q) v[i][q] = u[i][q] = 0.f;
    if (n >= limit) continue;
    long long row;
    uint32_t c;
    if (kSwiglu) {
      split_at(sp, n, &row, &c);
      const T* p = x + row * 2 * (8LL * sp.per_row) + 8LL * c;
      load8(p, v[i]);
      load8(p + 8LL * sp.per_row, u[i]);
    } else {
      load8(x + n * 8, v[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const long long n = g0 + i * kThreads;
    uint32_t word, sc;
    quantise8<T, kNv, kSwiglu>(v[i], u[i], g, &word, &sc);  // all lanes: it exchanges maxima
    if (n >= limit) continue;
    codes[n] = word;
    if (n % kLanes == 0) {
      long long row;
      uint32_t c;
      split_at(sp, n, &row, &c);
      uint8_t* d = scales + row * scale_stride + c / kLanes;
      *d = uint8_t(sc);
      if (c + kLanes == sp.per_row)  // the row's last block: zeros up to the stride
        for (int b = int(c / kLanes) + 1; b < scale_stride; ++b) *++d = 0;
    }
  }
}

// 8 elements per thread: one word of codes, one scale byte (its block's other
// lanes read the same), 16-byte stores.
template <typename T, bool kNv>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, long long rows, Split sp,
                  int scale_stride, const float* __restrict__ tscale, const int* __restrict__ rows_dev,
                  T* __restrict__ out) {
  constexpr int kLanes = kNv ? 2 : 4, kVecs = sizeof(T) / 2;
  const float g = kNv && tscale ? *tscale : 1.f;
  const long long limit = rows_in_use(rows_dev, rows) * sp.per_row;
  const long long n = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (n >= limit) return;
  long long row;
  uint32_t c;
  split_at(sp, n, &row, &c);
  const uint32_t word = codes[n];
  const float s = scale_value<kNv>(scales[row * scale_stride + c / kLanes]);
  Vec<T, 8 / kVecs> o[kVecs];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const __half2_raw q = __nv_cvt_fp4x2_to_halfraw2(__nv_fp4x2_storage_t(word >> (4 * i)), __NV_E2M1);
    // code * s is exact; NV rounds once for g, then to T
    o[i / (8 / kVecs)].v[i % (8 / kVecs)] = from_f32<T>(f16_to_f32(q.x) * s * g);
    o[(i + 1) / (8 / kVecs)].v[(i + 1) % (8 / kVecs)] = from_f32<T>(f16_to_f32(q.y) * s * g);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) reinterpret_cast<Vec<T, 8 / kVecs>*>(out + n * 8)[i] = o[i];
}

template <typename T, bool kNv, bool kSwiglu>
cudaError_t run_quantize(const void* x, long long rows, int cols, const float* tscale, const int* rows_dev,
                         void* codes, uint8_t* scales, cudaStream_t st) {
  const Split sp = make_split(rows, cols / 8);
  const int stride = scale_stride(kNv, cols);
  // four chunks per thread keep enough loads in flight once the grid fills the GPU; small inputs spread wider
  constexpr int kUnroll = sizeof(T) == 4 || kSwiglu ? 2 : 4;
  if (sp.total >= 148LL * 8 * kThreads * kUnroll) {
    const long long grid = (sp.total + kThreads * kUnroll - 1) / (kThreads * kUnroll);
    quantize_kernel<T, kNv, kSwiglu, kUnroll><<<unsigned(grid), kThreads, 0, st>>>(
        static_cast<const T*>(x), rows, sp, stride, tscale, rows_dev, static_cast<uint32_t*>(codes), scales);
  } else {
    quantize_kernel<T, kNv, kSwiglu, 1><<<unsigned((sp.total + kThreads - 1) / kThreads), kThreads, 0, st>>>(
        static_cast<const T*>(x), rows, sp, stride, tscale, rows_dev, static_cast<uint32_t*>(codes), scales);
  }
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t quantize_as(bool nv, bool swiglu, const void* x, long long rows, int cols, const float* tscale,
                        const int* rows_dev, void* codes, uint8_t* scales, cudaStream_t st) {
  if (nv)
    return swiglu ? run_quantize<T, true, true>(x, rows, cols, tscale, rows_dev, codes, scales, st)
                  : run_quantize<T, true, false>(x, rows, cols, tscale, rows_dev, codes, scales, st);
  return swiglu ? run_quantize<T, false, true>(x, rows, cols, tscale, rows_dev, codes, scales, st)
                : run_quantize<T, false, false>(x, rows, cols, tscale, rows_dev, codes, scales, st);
}

template <typename T>
cudaError_t dequantize_as(bool nv, const void* codes, const uint8_t* scales, long long rows, int cols,
                          const float* tscale, const int* rows_dev, void* out, cudaStream_t st) {
  const Split sp = make_split(rows, cols / 8);
  const unsigned grid = unsigned((sp.total + kThreads - 1) / kThreads);
  if (nv)
    dequantize_kernel<T, true><<<grid, kThreads, 0, st>>>(static_cast<const uint32_t*>(codes), scales, rows, sp,
                                                         scale_stride(true, cols), tscale, rows_dev,
                                                         static_cast<T*>(out));
  else
    dequantize_kernel<T, false><<<grid, kThreads, 0, st>>>(static_cast<const uint32_t*>(codes), scales, rows, sp,
                                                          scale_stride(false, cols), tscale, rows_dev,
                                                          static_cast<T*>(out));
  count_launches(1);
  return cudaGetLastError();
}

// Shared by both directions. The chunk count is bounded by the grid: 2^31
// blocks of one chunk per thread.
moe_status convert_check(const void* wide, const void* codes, const uint8_t* scales, int32_t dtype, int64_t rows,
                         int32_t cols, int32_t format, const float* tscale, const int32_t* rows_dev) {
  if (format != MOE_FP_MX && format != MOE_FP_NV) return MOE_ERR_UNSUPPORTED;
  if (dtype_size(dtype) < 2) return MOE_ERR_UNSUPPORTED;
  if (rows < 0 || cols < 32 || cols % 32 || cols > kMaxFpCols) return MOE_ERR_INVALID_ARG;
  if (rows > (1LL << 38) / cols) return MOE_ERR_INVALID_ARG;
  if (format == MOE_FP_MX && tscale) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!wide || !codes || !scales || !ptr_aligned(wide, 16) || !ptr_aligned(codes, 16) || !ptr_aligned(scales, 16) ||
      !ptr_aligned(tscale, 4) || !ptr_aligned(rows_dev, 4))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int32_t moe_mxfp_scale_stride(int32_t cols, int32_t format) {
  if ((format != MOE_FP_MX && format != MOE_FP_NV) || cols < 32 || cols % 32 || cols > kMaxFpCols) return 0;
  return scale_stride(format == MOE_FP_NV, cols);
}

moe_status moe_mxfp_quantize(const void* x, int32_t dtype, int64_t rows, int32_t cols, int32_t format, uint32_t flags,
                             const float* tensor_scale, const int32_t* rows_dev, uint8_t* codes, uint8_t* scales,
                             void* stream) {
  const CallRange range("moe_mxfp_quantize");
  if (flags & ~uint32_t(MOE_FP_SWIGLU)) return MOE_ERR_INVALID_ARG;
  const moe_status s = convert_check(x, codes, scales, dtype, rows, cols, format, tensor_scale, rows_dev);
  if (s != MOE_OK || rows == 0) return s;
  const bool nv = format == MOE_FP_NV, swiglu = (flags & MOE_FP_SWIGLU) != 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == MOE_DT_BF16)
    e = quantize_as<__nv_bfloat16>(nv, swiglu, x, rows, cols, tensor_scale, rows_dev, codes, scales, st);
  else if (dtype == MOE_DT_FP16)
    e = quantize_as<__half>(nv, swiglu, x, rows, cols, tensor_scale, rows_dev, codes, scales, st);
  else
    e = quantize_as<float>(nv, swiglu, x, rows, cols, tensor_scale, rows_dev, codes, scales, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_mxfp_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols, int32_t format,
                               const float* tensor_scale, const int32_t* rows_dev, void* out, int32_t dtype,
                               void* stream) {
  const CallRange range("moe_mxfp_dequantize");
  const moe_status s = convert_check(out, codes, scales, dtype, rows, cols, format, tensor_scale, rows_dev);
  if (s != MOE_OK || rows == 0) return s;
  const bool nv = format == MOE_FP_NV;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == MOE_DT_BF16)
    e = dequantize_as<__nv_bfloat16>(nv, codes, scales, rows, cols, tensor_scale, rows_dev, out, st);
  else if (dtype == MOE_DT_FP16)
    e = dequantize_as<__half>(nv, codes, scales, rows, cols, tensor_scale, rows_dev, out, st);
  else
    e = dequantize_as<float>(nv, codes, scales, rows, cols, tensor_scale, rows_dev, out, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
