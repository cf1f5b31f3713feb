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
// the other cases the fp32 quotient is rounded twice, lowered and raised by its
// largest error, and where the codes differ a comparison of x with border *
// scale in 64 bits decides. Approximate reciprocals and exponentials are
// therefore enough in the common path.
//
// 8 elements per thread by 16-byte loads, a block's 4 (MX) or 2 (NV) lanes
// exchange their maxima by shuffles, codes leave as one 32-bit word per thread.
// Dequantising is bound by HBM (63 M values to bf16: 26 us in MX, 6.1 TB/s, 27 in NV).
// Quantising comes close to it where instructions are saved: products and sums
// two at a time, maxima three at a time, offsets that are constants (lanes side
// by side on a row), small blocks at 56 registers, 36 warps per SM (of 64
// registers, 32 warps: 51 us instead of 50). 63 M SwiGLU values of bf16 halves
// take 50 us (88 % of the copy rate; 22 instructions per value, two of them
// MUFU), 17 M bf16 values to NV 10.6 us (63 %; 13 instructions, and a fifth of
// the time is the start of the grid). Both issue on 0.6 to 0.7 of the
// cycles with no pipe above two thirds. The other forms, at the same two sizes:
// MX 7.8 us (fp16 7.5, fp32 12.2), NV of fp16 10.4, of fp32 14.3; SwiGLU of fp16
// 51 us in MX, of bf16 and fp16 57 in NV, of fp32 99 and 105. Those last spill
// most (up to 180 bytes a thread), and would take 79 and 88 us with 80 registers,
// where the 16-bit ones take 57 and 62.
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "call_range.h"
#include "mxfp.cuh"
#include "op_util.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
// How far, in units of 2^-23 of its value, a computed quotient may be from the
// exact one. Plain NV: scale product 0.5, reciprocal 1, two products 1, the
// shift itself 0.5. SwiGLU adds the approximate exp (gate * log2(e) is below 128
// here: its rounding gives 0.35 x 128, that of the constant 10; ex2 itself 2),
// the sum, the reciprocal and two products (2.5): 63.
constexpr float kOffPlain = 4.f * 0x1p-23f, kOffSwiglu = 80.f * 0x1p-23f;
// Beyond this sum of exponentials a reciprocal may have left the normal range.
constexpr float kExpSum = 0x1p120f;
// Gates below this (bits of a float) are rounded away when they are halved: their
// silu is a subnormal number, while its product with up need not be one. Only
// fp32 has such gates: the lowest bit of a 16-bit subnormal survives.
constexpr uint32_t kTinyGate = (127u - 120u) << 23;  // 2^-120
constexpr float kLargest = 0x1.fffffep127f, kInf = __builtin_huge_valf();

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

// 8 elements in one or two 16-byte words.
template <typename T>
struct Eight {
  static constexpr int kN = 16 / sizeof(T), kVecs = 8 / kN;
  Pack<T, kN> p[kVecs];
  __device__ __forceinline__ void load(const T* x) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) p[i] = reinterpret_cast<const Pack<T, kN>*>(x)[i];
  }
  __device__ __forceinline__ void store(T* x) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) reinterpret_cast<Pack<T, kN>*>(x)[i] = p[i];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float q[kN];
      p[i].get(q);
#pragma unroll
      for (int j = 0; j < kN; ++j) v[i * kN + j] = q[j];
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float q[kN];
#pragma unroll
      for (int j = 0; j < kN; ++j) q[j] = v[i * kN + j];
      p[i].set(q);
    }
  }
};

__device__ __forceinline__ double swiglu_f64(float gate, float up) {
  return double(gate) / (1.0 + exp(-double(gate))) * double(up);
}
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// Largest magnitude of three, NaN if one of them is.
__device__ __forceinline__ float abs_max3(float a, float b, float c) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float abs_max8(const float (&v)[8]) {
  return abs_max3(abs_max3(v[0], v[1], v[2]), abs_max3(v[3], v[4], v[5]), max_nan(fabsf(v[6]), fabsf(v[7])));
}
// Two products or sums by one instruction, rounded as each alone.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, y;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 y, a, b;\n\tmov.b64 {%0, %1}, y;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, y;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 y, a, b;\n\tmov.b64 {%0, %1}, y;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
// The value with `keep` mantissa bits nearest to v.
__device__ __forceinline__ float border_of(float v, int keep) {
  const uint32_t low = (1u << (23 - keep)) - 1;
  return __uint_as_float((__float_as_uint(v) + (low >> 1) + 1) & ~low);
}
// The float next to the border on the side that `diff` (x minus border *
// scale) says, or the border itself.
__device__ __forceinline__ float beside(float border, double diff) {
  return __uint_as_float(__float_as_uint(border) + (diff > 0) - (diff < 0));
}
__device__ __forceinline__ uint32_t e2m1x2(float low, float high) {
  return __nv_cvt_float2_to_fp4x2(make_float2(low, high), __NV_E2M1, cudaRoundNearest);
}
// Codes of 8 values times f, the first in the low nibble. One instruction
// sequence, so that the conversions place their bytes themselves.
__device__ __forceinline__ uint32_t e2m1_word(const float (&h)[8], float f) {
  uint32_t w;
  float2 q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = mul2(make_float2(h[2 * i], h[2 * i + 1]), make_float2(f, f));
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(q[0].x), "f"(q[0].y), "f"(q[1].x), "f"(q[1].y), "f"(q[2].x), "f"(q[2].y), "f"(q[3].x), "f"(q[3].y));
  return w;
}
// Largest magnitude of 8 elements, NaN if one of them is. Without their signs
// the bits of 16-bit floats order like the values, NaN above infinity: two at a
// time by integer maxima.
template <typename T>
__device__ __forceinline__ float abs_max(const Eight<T>& v) {
  if constexpr (sizeof(T) == 2) {
    uint32_t m = v.p[0].w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __vmaxu2(m, v.p[0].w[i] & 0x7fff7fffu);
    const uint16_t b = uint16_t(max(m & 0xffffu, m >> 16));
    return std::is_same<T, __half>::value ? f16_to_f32(b) : bf16_to_f32(b);
  } else {
    float x[8];
    v.get(x);
    return abs_max8(x);
  }
}

// The rare exact decisions read the 8 elements again (`up` of SwiGLU inputs
// is up_at elements behind): out of line and from memory, they cost the common
// path neither registers nor instruction cache.
struct Floats8 {
  float v[8];
};
// silu(gate) up, for gates whose exponential overflows 32 bits or whose silu falls below them.
template <typename T>
__device__ __noinline__ Floats8 exact_swiglu(const T* x, long long up_at) {
  Eight<T> v, u;
  v.load(x);
  u.load(x + up_at);
  float a[8], b[8];
  v.get(a);
  u.get(b);
  Floats8 h;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    h.v[i] = float(a[i] < -80.f ? double(a[i]) * exp(double(a[i])) * double(b[i]) : swiglu_f64(a[i], b[i]));
  return h;
}
template <typename T, bool kSwiglu>
__device__ __noinline__ double exact_top(const T* x, long long up_at) {
  Eight<T> v, u;
  v.load(x);
  u.load(x + up_at);
  float a[8], b[8];
  v.get(a);
  u.get(b);
  double t = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) t = fmax(t, fabs(kSwiglu ? swiglu_f64(a[i], b[i]) : double(a[i])));
  return t;
}
// `word` with the codes that `differ` has bits in decided exactly; scale = s g,
// inv about its reciprocal.
template <typename T, bool kSwiglu>
__device__ __noinline__ uint32_t exact_codes(const T* x, long long up_at, float s, float g, float inv, uint32_t word,
                                             uint32_t differ) {
  Eight<T> v, u;
  v.load(x);
  u.load(x + up_at);
  float a[8], b[8];
  v.get(a);
  u.get(b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (differ >> (4 * i) & 15u) {
      const double h = kSwiglu ? swiglu_f64(a[i], b[i]) : double(a[i]);
      // borders between E2M1 values have 2 mantissa bits; border * s * g is exact in 64 bits
      const float border = border_of(fabsf(float(h)) * inv, 2);
      const float q = beside(border, fabs(h) - double(border) * double(s) * double(g));
      word = (word & ~(15u << (4 * i))) | (e2m1x2(copysignf(q, float(h)), 0.f) & 15u) << (4 * i);
    }
  }
  return word;
}

// Codes and the scale byte of one block whose lanes hold 8 elements each, read
// from x (lanes that read none, `has` false, hold zeros). g: the tensor scale,
// inv6g about 1 / (6 g).
template <typename T, bool kNv, bool kSwiglu>
__device__ __forceinline__ void quantise8(const Eight<T>& v, const Eight<T>& u, const T* x, long long up_at, bool has,
                                          float g, float inv6g, uint32_t* codes, uint32_t* scale) {
  constexpr int kLanes = kNv ? 2 : 4;
  constexpr float kOff = kSwiglu ? kOffSwiglu : kOffPlain;
  float h[8];
  float top = 0.f;
  v.get(h);
  if (kSwiglu) {
    float up[8];
    float2 exps = make_float2(0.f, 0.f);
    uint32_t least = 0xffffffffu;  // smallest gate, as twice its bits less one: no sign, zeros last
    u.get(up);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 gate = make_float2(h[i], h[i + 1]);
      if (sizeof(T) == 4)
        least = min(least, min(2 * __float_as_uint(gate.x) - 1, 2 * __float_as_uint(gate.y) - 1));
      float2 e = mul2(gate, make_float2(-1.4426950408889634f, -1.4426950408889634f));
      e = make_float2(ex2_approx(e.x), ex2_approx(e.y));
      exps = add2(exps, e);
      e = add2(e, make_float2(1.f, 1.f));
      e = mul2(mul2(gate, make_float2(rcp_approx(e.x), rcp_approx(e.y))), make_float2(up[i], up[i + 1]));
      h[i] = e.x;
      h[i + 1] = e.y;
    }
    if (!(exps.x + exps.y < kExpSum) || least < 2 * kTinyGate - 1) {
      const Floats8 r = exact_swiglu<T>(x, up_at);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = r.v[i];
    }
  }
  top = kSwiglu ? abs_max8(h) : abs_max<T>(v);
#pragma unroll
  for (int o = 1; o < kLanes; o *= 2) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));

  // largest |h| in 64 bits, for the rare border cases of the scale
  auto top_f64 = [&]() {
    double t = has ? exact_top<T, kSwiglu>(x, up_at) : 0.0;
#pragma unroll
    for (int o = 1; o < kLanes; o *= 2) t = fmax(t, __shfl_xor_sync(0xffffffffu, t, o));
    return t;
  };

  // SwiGLU values next to the end of the fp32 range: the computed one does not
  // tell whether they are inside, and may be infinite
  const float held = kSwiglu ? fminf(top, kLargest) : top;

  float s, inv;  // block scale without g, and about 1 / (s g)
  bool bad;      // an infinity or a NaN, or a value out of the range
  if (kNv) {
    float q = held * inv6g;
    __nv_fp8_storage_t b = __nv_cvt_float_to_fp8(q * (1.f - kOff), __NV_SATFINITE, __NV_E4M3);
    const bool near = b != __nv_cvt_float_to_fp8(q * (1.f + kOff), __NV_SATFINITE, __NV_E4M3);
    const bool end = kSwiglu && top > kLargest * (1.f - kOff);
    if (__any_sync(0xffffffffu, near || end)) {
      const double t = top_f64();
      if (near) {
        const float border = border_of(q, 4);  // borders between E4M3 values have 4 mantissa bits
        q = beside(border, t - double(border) * 6.0 * double(g));
        b = __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
      }
      if (end) top = t <= double(kLargest) ? held : kInf;
    }
    bad = !(top <= kLargest);
    *scale = bad ? 0x7fu : b;
    s = f16_to_f32(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3).x);
    inv = s > 0.f ? rcp_approx(s * g) : 0.f;
  } else {
    if (kSwiglu) {
      // the exponent changes at a power of two, infinity (the end of the range) among them;
      // the lowest that changes the scale byte (0 to 1) is 2^-124
      const uint32_t above = __float_as_uint(held * (1.f + kOff)) & 0xff800000u;
      const bool near = __float_as_uint(held * (1.f - kOff)) < above && held > 0x1p-125f;
      if (__any_sync(0xffffffffu, near)) {
        const double t = top_f64();
        const float border = __uint_as_float(above);
        if (near && top == top)  // a NaN stays
          top = (border == kInf ? t <= double(kLargest) : t < double(border)) ? __uint_as_float(above - 1) : border;
      }
    }
    bad = !(top <= kLargest);
    const int e = max(int(__float_as_uint(top) >> 23) - 2, 0);  // biased floor(log2), less E2M1's largest exponent
    *scale = bad ? 0xffu : uint32_t(e);
    s = e ? __uint_as_float(uint32_t(e) << 23) : 0x1p-127f;
    inv = __uint_as_float(uint32_t(254 - e) << 23);
  }

  uint32_t word = e2m1_word(h, kNv || kSwiglu ? inv * (1.f - kOff) : inv);
  if (kNv || kSwiglu) {
    // a code that the uncertainty of its quotient could change is decided exactly
    const uint32_t differ = word ^ e2m1_word(h, inv * (1.f + kOff));
    if (differ && has) word = exact_codes<T, kSwiglu>(x, up_at, s, g, inv, word, differ);
  }
  *codes = bad || (kNv && s == 0.f) ? 0u : word;
}

// How warps share the chunks of 8 elements: 2^lg lanes side by side on a row
// (32 >> lg rows per warp), each lane with up to kUnroll chunks 2^lg apart.
// Warps of a block take consecutive rows, blockIdx.y the parts of long ones.
struct WarpSplit {
  int per_row, lg, parts;
  long long groups;  // of 32 >> lg rows
};
WarpSplit warp_split(long long rows, int per_row, int unroll) {
  // as many lanes on a row as keep 9 of 10 busy; 4 lanes (a block) always do
  int lg = 5;
  while (lg > 2 && 10 * per_row < 9 * (((per_row + (1 << lg) - 1) >> lg) << lg)) --lg;
  return {per_row, lg, (per_row + (unroll << lg) - 1) / (unroll << lg), (rows + (32 >> lg) - 1) / (32 >> lg)};
}

// kLg: lanes on a row, so that all offsets are constants; -1 for any.
template <typename T, bool kNv, bool kSwiglu, int kUnroll, int kLg>
__global__ void __launch_bounds__(kThreads, 9)
quantize_kernel(const T* x, long long rows, int per_row, int lg, int scale_stride, const float* tscale,
                const int* rows_dev, uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr int kLanes = kNv ? 2 : 4;
  if (kLg >= 0) lg = kLg;
  chain_go();
  chain_wait();
  const uint32_t lane = threadIdx.x % 32;
  const long long row0 = ((long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32) << (5 - lg);
  const long long used = rows_in_use(rows_dev, rows);
  if (row0 >= used) return;
  const float g = kNv && tscale ? *tscale : 1.f;
  const float inv6g = 1.f / (6.f * g);
  const long long row = row0 + (lane >> lg);
  const int step = 1 << lg;
  const int c0 = int(blockIdx.y) * (kUnroll << lg) + int(lane & (step - 1));
  const int left = row < used ? per_row - c0 : 0;  // chunks of this lane's row from c0 on
  x += (row * (kSwiglu ? 2 : 1) * per_row + c0) * 8;
  codes += row * per_row + c0;
  scales += row * scale_stride + c0 / kLanes;
  const long long up_at = kSwiglu ? per_row * 8LL : 0;
  Eight<T> v[kUnroll], u[kSwiglu ? kUnroll : 1];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    v[i] = {};
    if (kSwiglu) u[i] = {};
    if (i * step < left) {
      v[i].load(x + i * step * 8);
      if (kSwiglu) u[i].load(x + i * step * 8 + up_at);
    }
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    uint32_t word, sc;
    // all lanes: it exchanges maxima
    quantise8<T, kNv, kSwiglu>(v[i], u[kSwiglu ? i : 0], x + i * step * 8, up_at, i * step < left, g, inv6g, &word,
                               &sc);
    if (i * step < left) {
      codes[i * step] = word;
      if (lane % kLanes == 0) scales[i * step / kLanes] = uint8_t(sc);
    }
  }
  // zeros behind the row's last block, up to the stride
  if (blockIdx.y == gridDim.y - 1 && row < used)
    for (int k = per_row / kLanes + int(lane & (step - 1)); k < scale_stride; k += step) scales[k - c0 / kLanes] = 0;
}

// The NV value of a 16-bit T is rounded once, although the product code * s * g
// goes through 32 bits: cut there and, where that loses something, made odd, it is
// on the same side of every tie between two T as the exact one.
__device__ __forceinline__ float times_odd(float v, float g) {
  const float p = __fmul_rz(v, g);
  return fmaf(v, g, -p) != 0.f ? __uint_as_float(__float_as_uint(p) | 1u) : p;
}
// That is needed only where the nearest 32-bit product is on a tie. Codes are
// powers of two, once or one and a half times, so that the values of a block have
// two mantissas, those of s g and of 1.5 s g: one look at both spares the rest
// (8,192 x 2,048: 7.4 us, 8.5 with every product made odd). Ties of fp16 below its
// normal range, 2^-14, are elsewhere: those blocks are all done with care. bf16 has
// fp32's range, and no value here is below 2^-101.
template <typename T>
__device__ __forceinline__ bool may_tie(float s, float g) {
  constexpr bool kHalf = std::is_same<T, __half>::value;
  constexpr uint32_t kMask = kHalf ? 0x1fffu : 0xffffu, kTie = kHalf ? 0x1000u : 0x8000u;
  const float a = s * g, b = 1.5f * s * g;
  return (__float_as_uint(a) & kMask) == kTie || (__float_as_uint(b) & kMask) == kTie || (kHalf && a < 0x1p-13f);
}

// 8 elements at a time: one word of codes, one scale byte (its block's other
// lanes read the same), 16-byte stores.
template <typename T, bool kNv, int kUnroll>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(const uint32_t* codes, const uint8_t* scales, long long rows, Split sp,
                  int scale_stride, const float* tscale, const int* rows_dev,
                  T* __restrict__ out) {
  constexpr int kLanes = kNv ? 2 : 4;
  chain_go();
  chain_wait();
  const float g = kNv && tscale ? *tscale : 1.f;
  const long long limit = rows_in_use(rows_dev, rows) * sp.per_row;
  const long long n0 = (long long)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  uint32_t word[kUnroll];
  uint8_t sc[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const long long n = n0 + i * kThreads;
    if (n >= limit) break;
    word[i] = codes[n];
    if (uint32_t(scale_stride) * kLanes == sp.per_row) {
      sc[i] = scales[n / kLanes];
    } else {
      long long row;
      uint32_t c;
      split_at(sp, n, &row, &c);
      sc[i] = scales[row * scale_stride + c / kLanes];
    }
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const long long n = n0 + i * kThreads;
    if (n >= limit) break;
    const float s = scale_value<kNv>(sc[i]);
    float v[8];  // code * s, which is exact
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const __half2_raw q = __nv_cvt_fp4x2_to_halfraw2(__nv_fp4x2_storage_t(word[i] >> (4 * j)), __NV_E2M1);
      v[j] = f16_to_f32(q.x) * s;
      v[j + 1] = f16_to_f32(q.y) * s;
    }
    if (kNv) {
      if (sizeof(T) == 2 && may_tie<T>(s, g)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = times_odd(v[j], g);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= g;
      }
    }
    Eight<T> o;
    o.set(v);
    o.store(out + n * 8);
  }
}

template <typename T, bool kNv, bool kSwiglu>
cudaError_t run_quantize(const void* x, long long rows, int cols, const float* tscale, const int* rows_dev,
                         void* codes, uint8_t* scales, cudaStream_t st) {
  // Several chunks per lane keep enough loads in flight once the grid fills
  // the GPU (NV of 2,048 columns: 9.7 us in fours, 10.8 in twos); small inputs
  // spread wider. Lanes behind a row's end compute all the same, so three chunks
  // where they leave fewer of those (rows of 96 chunks, SwiGLU: a third of the
  // lanes' work in twos). Rows have at most 2^21 chunks, 2^15 parts.
  constexpr int kUnroll = sizeof(T) == 4 || kSwiglu ? 2 : 4;
  const T* in = static_cast<const T*>(x);
  uint32_t* out = static_cast<uint32_t*>(codes);
  const int stride = scale_stride(kNv, cols), per_row = cols / 8;
  auto launch = [&](auto* kernel, const WarpSplit& w) {
    const dim3 grid(unsigned((w.groups + kThreads / 32 - 1) / (kThreads / 32)), unsigned(w.parts));
    return launch_chained(kernel, grid, kThreads, 0, st, in, rows, per_row, w.lg, stride, tscale, rows_dev, out, scales);
  };
  if (rows * per_row < 148LL * 8 * kThreads * kUnroll)
    return launch(quantize_kernel<T, kNv, kSwiglu, 1, -1>, warp_split(rows, per_row, 1));
  const WarpSplit a = warp_split(rows, per_row, kUnroll), b = warp_split(rows, per_row, 3);
  if (a.parts * kUnroll <= b.parts * 3)
    return launch(a.lg == 5 ? quantize_kernel<T, kNv, kSwiglu, kUnroll, 5> : quantize_kernel<T, kNv, kSwiglu, kUnroll, -1>, a);
  return launch(b.lg == 5 ? quantize_kernel<T, kNv, kSwiglu, 3, 5> : quantize_kernel<T, kNv, kSwiglu, 3, -1>, b);
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
  const int stride = scale_stride(nv, cols);
  const bool big = sp.total >= 148LL * 8 * kThreads * 4;  // as above
  const int per = kThreads * (big ? 4 : 1);
  const unsigned grid = unsigned((sp.total + per - 1) / per);
  auto* kernel = nv ? big ? dequantize_kernel<T, true, 4> : dequantize_kernel<T, true, 1>
                    : big ? dequantize_kernel<T, false, 4> : dequantize_kernel<T, false, 1>;
  return launch_chained(kernel, dim3(grid), kThreads, 0, st, static_cast<const uint32_t*>(codes), scales, rows, sp,
                        stride, tscale, rows_dev, static_cast<T*>(out));
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
  return launched(e);
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
  return launched(e);
}

}  // extern "C"
