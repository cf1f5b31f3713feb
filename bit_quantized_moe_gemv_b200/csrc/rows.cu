// Rows sorted by expert and back, with their gradients:
//   permute         xp[inv[t,j]] = x[t]
//   permute_grad    dx[t]        = sum_j dxp[inv[t,j]]
//   unpermute       out[t]       = sum_j w[t,j] y[inv[t,j]]
//   unpermute_grad  dy[inv[t,j]] = w[t,j] dout[t],  dw[t,j] = <dout[t], y[inv[t,j]]>
// inv is moe_dispatch's inv_perm; -1 is a pair without a row.
//
// All four are bound by HBM, and all four are driven by the token side of the
// permutation: a token's row is read (or written) once whatever k is, a row no
// pair points to is never touched, sums run over j in order in registers (no
// atomics, the same bits every time) and are rounded once. What decides is the
// bytes in flight: rows are loaded five at a time and kept packed until they
// are added, so that a thread needs 64 registers and 32 warps fit an SM (116
// registers and 14 warps with the elements taken apart: 97 us for unpermute).
// 8,192 tokens x 2,048 bf16, ten experts: permute 60 us, permute_grad 57,
// unpermute 58 (6.2 to 6.5 TB/s), unpermute_grad 111 (6.4 TB/s).
#include "call_range.h"
#include "op_util.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;     // of a block of the gradient kernel
constexpr int kSegWarps = 4;  // of the others: small blocks spread evenly over the SMs

// Row of pair p, or -1. A row outside [0, nrows) is reported and left out.
__device__ __forceinline__ int pair_row(const int* inv, long long p, long long nrows, WsHeader* hdr) {
  const int r = inv[p];
  if (r >= -1 && r < nrows) return r;
  flag_error(hdr, MOE_ERR_DEVICE_FAULT, r);
  return -1;
}

// One warp per segment of a token's row, the segments of all rows in one line.
// The sums take them as they are, so that no warp is without one however many a
// row has (8,192 tokens x 1,032 16-bit values, five segments: unpermute 28 us;
// with eight warps per row 35). permute, which waits for nothing but its own
// stores, rounds them up to a power of two and lets the surplus warps leave, as
// long as those are at most two for three that stay: five segments in eight warps
// take 4.3 us at 1,021 tokens x 1,032 (as they are 4.7; the same at 8,192), but
// nine in sixteen 34.6 us at 8,192 x 1,028 and 6.9 at 1,021 x 2,056 (as they are
// 24.7 and 6.0).
struct Segments {
  int per_row, shift;  // shift: log2(per_row) or -1
  long long all;
  unsigned blocks() const { return unsigned((all + kSegWarps - 1) / kSegWarps); }
};
Segments row_segments(long long T, int nvec, int seg, bool rounded) {
  const int n = (nvec + seg - 1) / seg;
  int l = 0;
  while ((1 << l) < n) ++l;
  const int per_row = rounded && 3LL << l <= 5LL * n ? 1 << l : n;
  return {per_row, per_row == 1 << l ? l : -1, T * per_row};
}
// This warp's token and segment; false if there is none.
__device__ __forceinline__ bool segment_at(const Segments& s, int* token, int* seg) {
  const long long w = (long long)blockIdx.x * kSegWarps + (threadIdx.x >> 5);
  if (w >= s.all) return false;
  if (s.shift >= 0)
    *token = int(w >> s.shift);
  else if (s.all <= 0xffffffffLL)
    *token = int(uint32_t(w) / uint32_t(s.per_row));
  else
    *token = int(w / s.per_row);
  *seg = int(w - (long long)*token * s.per_row);
  return true;
}

// Vectors that a lane takes of a segment: narrow ones (rows that are not
// 16-byte aligned) several at a time, to keep more bytes in flight.
template <typename V>
constexpr int lane_vecs() { return sizeof(V) >= 8 ? 1 : sizeof(V) == 4 ? 4 : 6; }

// One warp: a segment of a token's row is read once and written to the
// token's k rows.
template <typename V>
__global__ void __launch_bounds__(kSegWarps * 32)
permute_kernel(const V* x, const int* inv, long long nrows, int k, int nvec, Segments segs, V* __restrict__ xp,
               WsHeader* hdr) {
  constexpr int kU = lane_vecs<V>(), kSeg = 32 * kU;
  chain_go();
  chain_wait();
  const int lane = threadIdx.x & 31;
  int t, s;
  if (!segment_at(segs, &t, &s) || s * kSeg >= nvec) return;
  const long long p0 = (long long)t * k;
  const int c = s * kSeg + lane;
  V v[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) v[u] = x[(size_t)t * nvec + min(c + 32 * u, nvec - 1)];
  for (int j0 = 0; j0 < k; j0 += 32) {
    const int mine = j0 + lane < k ? pair_row(inv, p0 + j0 + lane, nrows, hdr) : -1;
    const int n = min(32, k - j0);
    for (int j = 0; j < n; ++j) {
      const int r = __shfl_sync(0xffffffffu, mine, j);
      if (r < 0) continue;
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (c + 32 * u < nvec) xp[(size_t)r * nvec + c + 32 * u] = v[u];
    }
  }
}

// Adds kB rows, all loads first. Rows of -1 are left out and not read.
template <typename T, int N, int kU, int kB, bool kWeighted>
__device__ __forceinline__ void add_rows(const Pack<T, N>* y, int mine, float wmine, int j, int nvec,
                                         const int (&c)[kU], float (&acc)[kU][N]) {
  int row[kB];
  bool all = true;
#pragma unroll
  for (int b = 0; b < kB; ++b) {
    row[b] = __shfl_sync(0xffffffffu, mine, j + b);
    all = all && row[b] >= 0;
  }
  Pack<T, N> v[kB][kU];
  if (all) {
#pragma unroll
    for (int b = 0; b < kB; ++b)
#pragma unroll
      for (int u = 0; u < kU; ++u) v[b][u] = y[(size_t)row[b] * nvec + c[u]];
  } else {
#pragma unroll
    for (int b = 0; b < kB; ++b)
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (row[b] >= 0) v[b][u] = y[(size_t)row[b] * nvec + c[u]];
  }
#pragma unroll
  for (int b = 0; b < kB; ++b) {
    const float w = kWeighted ? __shfl_sync(0xffffffffu, wmine, j + b) : 1.f;
    if (all || row[b] >= 0) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        float x[N];
        v[b][u].get(x);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[u][i] = kWeighted ? fmaf(w, x[i], acc[u][i]) : acc[u][i] + x[i];
      }
    }
  }
}

// One warp: a segment of out[t], the rows of several pairs in flight.
template <typename T, int N, bool kWeighted>
__global__ void __launch_bounds__(kSegWarps * 32, 8)
unpermute_kernel(const Pack<T, N>* y, const int* inv, const float* w, long long nrows, int k, int nvec, Segments segs,
                 Pack<T, N>* __restrict__ out, WsHeader* hdr) {
  constexpr int kU = lane_vecs<Pack<T, N>>(), kSeg = 32 * kU;
  chain_go();
  chain_wait();
  const int lane = threadIdx.x & 31;
  int t, s;
  if (!segment_at(segs, &t, &s)) return;
  const long long p0 = (long long)t * k;
  int c[kU];  // lanes behind the row's end read its last vector again
  float acc[kU][N];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    c[u] = min(s * kSeg + 32 * u + lane, nvec - 1);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[u][i] = 0.f;
  }
  for (int j0 = 0; j0 < k; j0 += 32) {
    const bool has = j0 + lane < k;
    const int mine = has ? pair_row(inv, p0 + j0 + lane, nrows, hdr) : -1;
    float wm = 1.f;
    if (kWeighted && has) wm = w[p0 + j0 + lane];
    const int n = min(32, k - j0);
    int j = 0;
    constexpr int kB = kU == 1 ? 5 : kU == 4 ? 3 : 2;  // as the registers of 32 warps per SM allow
    for (; j + kB <= n; j += kB) add_rows<T, N, kU, kB, kWeighted>(y, mine, wm, j, nvec, c, acc);
    for (; j + 2 <= n; j += 2) add_rows<T, N, kU, 2, kWeighted>(y, mine, wm, j, nvec, c, acc);
    if (j < n) add_rows<T, N, kU, 1, kWeighted>(y, mine, wm, j, nvec, c, acc);
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    Pack<T, N> o;
    o.set(acc[u]);
    if (s * kSeg + 32 * u + lane < nvec) out[(size_t)t * nvec + c[u]] = o;
  }
}

// One pair per kPW warps: dy = w dout is written while <dout, y> is summed,
// so y, dout and dy are each touched once per pair (dout comes from L1 or L2
// for all but a token's first pair).
template <typename T, int N, int kPW>
__global__ void __launch_bounds__(kWarps * 32)
unpermute_grad_kernel(const Pack<T, N>* dout, const Pack<T, N>* y,
                      const int* inv, const float* w, long long pairs, int k, int nvec,
                      Pack<T, N>* __restrict__ dy, float* __restrict__ dw, WsHeader* hdr) {
  constexpr int kUnroll = kPW > 1 ? 1 : N * sizeof(T) == 16 ? 4 : 8;
  __shared__ float part[kWarps];
  chain_go();
  chain_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long p = (long long)blockIdx.x * (kWarps / kPW) + warp / kPW;
  float sum = 0.f;
  if (p < pairs) {
    const int r = pair_row(inv, p, pairs, hdr);
    if (r >= 0) {
      const float wp = w[p];
      const Pack<T, N>* d = dout + (size_t)(p / k) * nvec;
      const Pack<T, N>* yr = y + (size_t)r * nvec;
      Pack<T, N>* o = dy + (size_t)r * nvec;
      for (int c0 = (warp % kPW) * 32 * kUnroll; c0 < nvec; c0 += kPW * 32 * kUnroll) {
        Pack<T, N> a[kUnroll], b[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int c = c0 + u * 32 + lane;
          if (c < nvec) {
            b[u] = yr[c];
            a[u] = d[c];
          }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int c = c0 + u * 32 + lane;
          if (c < nvec) {
            float x[N], z[N];
            a[u].get(x);
            b[u].get(z);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              sum = fmaf(x[i], z[i], sum);
              x[i] *= wp;
            }
            Pack<T, N> g;
            g.set(x);
            o[c] = g;
          }
        }
      }
    }
  }
  sum = warp_sum(sum);
  if (kPW == 1) {
    if (lane == 0 && p < pairs) dw[p] = sum;
  } else {
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0 && p < pairs) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) s += part[i];
      dw[p] = s;
    }
  }
}

// Largest vector (bytes, at most 16) that the row size and every pointer allow.
int vector_bytes(size_t row_bytes, const void* a, const void* b, const void* c, const void* d) {
  const uintptr_t all = uintptr_t(row_bytes) | reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |
                        reinterpret_cast<uintptr_t>(c) | reinterpret_cast<uintptr_t>(d);
  return int(all & 15 ? all & (~all + 1) & 15 : 16);
}

template <typename V>
cudaError_t run_permute(const void* x, const int* inv, int T, int k, size_t row_bytes, void* xp, WsHeader* hdr,
                        cudaStream_t st) {
  const int nvec = int(row_bytes / sizeof(V));
  const Segments s = row_segments(T, nvec, 32 * lane_vecs<V>(), true);
  return launch_chained(permute_kernel<V>, dim3(s.blocks()), kSegWarps * 32, 0, st, static_cast<const V*>(x), inv,
                        (long long)T * k, k, nvec, s, static_cast<V*>(xp), hdr);
}

template <typename T, int N>
cudaError_t run_unpermute(const void* y, const int* inv, const float* w, int tokens, int k, int H, void* out,
                          WsHeader* hdr, cudaStream_t st) {
  using V = Pack<T, N>;
  const int nvec = H / N;
  const Segments s = row_segments(tokens, nvec, 32 * lane_vecs<V>(), false);
  return launch_chained(w ? unpermute_kernel<T, N, true> : unpermute_kernel<T, N, false>, dim3(s.blocks()), kSegWarps * 32,
                        0, st, static_cast<const V*>(y), inv, w, (long long)tokens * k, k, nvec, s,
                        static_cast<V*>(out), hdr);
}

template <typename T, int N>
cudaError_t run_unpermute_grad(const void* dout, const void* y, const int* inv, const float* w, int tokens, int k,
                               int H, void* dy, float* dw, WsHeader* hdr, cudaStream_t st) {
  using V = Pack<T, N>;
  const long long pairs = (long long)tokens * k;
  // few pairs (fewer than eight blocks per SM of eight): a block per pair, so
  // that a row is read by eight warps at once
  const bool few = pairs < 1184;
  return launch_chained(few ? unpermute_grad_kernel<T, N, kWarps> : unpermute_grad_kernel<T, N, 1>,
                        dim3(unsigned(few ? pairs : (pairs + kWarps - 1) / kWarps)), kWarps * 32, 0, st,
                        static_cast<const V*>(dout), static_cast<const V*>(y), inv, w, pairs, k, H / N,
                        static_cast<V*>(dy), dw, hdr);
}

// f<T, N> for the element type and the vector width that fits.
#define MOE_DISPATCH_VEC(F, dtype, vb, ...)                                            \
  do {                                                                                 \
    if ((dtype) == MOE_DT_FP32) {                                                      \
      if ((vb) == 16) return F<float, 4>(__VA_ARGS__);                                 \
      if ((vb) == 8) return F<float, 2>(__VA_ARGS__);                                  \
      return F<float, 1>(__VA_ARGS__);                                                 \
    }                                                                                  \
    if ((dtype) == MOE_DT_BF16) {                                                      \
      if ((vb) == 16) return F<__nv_bfloat16, 8>(__VA_ARGS__);                         \
      if ((vb) >= 4) return F<__nv_bfloat16, 2>(__VA_ARGS__);                          \
      return F<__nv_bfloat16, 1>(__VA_ARGS__);                                         \
    }                                                                                  \
    if ((vb) == 16) return F<__half, 8>(__VA_ARGS__);                                  \
    if ((vb) >= 4) return F<__half, 2>(__VA_ARGS__);                                   \
    return F<__half, 1>(__VA_ARGS__);                                                  \
  } while (0)

cudaError_t launch_permute(const void* x, int size, int T, int H, int k, const int* inv, void* xp, WsHeader* hdr,
                           cudaStream_t st) {
  const size_t row = size_t(H) * size;
  switch (vector_bytes(row, x, xp, nullptr, nullptr)) {
    case 16: return run_permute<uint4>(x, inv, T, k, row, xp, hdr, st);
    case 8: return run_permute<uint2>(x, inv, T, k, row, xp, hdr, st);
    case 4: return run_permute<uint32_t>(x, inv, T, k, row, xp, hdr, st);
    case 2: return run_permute<uint16_t>(x, inv, T, k, row, xp, hdr, st);
    default: return run_permute<uint8_t>(x, inv, T, k, row, xp, hdr, st);
  }
}

cudaError_t launch_unpermute(const void* y, int dtype, int T, int H, int k, const int* inv, const float* w, void* out,
                             WsHeader* hdr, cudaStream_t st) {
  const int vb = vector_bytes(size_t(H) * dtype_size(dtype), y, out, nullptr, nullptr);
  MOE_DISPATCH_VEC(run_unpermute, dtype, vb, y, inv, w, T, k, H, out, hdr, st);
}

cudaError_t launch_unpermute_grad(const void* dout, const void* y, int dtype, int T, int H, int k, const int* inv,
                                  const float* w, void* dy, float* dw, WsHeader* hdr, cudaStream_t st) {
  const int vb = vector_bytes(size_t(H) * dtype_size(dtype), dout, y, dy, nullptr);
  MOE_DISPATCH_VEC(run_unpermute_grad, dtype, vb, dout, y, inv, w, T, k, H, dy, dw, hdr, st);
}

// Shapes of the row operators: the pair index in 32 bits, and at most 2^38 bytes
// of rows, which keeps the blocks within a grid (a row of several segments has
// less than four for every 192 bytes, a block four).
bool rows_shape_ok(int64_t T, int64_t H, int64_t k, int32_t dtype) {
  return T >= 0 && H >= 1 && H <= (1 << 24) && k >= 1 && k <= kMaxK && T * k <= 0x7fffffffLL &&
         T * k * dtype_size(dtype) <= (1LL << 38) / H;
}

moe_status rows_check(const void* a, const void* b, int32_t dtype, bool bytes_ok, const void* inv, void* ws,
                      size_t ws_bytes) {
  const int size = dtype_size(dtype);
  if (size == 0 || (size == 1 && !bytes_ok)) return MOE_ERR_UNSUPPORTED;
  if (!a || !b || !inv || !ptr_aligned(a, size) || !ptr_aligned(b, size) || !ptr_aligned(inv, 4))
    return MOE_ERR_INVALID_ARG;
  return status_ws_check(ws, ws_bytes);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_permute(const void* x, int32_t dtype, int32_t T, int32_t H, int32_t k, const int32_t* inv_perm,
                       void* x_perm, void* ws, size_t ws_bytes, void* stream) {
  const CallRange range("moe_permute");
  if (!rows_shape_ok(T, H, k, dtype)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const moe_status s = rows_check(x, x_perm, dtype, true, inv_perm, ws, ws_bytes);
  if (s != MOE_OK) return s;
  return launched(launch_permute(x, dtype_size(dtype), T, H, k, inv_perm, x_perm, ws_at<WsHeader>(ws, 0),
                                 static_cast<cudaStream_t>(stream)));
}

moe_status moe_permute_grad(const void* dx_perm, int32_t dtype, int32_t T, int32_t H, int32_t k,
                            const int32_t* inv_perm, void* dx, void* ws, size_t ws_bytes, void* stream) {
  const CallRange range("moe_permute_grad");
  if (!rows_shape_ok(T, H, k, dtype)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const moe_status s = rows_check(dx_perm, dx, dtype, false, inv_perm, ws, ws_bytes);
  if (s != MOE_OK) return s;
  return launched(launch_unpermute(dx_perm, dtype, T, H, k, inv_perm, nullptr, dx, ws_at<WsHeader>(ws, 0),
                                   static_cast<cudaStream_t>(stream)));
}

moe_status moe_unpermute(const void* y_perm, int32_t dtype, int32_t T, int32_t H, int32_t k, const int32_t* inv_perm,
                         const float* topk_w, void* out, void* ws, size_t ws_bytes, void* stream) {
  const CallRange range("moe_unpermute");
  if (!rows_shape_ok(T, H, k, dtype)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const moe_status s = rows_check(y_perm, out, dtype, false, inv_perm, ws, ws_bytes);
  if (s != MOE_OK) return s;
  if (!topk_w || !ptr_aligned(topk_w, 4)) return MOE_ERR_INVALID_ARG;
  return launched(launch_unpermute(y_perm, dtype, T, H, k, inv_perm, topk_w, out, ws_at<WsHeader>(ws, 0),
                                   static_cast<cudaStream_t>(stream)));
}

moe_status moe_unpermute_grad(const void* dout, const void* y_perm, int32_t dtype, int32_t T, int32_t H, int32_t k,
                              const int32_t* inv_perm, const float* topk_w, void* dy_perm, float* dtopk_w, void* ws,
                              size_t ws_bytes, void* stream) {
  const CallRange range("moe_unpermute_grad");
  if (!rows_shape_ok(T, H, k, dtype)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  moe_status s = rows_check(dout, dy_perm, dtype, false, inv_perm, ws, ws_bytes);
  if (s != MOE_OK) return s;
  if (!y_perm || !ptr_aligned(y_perm, dtype_size(dtype)) || !topk_w || !ptr_aligned(topk_w, 4) || !dtopk_w ||
      !ptr_aligned(dtopk_w, 4))
    return MOE_ERR_INVALID_ARG;
  return launched(launch_unpermute_grad(dout, y_perm, dtype, T, H, k, inv_perm, topk_w, dy_perm, dtopk_w,
                                        ws_at<WsHeader>(ws, 0), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
