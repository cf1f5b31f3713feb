// Grouped product of microscaled fp4 matrices on the fp4 tensor cores:
//   y[r, n] = ga gb[e] sum_k a[r, k] w[e, n, k]     for rows r of expert e.
//
// The weights are the M side of tcgen05.mma (128 rows per tile), the tokens
// its N side, so that an expert with a handful of rows costs a narrow MMA
// (N = 16) and never a padded 128-row tile. Block scales are applied inside
// the MMA (kind::mxf4 for MX, kind::mxf4nvf4 for NV); products are exact and
// sums stay in fp32 in TMEM until the one rounding of the epilogue.
//
// One persistent CTA per SM, 12 warps:
//   warp 0      codes: TMA tiles of 128 bytes (256 elements of K) per row,
//               128-byte swizzle, kStages deep
//   warp 1      MMA issuer (one thread): scale words smem -> TMEM
//               (tcgen05.cp), then four K = 64 MMAs per stage
//   warps 4-7   epilogue: TMEM -> registers -> smem (transposed) -> global,
//               on the other of two accumulators
//   warps 8-11  scales: 4-byte asynchronous copies that place each row's
//               scale words in the blocked order tcgen05.cp wants
// The scales come row-major, 4 bytes per row and K step apart by the row
// stride, so no tiled copy can block them; per-thread copies can, and can mask
// the bytes behind K.
//
// Tiles: every CTA sums up the experts' token tiles (offsets are on the
// device) in shared memory and takes tiles b, b + grid, ... of the list
// "expert, token tile, 128 weight rows": neighbours share the tokens, and an
// expert's weights are read from HBM once, later token tiles hit L2.
#include <cuda.h>

#include <atomic>

#include "call_range.h"
#include "mxfp.cuh"
#include "op_util.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

constexpr int kBM = 128;       // weight rows per tile
constexpr int kBKBytes = 128;  // code bytes of a row per stage: 256 elements
constexpr int kBoxRows = 32;   // token rows per TMA box
constexpr int kThreads = 384;
constexpr int kEpiWarps = 4, kScaleWarps = 4;
constexpr int kScratch = 2048;  // epilogue staging per warp: 16 tokens x 32 rows x 4 bytes

// kTN: tokens per tile (a multiple of 32); kStages: ring depth.
template <bool kNv, int kTN, int kStages_>
struct Cfg {
  static constexpr int kStages = kStages_;
  static constexpr int kWords = kNv ? 4 : 2;            // scale words per row and stage
  static constexpr int kHalves = (kTN + 127) / 128;     // 128-row scale blocks of the token side
  static constexpr int kABytes = kBM * kBKBytes;
  static constexpr int kBBytes = kTN * kBKBytes;
  static constexpr int kSfA = kABytes + kBBytes;        // offsets inside a stage
  static constexpr int kSfB = kSfA + kWords * 512;
  static constexpr int kStageBytes = (kSfB + kWords * kHalves * 512 + 1023) / 1024 * 1024;
  static constexpr int kSfCols = kWords * 4 * (1 + kHalves);
  // TMEM: two accumulators of kTN columns, then the scale words of kSfBufs stages
  static constexpr int kSfBufs = (512 - 2 * kTN) / kSfCols >= 4 ? 4 : 2;
  static constexpr int kCols = 2 * kTN + kSfBufs * kSfCols;
  static constexpr int kTmemCols = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512, "TMEM");
  static_assert(kStages > kSfBufs / 2 && kStages >= 3, "the scale loader runs kStages / 2 stages ahead");
  static constexpr int kSmem = kStages * kStageBytes + kEpiWarps * kScratch + 1024;
};

struct Args {
  const uint8_t* a_scales;
  const uint8_t* b_scales;
  const float* a_tscale;   // [1] or null
  const float* b_tscale;   // [E] or null
  const int* offsets;      // [E + 1] or null (one group of R rows)
  void* out;
  WsHeader* hdr;
  int R, K, N, E;
  int vec_store;           // rows of out are 16-byte aligned
};

struct Tile {
  int e, m0, row0, rows;
};

// Token tiles of an expert with `rows` rows.
__device__ __forceinline__ int token_tiles(int rows, int tn) { return (rows + tn - 1) / tn; }

template <bool kNv, int kTN, int kStages_, typename OT>
__global__ void __launch_bounds__(kThreads, 1)
fp4_gemm_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap tmap, Args a) {
  using C = Cfg<kNv, kTN, kStages_>;
  constexpr int kStages = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[kStages], scale_bar[kStages], empty_bar[kStages], accf_bar[2], acce_bar[2],
      drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ int off_sh[kMaxE + 1];    // first row of each expert
  __shared__ int first_sh[kMaxE + 1];  // first token tile of each expert
  __shared__ int wsum_sh[kThreads / 32];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_p = &abort_sh;

  if (threadIdx.x == 0) {
    ptx::tma_prefetch_map(&wmap);
    ptx::tma_prefetch_map(&tmap);
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(ptx::smem_addr(&full_bar[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&scale_bar[s]), kScaleWarps);
      ptx::mbar_init(ptx::smem_addr(&empty_bar[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_addr(&accf_bar[b]), 1);
      ptx::mbar_init(ptx::smem_addr(&acce_bar[b]), kEpiWarps);
    }
    ptx::mbar_init(ptx::smem_addr(&drain_bar), 1);
    abort_sh = 0;
    ptx::mbar_init_fence();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(&tmem_base_sh), C::kTmemCols);
    ptx::tmem_relinquish();
  }
  // ---- the tile list: offsets, then the running sum of token tiles
  for (int e = threadIdx.x; e <= a.E; e += kThreads) off_sh[e] = a.offsets ? a.offsets[e] : (e ? a.R : 0);
  __syncthreads();
  bool ok = true;
  {
    constexpr int kPer = (kMaxE + kThreads - 1) / kThreads;
    int cnt[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = threadIdx.x * kPer + i;
      cnt[i] = 0;
      if (e < a.E) {
        const int lo = off_sh[e], hi = off_sh[e + 1];
        if (lo < 0 || hi < lo || hi > a.R)
          ok = false;
        else
          cnt[i] = token_tiles(hi - lo, kTN);
      }
      sum += cnt[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) wsum_sh[warp] = incl;
    ok = !__syncthreads_or(!ok);
    int base = incl - sum;
    for (int w = 0; w < warp; ++w) base += wsum_sh[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = threadIdx.x * kPer + i;
      if (e <= a.E) first_sh[e] = base;
      base += cnt[i];
    }
  }
  if (!ok && threadIdx.x == 0) flag_error(a.hdr, MOE_ERR_DEVICE_FAULT, -1);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const int MT = (a.N + kBM - 1) / kBM;
  const int KB = (a.K + 2 * kBKBytes - 1) / (2 * kBKBytes);
  const long long ntiles = ok ? (long long)first_sh[a.E] * MT : 0;

  auto tile_at = [&](long long t) {
    Tile r;
    const int tt = int(t / MT);
    r.m0 = int(t - (long long)tt * MT) * kBM;
    int lo = 0, hi = a.E;  // the last expert whose first tile is <= tt
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_sh[mid] <= tt)
        lo = mid;
      else
        hi = mid;
    }
    r.e = lo;
    const int rows = off_sh[lo + 1] - off_sh[lo], nt = first_sh[lo + 1] - first_sh[lo], i = tt - first_sh[lo];
    // tiles of one size, a multiple of 16 (at most kTN, so none is empty)
    const int per = ((rows + nt - 1) / nt + 15) & ~15;
    r.row0 = off_sh[lo] + i * per;
    r.rows = min(per, rows - i * per);
    return r;
  };
  auto fail = [&](int where) {
    flag_error(a.hdr, MOE_ERR_TIMEOUT, where);
    *abort_p = 1;
  };
  // For roles that run as whole warps: the lanes agree, so that none leaves a
  // loop alone when a wait gives up.
  auto all_ok = [&](bool good) { return __all_sync(0xffffffffu, good) != 0; };
  auto stage = [&](int s) { return ptx::smem_addr(smem) + uint32_t(s) * C::kStageBytes; };

  if (warp == 0) {
    // ------------------------------------------------ codes
    if (lane == 0) {
      int s = 0, issued = 0;
      uint32_t ph = 0;
      for (long long t = blockIdx.x; t < ntiles && !*abort_p; t += gridDim.x) {
        const Tile ti = tile_at(t);
        const int boxes = (ti.rows + kBoxRows - 1) / kBoxRows;
        const uint32_t bytes = uint32_t(C::kABytes + boxes * kBoxRows * kBKBytes);
        for (int kb = 0; kb < KB; ++kb) {
          if (!ptx::mbar_wait(ptx::smem_addr(&empty_bar[s]), ph ^ 1u, abort_p)) {
            fail(7000001);
            break;
          }
          const uint32_t bar = ptx::smem_addr(&full_bar[s]), dst = stage(s);
          ptx::mbar_arrive_expect_tx(bar, bytes);
          ptx::tma_load_3d(dst, &wmap, kb * kBKBytes, ti.m0, ti.e, bar);
          for (int b = 0; b < boxes; ++b)
            ptx::tma_load_2d(dst + C::kABytes + b * kBoxRows * kBKBytes, &tmap, kb * kBKBytes, ti.row0 + b * kBoxRows,
                             bar);
          issued = min(issued + 1, kStages);
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // no copy may be in flight when the CTA leaves
      for (int i = 0; i < issued; ++i) {
        if (--s < 0) {
          s = kStages - 1;
          ph ^= 1u;
        }
        ptx::mbar_wait(ptx::smem_addr(&full_bar[s]), ph, nullptr);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0) {
      int s = 0, it = 0;
      uint32_t ph = 0;
      long long n = 0;  // stages consumed
      const uint32_t sf_base = tmem + 2 * kTN;
      for (long long t = blockIdx.x; t < ntiles && !*abort_p; t += gridDim.x, ++it) {
        const Tile ti = tile_at(t);
        const int N = (ti.rows + 15) & ~15;
        const int halves = N > 128 ? 2 : 1;
        const int buf = it & 1;
        if (!ptx::mbar_wait(ptx::smem_addr(&acce_bar[buf]), (uint32_t(it >> 1) & 1u) ^ 1u, abort_p)) {
          fail(7000002);
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d = tmem + uint32_t(buf * kTN);
        bool good = true;
        for (int kb = 0; kb < KB; ++kb, ++n) {
          // the MMAs that read this scale buffer last are done: their stage was given back
          if (n >= C::kSfBufs) {
            const long long old = n - C::kSfBufs;
            good = ptx::mbar_wait(ptx::smem_addr(&empty_bar[old % kStages]), uint32_t(old / kStages) & 1u, abort_p);
          }
          good = good && ptx::mbar_wait(ptx::smem_addr(&scale_bar[s]), ph, abort_p) &&
                 ptx::mbar_wait(ptx::smem_addr(&full_bar[s]), ph, abort_p);
          if (!good) {
            fail(7000003);
            break;
          }
          ptx::tc_fence_after();
          const uint32_t base = stage(s);
          const uint32_t sfa = sf_base + uint32_t(n % C::kSfBufs) * C::kSfCols, sfb = sfa + 4 * C::kWords;
#pragma unroll
          for (int w = 0; w < C::kWords; ++w) {
            ptx::tmem_cp_32x128(sfa + 4 * w, ptx::smem_desc_rows16(base + C::kSfA + w * 512));
            for (int h = 0; h < halves; ++h)
              ptx::tmem_cp_32x128(sfb + 4 * (w * C::kHalves + h),
                                  ptx::smem_desc_rows16(base + C::kSfB + (w * C::kHalves + h) * 512));
          }
          const int steps = min(4, (a.K - kb * 2 * kBKBytes + 63) / 64);
          for (int ks = 0; ks < steps; ++ks) {
            const int w = kNv ? ks : ks >> 1, sf = kNv ? 0 : 2 * (ks & 1);
            ptx::mma_fp4<kNv>(d, ptx::smem_desc_k128(base + 32 * ks),
                              ptx::smem_desc_k128(base + C::kABytes + 32 * ks), ptx::idesc_fp4<kNv>(kBM, N, sf),
                              sfa + 4 * w, sfb + 4 * w * C::kHalves, (kb | ks) != 0);
          }
          ptx::mma_commit(ptx::smem_addr(&empty_bar[s]));
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!good) break;
        ptx::mma_commit(ptx::smem_addr(&accf_bar[buf]));
      }
      ptx::mma_commit(ptx::smem_addr(&drain_bar));
      ptx::mbar_wait(ptx::smem_addr(&drain_bar), 0, nullptr);
    }
  } else if (warp >= 8) {
    // ------------------------------------------------ scales
    constexpr int kAhead = kStages / 2;  // copies of this many stages are in flight per thread
    constexpr int kRowsPer = 32 * kScaleWarps / C::kWords;
    const int tid = threadIdx.x - 256;
    const int word = tid % C::kWords, r0 = tid / C::kWords;
    const int stride = scale_stride(kNv, a.K), blocks = a.K / (kNv ? 16 : 32);
    int s = 0, pending = 0, sd = 0;  // stage to fill, stages in flight, next stage to hand over
    uint32_t ph = 0;
    auto hand_over = [&]() {
      ptx::fence_proxy_async_smem();  // written by this thread, read by the tensor core's copies
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&scale_bar[sd]));
      sd = sd + 1 == kStages ? 0 : sd + 1;
      --pending;
    };
    for (long long t = blockIdx.x; t < ntiles && all_ok(!*abort_p); t += gridDim.x) {
      const Tile ti = tile_at(t);
      const uint8_t* wsrc = a.b_scales + ((size_t)ti.e * a.N + ti.m0) * stride;
      const uint8_t* tsrc = a.a_scales + (size_t)ti.row0 * stride;
      const int wrows = min(kBM, a.N - ti.m0);
      const int tpad = (ti.rows + 15) & ~15;
      for (int kb = 0; kb < KB; ++kb) {
        if (!all_ok(ptx::mbar_wait(ptx::smem_addr(&empty_bar[s]), ph ^ 1u, abort_p))) {
          fail(7000004);
          break;
        }
        const int at = (kb * C::kWords + word) * 4;
        const uint32_t left = uint32_t(max(0, min(4, blocks - at)));  // bytes of this word inside K
        const uint32_t dst = stage(s) + C::kSfA + word * 512;
#pragma unroll
        for (int r = r0; r < kBM; r += kRowsPer) {
          const uint32_t valid = r < wrows ? left : 0;
          ptx::cp_async4(dst + (r & 31) * 16 + (r >> 5) * 4, valid ? wsrc + (size_t)r * stride + at : wsrc, valid);
        }
        const uint32_t dstb = stage(s) + C::kSfB + word * C::kHalves * 512;
        for (int r = r0; r < tpad; r += kRowsPer) {
          const uint32_t valid = r < ti.rows ? left : 0;
          ptx::cp_async4(dstb + (r >> 7) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4,
                         valid ? tsrc + (size_t)r * stride + at : tsrc, valid);
        }
        ptx::cp_async_commit();
        if (++pending > kAhead) {
          ptx::cp_async_wait<kAhead>();
          hand_over();
        }
        if (++s == kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    ptx::cp_async_wait<0>();
    while (pending > 0) hand_over();
  } else if (warp >= 4) {
    // ------------------------------------------------ epilogue
    const int q = warp & 3;  // TMEM lane quarter this warp may read
    uint8_t* scratch = smem + kStages * C::kStageBytes + q * kScratch;
    OT* out = static_cast<OT*>(a.out);
    const float ga = a.a_tscale ? *a.a_tscale : 1.f;
    constexpr int kPieces = 2 * sizeof(OT);  // 16-byte pieces of a token's 32 values
    constexpr int kPerPiece = 16 / sizeof(OT);
    int it = 0;
    for (long long t = blockIdx.x; t < ntiles && all_ok(!*abort_p); t += gridDim.x, ++it) {
      const Tile ti = tile_at(t);
      const float alpha = a.b_tscale ? ga * a.b_tscale[ti.e] : ga;
      const int buf = it & 1;
      const int n0 = ti.m0 + 32 * q;
      if (!all_ok(ptx::mbar_wait_sleep(ptx::smem_addr(&accf_bar[buf]), uint32_t(it >> 1) & 1u, abort_p, 32))) {
        fail(7000005);
        break;
      }
      ptx::tc_fence_after();
      const uint32_t taddr = tmem + (uint32_t(32 * q) << 16) + uint32_t(buf * kTN);
      for (int c0 = 0; c0 < ti.rows; c0 += 16) {
        uint32_t v[16];
        ptx::tmem_ld16(taddr + uint32_t(c0), v);
        ptx::tmem_ld_wait();
        if (a.vec_store) {
          OT* sc = reinterpret_cast<OT*>(scratch);
#pragma unroll
          for (int i = 0; i < 16; ++i) sc[i * 32 + lane] = from_f32<OT>(__uint_as_float(v[i]) * alpha);
          __syncwarp();
#pragma unroll
          for (int p = lane; p < 16 * kPieces; p += 32) {
            const int tok = p / kPieces, n = n0 + p % kPieces * kPerPiece;
            if (c0 + tok < ti.rows && n < a.N)
              *reinterpret_cast<uint4*>(out + (size_t)(ti.row0 + c0 + tok) * a.N + n) =
                  *reinterpret_cast<const uint4*>(scratch + p * 16);
          }
          __syncwarp();
        } else if (n0 + lane < a.N) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c0 + i < ti.rows)
              out[(size_t)(ti.row0 + c0 + i) * a.N + n0 + lane] = from_f32<OT>(__uint_as_float(v[i]) * alpha);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&acce_bar[buf]));
    }
  }
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// cuTensorMapEncodeTiled through the runtime's entry-point table, so the
// library loads on machines without a driver.
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encoder() {
  static std::atomic<EncodeFn> fn{nullptr};
  EncodeFn f = fn.load(std::memory_order_acquire);
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q{};
  if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<EncodeFn>(p);
  fn.store(f, std::memory_order_release);
  return f;
}

// Codes [planes, rows, row_bytes] in boxes of 128 bytes x box_rows.
bool code_map(CUtensorMap* map, const uint8_t* base, uint64_t row_bytes, uint64_t rows, uint64_t planes, int dims,
              uint32_t box_rows) {
  const EncodeFn f = encoder();
  if (!f) return false;
  const cuuint64_t size[3] = {row_bytes, rows, planes};
  const cuuint64_t stride[2] = {row_bytes, row_bytes * rows};
  const cuuint32_t box[3] = {kBKBytes, box_rows, 1}, step[3] = {1, 1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, cuuint32_t(dims), const_cast<uint8_t*>(base), size, stride, box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return n;
}

template <bool kNv, int kTN, int kStages, typename OT>
cudaError_t run(const CUtensorMap& wm, const CUtensorMap& tm, const Args& a, cudaStream_t st) {
  using C = Cfg<kNv, kTN, kStages>;
  auto* kernel = fp4_gemm_kernel<kNv, kTN, kStages, OT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  // at most this many tiles: every group with rows may end in a partial one
  const long long most = ((long long)a.R / kTN + (a.R < a.E ? a.R : a.E) + 1) * ((a.N + kBM - 1) / kBM);
  const int sms = sm_count();
  kernel<<<unsigned(most < sms ? most : sms), kThreads, C::kSmem, st>>>(wm, tm, a);
  count_launches(1);
  return cudaGetLastError();
}

template <bool kNv, typename OT>
cudaError_t run_tiles(const CUtensorMap& wm, const CUtensorMap& tm, const Args& a, cudaStream_t st) {
  // few rows per expert: narrow tiles leave room for a ring twice as deep, and
  // the weights stream through it
  if (a.R <= 32LL * a.E) return run<kNv, 32, 8, OT>(wm, tm, a, st);
  return run<kNv, 192, 4, OT>(wm, tm, a, st);
}

template <bool kNv>
cudaError_t run_out(int32_t dtype, const CUtensorMap& wm, const CUtensorMap& tm, const Args& a, cudaStream_t st) {
  if (dtype == MOE_DT_BF16) return run_tiles<kNv, __nv_bfloat16>(wm, tm, a, st);
  if (dtype == MOE_DT_FP16) return run_tiles<kNv, __half>(wm, tm, a, st);
  return run_tiles<kNv, float>(wm, tm, a, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_mxfp_matmul(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_tensor_scale,
                                      int32_t R, int32_t K, const uint8_t* b_codes, const uint8_t* b_scales,
                                      const float* b_tensor_scale, int32_t E, int32_t N, const int32_t* offsets,
                                      int32_t format, void* out, int32_t out_dtype, void* ws, size_t ws_bytes,
                                      void* stream) {
  const CallRange range("moe_mxfp_matmul");
  if (format != MOE_FP_MX && format != MOE_FP_NV) return MOE_ERR_UNSUPPORTED;
  const int size = dtype_size(out_dtype);
  if (size < 2) return MOE_ERR_UNSUPPORTED;
  // one expert's codes stay below the 2^40 bytes a tensor map can stride over
  if (R < 0 || R > (1 << 30) || E < 1 || E > kMaxE || N < 1 || N > kMaxFpCols || K < 32 || K % 32 || K > kMaxFpCols ||
      (int64_t)N * K >= (1LL << 41))
    return MOE_ERR_INVALID_ARG;
  if (!offsets && E != 1) return MOE_ERR_INVALID_ARG;
  if (format == MOE_FP_MX && (a_tensor_scale || b_tensor_scale)) return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (!a_codes || !a_scales || !b_codes || !b_scales || !out) return MOE_ERR_INVALID_ARG;
  if (!ptr_aligned(a_codes, 16) || !ptr_aligned(a_scales, 16) || !ptr_aligned(b_codes, 16) ||
      !ptr_aligned(b_scales, 16) || !ptr_aligned(out, size) || !ptr_aligned(offsets, 4) ||
      !ptr_aligned(a_tensor_scale, 4) || !ptr_aligned(b_tensor_scale, 4))
    return MOE_ERR_INVALID_ARG;
  const moe_status s = status_ws_check(ws, ws_bytes);
  if (s != MOE_OK) return s;
  CUtensorMap wm, tm;
  if (!code_map(&wm, b_codes, K / 2, N, E, 3, kBM) || !code_map(&tm, a_codes, K / 2, R, 1, 2, kBoxRows))
    return MOE_ERR_CUDA;
  Args a{a_scales, b_scales, a_tensor_scale, b_tensor_scale, offsets, out, ws_at<WsHeader>(ws, 0), R, K, N, E,
         int((size_t(N) * size) % 16 == 0 && ptr_aligned(out, 16))};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = format == MOE_FP_NV ? run_out<true>(out_dtype, wm, tm, a, st)
                                            : run_out<false>(out_dtype, wm, tm, a, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
