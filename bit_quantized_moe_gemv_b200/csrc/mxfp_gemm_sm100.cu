// Grouped product of microscaled fp4 matrices on the fp4 tensor cores:
//   y[r, n] = ga gb[e] sum_k a[r, k] w[e, n, k]     for rows r of expert e.
//
// The weights are the M side of tcgen05.mma (128 rows per tile), the tokens
// its N side, so that an expert with a handful of rows costs a narrow MMA
// (N = 16) and never a padded 128-row tile. Block scales are applied inside
// the MMA (kind::mxf4 for MX, kind::mxf4nvf4 for NV); products are exact and
// sums stay in fp32 in TMEM until the one rounding of the epilogue.
//
// One persistent CTA per SM (two for narrow tiles), 16 warps:
//   warps 0, 3   codes of the weights, of the tokens: TMA tiles of 128 bytes
//                (256 elements of K) per row, 128-byte swizzle, kStages deep
//   warp 1       MMA issuer: the scale words of 16 bytes of each row from
//                shared memory to TMEM (tcgen05.cp, in the MMAs' own queue), then
//                four K = 64 MMAs per stage
//   warp 2       scales: TMA tiles of 32 bytes per row, kSlots deep
//   warps 4-6    scales, in place: row-major 32-byte rows become the blocks
//                tcgen05.cp wants, 4 bytes of each of 128 rows together (the
//                weights' rows, the first and the second 128 tokens); what
//                lies behind K becomes 0
//   warps 8-15   epilogue: TMEM -> registers -> smem (transposed) -> global,
//                on the other of two accumulators
// The scale words could go straight to TMEM from the warps' registers, but
// those stores and the MMAs get in each other's way: 8192^3 MX in 326 us, in
// 295 with tcgen05.cp. One thread that waits, copies and multiplies is the next
// limit, then the threads that issue the TMA copies (about 70 cycles each):
// 251 us now (MX; NV 276; back to back, under the power limit, 292 and 322), of
// which the MMAs alone take 141.
//
// Tiles: every CTA sums up the experts' token tiles (offsets are on the
// device) and takes tiles b, b + grid, ... of the list "token tile, 128 weight
// rows": neighbours share the tokens. Token tiles of experts with several of
// them, bound by L2 and the tensor core, alternate with those of experts with
// one, bound by HBM (8K tokens, 512 experts with Zipf routing: 242 us, 249 in
// the experts' order); each kind keeps the experts' order, so that an expert's
// weights are read from HBM once and its later token tiles hit L2. What a tile
// is (expert, rows) is worked out by all threads at once for the next kListed
// tiles of the CTA: the search and the divisions cost one warp about 900 cycles
// a tile.
//
// Bound: HBM where an expert has up to about 160 rows (512 experts of 160 rows,
// gate and up: 189 us, 98 % of the measured copy rate; of 16 rows: 135 us), the
// operands' way beyond (a stage of 160 tokens brings 36 KB from L2 at 64 bytes a
// cycle and takes 72 KB through shared memory at 128: 576 cycles either way, of
// 670 measured at 8192^3, where its MMAs take 372), the start of a CTA (barriers,
// list, first copies: about 3 us) for a token's ten experts (9.2 us, 2.6 us of
// them HBM time), and the few CTAs at work for few rows of one matrix (32 of them
// for 8 x 4,096 x 4,096: 9.7 us, 1.4 us of HBM time; K is not split).
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
constexpr int kScaleWarps = 3;
constexpr int kSlotRow = 32;   // scale bytes of a row per slot
constexpr int kScratch = 2048;  // epilogue staging per warp: 32 weight rows of 32 (16 bits) or 16 tokens

// kTN: tokens per tile (a multiple of 32); kStages, kSlots: depth of the rings of codes and of scales.
template <int kTN, int kStages, int kSlots>
struct Cfg {
  static constexpr bool kNarrow = kTN <= 32;  // two CTAs per SM
  static constexpr int kEpiWarps = kNarrow ? 4 : 8, kThreads = 32 * (8 + kEpiWarps);
  static constexpr int kListed = kNarrow ? 128 : 256;  // tiles listed at a time
  static constexpr int kHalves = (kTN + 127) / 128;  // 128-row scale blocks of the token side
  static constexpr int kABytes = kBM * kBKBytes;
  static constexpr int kStageBytes = kABytes + kTN * kBKBytes;
  static constexpr int kSlotBytes = 128 * (1 + kHalves) * kSlotRow;
  // TMEM: two accumulators of kTN columns, then buffers of the scale words of
  // 16 bytes of each row: 4 x 4 columns of weights, 4 x kBCols of tokens
  static constexpr int kBCols = 4 * kHalves;
  static constexpr int kSfCols = 4 * (4 + kBCols);
  // as many as code stages: a stage that is full again tells that the MMAs of
  // its last use are done, and with them those on the scale buffer's last use
  static constexpr int kSfBufs = kStages;
  static constexpr int kCols = 2 * kTN + kSfBufs * kSfCols;
  static constexpr int kTmemCols = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512, "TMEM");
  static constexpr int kScaleAt = kStages * kStageBytes;  // offsets in shared memory
  static constexpr int kScratchAt = kScaleAt + kSlots * kSlotBytes;
  static constexpr int kSmem = kScratchAt + kEpiWarps * kScratch + 1024;
};

struct Args {
  const float* a_tscale;   // [1] or null
  const float* b_tscale;   // [E] or null
  const int* offsets;      // [E + 1] or null (one group of R rows)
  void* out;
  WsHeader* hdr;
  int R, K, N, E;
  int vec_store;           // rows of out are 16-byte aligned
  long long wait_cycles;   // budget of every wait of the pipeline
};

// Tensor maps: codes and scales of the weights and of the tokens.
struct Maps {
  CUtensorMap wcodes, tcodes, tall, wscales, tscales;  // tcodes in boxes of kBoxRows rows, tall of a whole tile's
};

struct alignas(16) Tile {
  int e, m0, row0, rows;
};

// ga gb as the product of two factors that are each in the normal range, and
// with which no product on the way to the result leaves it before the result
// does: 2^-180 to 2^180 is more than fp32 holds, while the sums, 2^-20 to 2^47
// in size, take most of it back.
struct Factors {
  float first, second;
};
__device__ __forceinline__ Factors factors(float ga, float gb) {
  const float p = ga * gb;
  if (p >= 0x1p-90f && p <= 0x1p90f) return {p, 1.f};
  int ea, eb;
  const float m = frexpf(ga, &ea) * frexpf(gb, &eb);
  const int half = (ea + eb) / 2;
  return {ldexpf(m, half), ldexpf(1.f, ea + eb - half)};
}

// Token tiles of an expert with `rows` rows.
__device__ __forceinline__ int token_tiles(int rows, int tn) { return (rows + tn - 1) / tn; }

template <bool kNv, int kTN, int kStages, int kSlots, typename OT>
__global__ void __launch_bounds__(Cfg<kTN, kStages, kSlots>::kThreads, Cfg<kTN, kStages, kSlots>::kNarrow ? 2 : 1)
fp4_gemm_kernel(const __grid_constant__ Maps maps, Args a) {
  using C = Cfg<kTN, kStages, kSlots>;
  constexpr int kThreads = C::kThreads, kEpiWarps = C::kEpiWarps;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages];                      // codes
  __shared__ __align__(8) uint64_t sfull_bar[kSlots], sblock_bar[kSlots], sempty_bar[kSlots];  // scales: come, in blocks
  __shared__ __align__(8) uint64_t accf_bar[2], acce_bar[2], drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ uint32_t sent_sh[2];        // stages that the weights' and the tokens' warp have copied (mod 2^32)
  constexpr int kExperts = C::kNarrow ? 1 : kMaxE + 1;
  __shared__ int off_sh[kExperts];       // first row of each expert
  __shared__ int first_sh[2][kExperts];  // its first token tile among experts with one, with several
  __shared__ int wsum_sh[2][kThreads / 32];
  __shared__ int all_sh;                 // token tiles
  __shared__ Tile list_sh[C::kListed];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_p = &abort_sh;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(ptx::smem_addr(&full_bar[s]), 2);
      ptx::mbar_init(ptx::smem_addr(&empty_bar[s]), 1);
    }
    for (int s = 0; s < kSlots; ++s) {
      ptx::mbar_init(ptx::smem_addr(&sfull_bar[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&sblock_bar[s]), kScaleWarps);
      ptx::mbar_init(ptx::smem_addr(&sempty_bar[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_addr(&accf_bar[b]), 1);
      ptx::mbar_init(ptx::smem_addr(&acce_bar[b]), kEpiWarps);
    }
    ptx::mbar_init(ptx::smem_addr(&drain_bar), 1);
    abort_sh = 0;
    sent_sh[0] = sent_sh[1] = 0;
    ptx::mbar_init_fence();
  } else if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(&tmem_base_sh), C::kTmemCols);
    ptx::tmem_relinquish();
  } else if (warp == 2 && lane == 0) {
    ptx::tma_prefetch_map(&maps.wcodes);
    ptx::tma_prefetch_map(&maps.tcodes);
    if (!C::kNarrow) ptx::tma_prefetch_map(&maps.tall);
    ptx::tma_prefetch_map(&maps.wscales);
    ptx::tma_prefetch_map(&maps.tscales);
  }
  chain_wait();
  // ---- the running sum of token tiles
  constexpr int kPer = (kMaxE + kThreads - 1) / kThreads;
  int row_at[kPer + 1];
#pragma unroll
  for (int i = 0; i <= kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    row_at[i] = e > a.E ? 0 : a.offsets ? a.offsets[e] : e ? a.R : 0;
  }
  bool ok = true;
  int cnt[kPer], one = 0, many = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    cnt[i] = 0;
    if (e < a.E) {
      if (row_at[i] < 0 || row_at[i + 1] < row_at[i] || row_at[i + 1] > a.R)
        ok = false;
      else
        cnt[i] = token_tiles(row_at[i + 1] - row_at[i], kTN);
    }
    (!C::kNarrow && cnt[i] > 1 ? many : one) += cnt[i];
  }
  int incl1 = one, incl2 = many;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl1, o), v = __shfl_up_sync(0xffffffffu, incl2, o);
    if (lane >= o) {
      incl1 += u;
      incl2 += v;
    }
  }
  if (lane == 31) {
    wsum_sh[0][warp] = incl1;
    wsum_sh[1][warp] = incl2;
  }
  ok = !__syncthreads_or(!ok);
  int base1 = incl1 - one, base2 = incl2 - many;
  for (int w = 0; w < warp; ++w) {
    base1 += wsum_sh[0][w];
    base2 += wsum_sh[1][w];
  }
  int first_of[kPer];  // first token tiles of this thread's experts
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    first_of[i] = base1;
    if (!C::kNarrow && e < a.E) {
      off_sh[e] = row_at[i];
      first_sh[0][e] = base1;
      first_sh[1][e] = base2;
    }
    (!C::kNarrow && cnt[i] > 1 ? base2 : base1) += cnt[i];
    if (e == a.E - 1) {  // the end behind the last expert
      if (C::kNarrow) {
        all_sh = base1;
      } else {
        off_sh[a.E] = row_at[i + 1];
        first_sh[0][a.E] = base1;
        first_sh[1][a.E] = base2;
      }
    }
  }
  if (!ok && threadIdx.x == 0) flag_error(a.hdr, MOE_ERR_DEVICE_FAULT, -1);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  chain_go();  // every CTA has its TMEM: a successor that waits for some takes none from this grid
  const uint32_t tmem = tmem_base_sh;
  const int MT = (a.N + kBM - 1) / kBM;
  const int KB = (a.K + 2 * kBKBytes - 1) / (2 * kBKBytes);
  const int stride = scale_stride(kNv, a.K);
  const int chunks = stride / 16;  // 16 scale bytes of each row: one TMEM buffer, half a slot
  // token tiles of experts with one (narrow tiles: of all), and with several
  const int ones = C::kNarrow ? all_sh : first_sh[0][a.E], manys = C::kNarrow ? 0 : first_sh[1][a.E];
  const int ntiles = ok ? (ones + manys) * MT : 0;
  const int mine = int(blockIdx.x) < ntiles ? (ntiles - 1 - int(blockIdx.x)) / int(gridDim.x) + 1 : 0;

  // The CTA's tiles [from, from + n) into the list. Few rows: every expert's
  // thread writes its own, which takes the fewest instructions. Else thread i
  // finds the i-th.
  auto write_list = [&](int from, int n) {
    for (int i = 0; i < kPer; ++i) {
      const int rows = row_at[i + 1] - row_at[i], t0 = first_of[i] * MT, t1 = (first_of[i] + cnt[i]) * MT;
      if (cnt[i] == 0) continue;
      // the CTA's first tile from t0 on, as its place in the list
      int at = max(0, int(uint32_t(max(t0 - int(blockIdx.x), 0) + int(gridDim.x) - 1) / gridDim.x) - from);
      for (; at < n; ++at) {
        const int t = int(blockIdx.x) + (from + at) * int(gridDim.x);
        if (t >= t1) break;
        const int tt = int(uint32_t(t - t0) / uint32_t(MT)), row0 = tt * kTN;
        list_sh[at] = Tile{int(threadIdx.x) * kPer + i, (t - t0 - tt * MT) * kBM, row_at[i] + row0, min(kTN, rows - row0)};
      }
    }
  };
  auto tile_at = [&](int t) {
    const int tt = int(uint32_t(t) / uint32_t(MT));
    // of the first tt token tiles, tt * manys / all are of experts with several
    int kind = 0, at = tt;
    if (manys) {
      const int before = int(uint64_t(tt) * uint32_t(manys) / uint32_t(ones + manys));
      kind = int(uint64_t(tt + 1) * uint32_t(manys) / uint32_t(ones + manys)) > before;
      at = kind ? before : tt - before;
    }
    const int* first = first_sh[kind];
    int e = 0, hi = a.E;  // the last expert whose first token tile of this kind is <= at
    while (hi - e > 1) {
      const int mid = (e + hi) >> 1;
      if (first[mid] <= at)
        e = mid;
      else
        hi = mid;
    }
    const int lo = off_sh[e], rows = off_sh[e + 1] - lo, nt = first[e + 1] - first[e], i = at - first[e];
    // token tiles of one size, a multiple of 16 (at most kTN, so none is empty)
    const int per = nt == 1 ? rows : (int(uint32_t(rows + nt - 1) / uint32_t(nt)) + 15) & ~15;
    return Tile{e, (t - tt * MT) * kBM, lo + i * per, min(per, rows - i * per)};
  };
  auto fail = [&](int where) {
    flag_error(a.hdr, MOE_ERR_TIMEOUT, where);
    *abort_p = 1;
  };
  auto wait = [&](uint32_t bar, uint32_t parity) { return ptx::mbar_wait(bar, parity, abort_p, a.wait_cycles); };
  // One lane polls, the warp follows and agrees on the outcome, so that no
  // lane leaves a loop alone when a wait gives up. A vote orders no memory: every
  // lane then looks at the completed phase itself, which is what shows it the data.
  auto follow = [&](bool got, uint32_t bar, uint32_t parity) {
    const bool all = __all_sync(0xffffffffu, got) != 0;
    ptx::mbar_test_wait(bar, parity);
    return all;
  };
  auto warp_wait = [&](uint64_t& bar, uint32_t parity) {
    const uint32_t at = ptx::smem_addr(&bar);
    return follow(lane != 0 || wait(at, parity), at, parity);
  };
  auto warp_wait_sleep = [&](uint64_t& bar, uint32_t parity) {
    const uint32_t at = ptx::smem_addr(&bar);
    return follow(lane != 0 || ptx::mbar_wait_sleep(at, parity, abort_p, 32, a.wait_cycles), at, parity);
  };
  auto stage = [&](int s) { return ptx::smem_addr(smem) + uint32_t(s) * C::kStageBytes; };

  // State that a role carries from one list of tiles to the next: its place in
  // its ring and that place's phase, the same of the scale slots and the TMEM
  // scale buffers, tiles done, copies it may have in flight.
  int s = 0, ss = 0, wb = 0, it = 0, issued = 0;
  uint32_t ph = 0, sph = 0;

  for (int first_tile = 0; first_tile < mine; first_tile += C::kListed) {
    const int n = min(C::kListed, mine - first_tile);
    if (C::kNarrow)
      write_list(first_tile, n);
    else if (int(threadIdx.x) < n)
      list_sh[threadIdx.x] = tile_at(int(blockIdx.x) + (first_tile + int(threadIdx.x)) * int(gridDim.x));
    __syncthreads();
    if ((warp == 0 || warp == 3) && ptx::elect_one()) {
      // ------------------------------------------------ codes: weights, tokens
      // A copy takes its thread about 70 cycles, hence two threads and, for a
      // token tile that is nearly full, one copy.
      bool ready = false;
      sent_sh[warp != 0] = uint32_t(first_tile + n) * uint32_t(KB);
      for (int i = 0; i < n; ++i) {
        const Tile ti = list_sh[i];
        const bool whole = !C::kNarrow && ti.rows > kTN - kBoxRows;
        const int boxes = whole ? 1 : (ti.rows + kBoxRows - 1) / kBoxRows;
        const uint32_t bytes = warp == 0 ? C::kABytes : (whole ? kTN : boxes * kBoxRows) * kBKBytes;
        const CUtensorMap* tmap = whole ? &maps.tall : &maps.tcodes;
        int kb = 0;
        for (; kb < KB; ++kb) {
          if (!ready && !wait(ptx::smem_addr(&empty_bar[s]), ph ^ 1u)) break;
          const uint32_t bar = ptx::smem_addr(&full_bar[s]), dst = stage(s);
          ptx::mbar_arrive_expect_tx(bar, bytes);
          if (warp == 0)
            ptx::tma_load_3d(dst, &maps.wcodes, kb * kBKBytes, ti.m0, ti.e, bar);
          else
            for (int b = 0; b < boxes; ++b)
              ptx::tma_load_2d(dst + C::kABytes + b * kBoxRows * kBKBytes, tmap, kb * kBKBytes, ti.row0 + b * kBoxRows,
                               bar);
          issued = min(issued + 1, kStages);
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
          ready = ptx::mbar_test_wait(ptx::smem_addr(&empty_bar[s]), ph ^ 1u);
        }
        if (kb < KB) {
          sent_sh[warp != 0] = uint32_t(first_tile + i) * uint32_t(KB) + uint32_t(kb);
          fail(7000001);
          break;
        }
      }
    } else if (warp == 1 && ptx::elect_one()) {
      // ------------------------------------------------ MMA issuer
      // One thread feeds the tensor core, and a stage's MMAs take 4 x N / 2
      // cycles: every instruction here counts. Descriptors and TMEM columns
      // are carried along, and the next stage's barrier is looked at while
      // this stage's MMAs are issued.
      const uint32_t sf0 = tmem + 2 * kTN;
      const uint64_t da0 = ptx::smem_desc_k128(stage(0));
      const uint64_t ds0 = ptx::smem_desc_rows16(ptx::smem_addr(smem) + C::kScaleAt);
      const uint32_t full0 = ptx::smem_addr(&full_bar[0]), empty0 = ptx::smem_addr(&empty_bar[0]);
      const int full_stages = a.K / (2 * kBKBytes), tail_steps = (a.K - full_stages * 2 * kBKBytes + 63) / 64;
      uint64_t da = da0 + uint32_t(s * (C::kStageBytes / 16)), ds = ds0 + uint32_t(ss * (C::kSlotBytes / 16));
      uint32_t sf = sf0 + uint32_t(wb * C::kSfCols);
      bool ready = false, sready = false;
      for (int i = 0; i < n; ++i, ++it) {
        const int N = (list_sh[i].rows + 15) & ~15;
        const bool wide = N > 128;
        const uint32_t d = tmem + uint32_t((it & 1) * kTN);
        const uint32_t idesc = ptx::idesc_fp4<kNv>(kBM, N, 0), idesc2 = ptx::idesc_fp4<kNv>(kBM, N, kNv ? 0 : 2);
        uint32_t acc = 0;
        // One stage: descriptors count in 16 bytes. `second`: MX, the other
        // half of the scale words that the stage before copied.
        auto step = [&](bool second, uint64_t dsc, int steps) {
          if (!ready && !wait(full0 + 8 * s, ph)) return false;
          ptx::tc_fence_after();
          if (!second) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              ptx::tmem_cp_32x128(sf + 4 * w, dsc + 32 * w);
              ptx::tmem_cp_32x128(sf + 16 + C::kBCols * w, dsc + 256 + 32 * w);
              if (C::kHalves == 2 && wide) ptx::tmem_cp_32x128(sf + 16 + C::kBCols * w + 4, dsc + 512 + 32 * w);
            }
          }
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint32_t w = (second ? 2 : 0) + (kNv ? ks : ks >> 1);
            if (ks < steps)
              ptx::mma_fp4<kNv>(d, da + 2 * ks, da + C::kABytes / 16 + 2 * ks, ks & 1 ? idesc2 : idesc, sf + 4 * w,
                                sf + 16 + C::kBCols * w, acc);
            acc = 1;
          }
          ptx::mma_commit(empty0 + 8 * s);
          da += C::kStageBytes / 16;
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
            da = da0;
          }
          ready = ptx::mbar_test_wait(full0 + 8 * s, ph);
          return true;
        };
        auto next_buffer = [&]() {  // of the scale words in TMEM
          sf += C::kSfCols;
          if (++wb == C::kSfBufs) {
            wb = 0;
            sf = sf0;
          }
        };
        auto next_slot = [&]() {
          ptx::mma_commit(ptx::smem_addr(&sempty_bar[ss]));
          ds += C::kSlotBytes / 16;
          if (++ss == kSlots) {
            ss = 0;
            sph ^= 1u;
            ds = ds0;
          }
          sready = ptx::mbar_test_wait(ptx::smem_addr(&sblock_bar[ss]), sph);
        };
        auto slot_ready = [&]() { return sready || wait(ptx::smem_addr(&sblock_bar[ss]), sph); };
        bool good = wait(ptx::smem_addr(&acce_bar[it & 1]), (uint32_t(it >> 1) & 1u) ^ 1u);
        constexpr int kPerSlot = kNv ? 2 : 4;  // stages whose scales a slot holds
        int kb = 0;
        for (; good && kb + kPerSlot <= full_stages; kb += kPerSlot) {
          good = slot_ready();
          if (kNv) {
            good = good && step(false, ds, 4);
            next_buffer();
            good = good && step(false, ds + 128, 4);
          } else {
            good = good && step(false, ds, 4) && step(true, ds, 4);
            next_buffer();
            good = good && step(false, ds + 128, 4) && step(true, ds + 128, 4);
          }
          if (!good) break;  // a slot that was not waited for is not given back
          next_buffer();
          next_slot();
        }
        if (kb < KB && good) {  // the slot that K ends in
          const int kb0 = kb;
          good = slot_ready();
          for (; kb < KB && good; ++kb) {
            const int j = kb - kb0;
            const bool second = !kNv && (j & 1);
            good = step(second, ds + ((kNv ? j : j >> 1) & 1) * 128, kb < full_stages ? 4 : tail_steps);
            if (kNv || second || kb + 1 == KB) next_buffer();
          }
          if (good) next_slot();
        }
        if (!good) {
          fail(7000002);
          break;
        }
        ptx::mma_commit(ptx::smem_addr(&accf_bar[it & 1]));
      }
    } else if (warp == 2 && ptx::elect_one()) {
      // ------------------------------------------------ scales to shared memory
      for (int i = 0; i < n; ++i) {
        const Tile ti = list_sh[i];
        const int boxes = (ti.rows + kBoxRows - 1) / kBoxRows;
        const uint32_t bytes = uint32_t((kBM + boxes * kBoxRows) * kSlotRow);
        int x = 0;
        for (; x < stride; x += kSlotRow) {
          if (!wait(ptx::smem_addr(&sempty_bar[ss]), sph ^ 1u)) break;
          const uint32_t bar = ptx::smem_addr(&sfull_bar[ss]);
          const uint32_t dst = ptx::smem_addr(smem) + C::kScaleAt + ss * C::kSlotBytes;
          ptx::mbar_arrive_expect_tx(bar, bytes);
          ptx::tma_load_3d(dst, &maps.wscales, x, ti.m0, ti.e, bar);
          for (int b = 0; b < boxes; ++b)
            ptx::tma_load_2d(dst + (kBM + b * kBoxRows) * kSlotRow, &maps.tscales, x, ti.row0 + b * kBoxRows, bar);
          issued = min(issued + 1, kSlots);
          if (++ss == kSlots) {
            ss = 0;
            sph ^= 1u;
          }
        }
        if (x < stride) {
          fail(7000003);
          break;
        }
      }
    } else if (warp >= 4 && warp < 4 + kScaleWarps) {
      // ------------------------------------------------ scales into blocks
      const int blocks = a.K / (kNv ? 16 : 32);
      const int unit = warp - 4;  // weights, first 128 tokens, second 128 tokens
      bool good = true;
      for (int i = 0; i < n && good; ++i) {
        const int rows = unit == 0 ? kBM : list_sh[i].rows - 128 * (unit - 1);
        for (int c0 = 0; c0 < chunks; c0 += 2) {
          good = warp_wait(sfull_bar[ss], sph);
          if (!good) {
            fail(7000004);
            break;
          }
          uint8_t* raw = smem + C::kScaleAt + ss * C::kSlotBytes + unit * 128 * kSlotRow;
          if (unit <= C::kHalves && rows > 0) {
            // rows 32 b + lane, both halves (32-byte swizzle: the halves of
            // rows 4-7 of every 8 change places)
            uint4 v[2][4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              if (32 * b < rows) {
                const uint8_t* r = raw + (32 * b + lane) * kSlotRow;
                const int swap = (lane & 4) << 2;
                v[0][b] = *reinterpret_cast<const uint4*>(r + swap);
                v[1][b] = *reinterpret_cast<const uint4*>(r + (swap ^ 16));
              } else {
                v[0][b] = v[1][b] = make_uint4(0, 0, 0, 0);
              }
            }
            const int left = blocks - 16 * c0;  // scale bytes from here to the end of K
            if (left < 32) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t m[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                  const int l = left - 16 * h - 4 * w;
                  m[w] = l >= 4 ? 0xffffffffu : l <= 0 ? 0u : (1u << (8 * l)) - 1;
                }
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                  v[h][b].x &= m[0];
                  v[h][b].y &= m[1];
                  v[h][b].z &= m[2];
                  v[h][b].w &= m[3];
                }
              }
            }
            __syncwarp();  // all read before any writes
            uint4* o = reinterpret_cast<uint4*>(raw) + lane;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              o[128 * h] = make_uint4(v[h][0].x, v[h][1].x, v[h][2].x, v[h][3].x);
              o[128 * h + 32] = make_uint4(v[h][0].y, v[h][1].y, v[h][2].y, v[h][3].y);
              o[128 * h + 64] = make_uint4(v[h][0].z, v[h][1].z, v[h][2].z, v[h][3].z);
              o[128 * h + 96] = make_uint4(v[h][0].w, v[h][1].w, v[h][2].w, v[h][3].w);
            }
            ptx::fence_proxy_async_smem();  // written by threads, read by the tensor core's copies
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&sblock_bar[ss]));
          if (++ss == kSlots) {
            ss = 0;
            sph ^= 1u;
          }
        }
      }
    } else if (warp >= 8) {
      // ------------------------------------------------ epilogue
      constexpr int kTok = sizeof(OT) == 2 && kTN > 32 ? 32 : 16;  // tokens staged at a time
      constexpr int kPieces = 2 * sizeof(OT);                      // 16-byte pieces of a token's 32 values
      constexpr int kPerPiece = 16 / sizeof(OT);
      const int q = warp & 3;             // TMEM lane quarter this warp may read
      const int half = (warp - 8) >> 2;   // the warps of a quarter take turns
      constexpr int kTurns = kEpiWarps / 4;
      uint8_t* scratch = smem + C::kScratchAt + (warp - 8) * kScratch;
      OT* out = static_cast<OT*>(a.out);
      const float ga = a.a_tscale ? *a.a_tscale : 1.f;
      for (int i = 0; i < n; ++i, ++it) {
        const Tile ti = list_sh[i];
        const Factors f = kNv ? factors(ga, a.b_tscale ? a.b_tscale[ti.e] : 1.f) : Factors{1.f, 1.f};
        auto scaled = [&](uint32_t sum) { return from_f32<OT>(__uint_as_float(sum) * f.first * f.second); };
        const int n0 = ti.m0 + 32 * q;
        if (!warp_wait_sleep(accf_bar[it & 1], uint32_t(it >> 1) & 1u)) {
          fail(7000005);
          break;
        }
        ptx::tc_fence_after();
        const uint32_t taddr = tmem + (uint32_t(32 * q) << 16) + uint32_t((it & 1) * kTN);
        for (int c0 = kTok * half; c0 < ti.rows; c0 += kTurns * kTok) {
          uint32_t v[kTok];
          if constexpr (kTok == 32)
            ptx::tmem_ld32(taddr + uint32_t(c0), v);
          else
            ptx::tmem_ld16(taddr + uint32_t(c0), v);
          ptx::tmem_ld_wait();
          if (a.vec_store) {
            OT* sc = reinterpret_cast<OT*>(scratch);
#pragma unroll
            for (int j = 0; j < kTok; ++j) sc[j * 32 + lane] = scaled(v[j]);
            __syncwarp();
            OT* o = out + (size_t)(ti.row0 + c0 + lane / kPieces) * a.N + n0 + lane % kPieces * kPerPiece;
            const bool in = n0 + lane % kPieces * kPerPiece < a.N;
#pragma unroll
            for (int p = 0; p < kTok * kPieces / 32; ++p) {
              const int tok = lane / kPieces + p * (32 / kPieces);
              if (in && c0 + tok < ti.rows)
                *reinterpret_cast<uint4*>(o + (size_t)p * (32 / kPieces) * a.N) =
                    *reinterpret_cast<const uint4*>(scratch + (p * 32 + lane) * 16);
            }
            __syncwarp();
          } else if (n0 + lane < a.N) {
            OT* o = out + (size_t)(ti.row0 + c0) * a.N + n0 + lane;
#pragma unroll
            for (int j = 0; j < kTok; ++j)
              if (c0 + j < ti.rows) o[(size_t)j * a.N] = scaled(v[j]);
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&acce_bar[it & 1]));
      }
    }
    if (warp < 4) {  // the elected lane's state, whichever lane is elected next
      const int from = ptx::elected_lane();
      s = __shfl_sync(0xffffffffu, s, from);
      ph = __shfl_sync(0xffffffffu, ph, from);
      ss = __shfl_sync(0xffffffffu, ss, from);
      sph = __shfl_sync(0xffffffffu, sph, from);
      wb = __shfl_sync(0xffffffffu, wb, from);
      it = __shfl_sync(0xffffffffu, it, from);
      issued = __shfl_sync(0xffffffffu, issued, from);
    }
    __syncthreads();  // the list may be written again
    if (*abort_p) break;
  }

  // No copy and no MMA may be in flight when the CTA leaves. They end by
  // themselves, also after a wait that gave up, so that these waits are met; were
  // one not within its limit of a second, the CTA would leave all the same.
  if (warp == 1 && ptx::elect_one()) {
    ptx::mma_commit(ptx::smem_addr(&drain_bar));
    ptx::mbar_wait(ptx::smem_addr(&drain_bar), 0, nullptr);
  } else if (warp == 0 || warp == 3) {
    // A stage is full when both warps' copies are there. After a wait that gave
    // up one of them may have stopped earlier: it arrives without a copy (it is at
    // most a ring behind, and where it stopped the stage waits for it alone).
    for (uint32_t i = sent_sh[warp != 0]; int(sent_sh[warp == 0] - i) > 0; ++i) {
      if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&full_bar[s]));
      issued = min(issued + 1, kStages);
      if (++s == kStages) {
        s = 0;
        ph ^= 1u;
      }
    }
    __syncwarp();
    for (int i = 0; i < issued; ++i) {
      if (--s < 0) {
        s = kStages - 1;
        ph ^= 1u;
      }
      ptx::mbar_wait(ptx::smem_addr(&full_bar[s]), ph, nullptr);
    }
  } else if (warp == 2) {
    for (int i = 0; i < issued; ++i) {
      if (--ss < 0) {
        ss = kSlots - 1;
        sph ^= 1u;
      }
      ptx::mbar_wait(ptx::smem_addr(&sfull_bar[ss]), sph, nullptr);
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

// Bytes [planes, rows, row_bytes] in boxes of box_bytes x box_rows.
bool byte_map(CUtensorMap* map, const uint8_t* base, uint64_t row_bytes, uint64_t rows, uint64_t planes, int dims,
              uint32_t box_bytes, uint32_t box_rows) {
  const EncodeFn f = encoder();
  if (!f) return false;
  const cuuint64_t size[3] = {row_bytes, rows, planes};
  const cuuint64_t stride[2] = {row_bytes, row_bytes * rows};
  const cuuint32_t box[3] = {box_bytes, box_rows, 1}, step[3] = {1, 1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, cuuint32_t(dims), const_cast<uint8_t*>(base), size, stride, box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE, box_bytes == 32 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tokens per tile. Few rows per expert (at most 32 on average): narrow tiles,
// two CTAs per SM, so that one's weights stream while the other computes. The host
// knows the average alone. 512 experts, 1,536 x 2,048 MX, cold, narrow and wide:
// evenly 40 rows 25 and 27 us, 640: 145 and 154, 8,192: 152 and 158, 16,384: 154
// and 160, 32,768: 180 and 168; skewed (Zipf, an expert at most once a token)
// 640: 82 and 84, 8,192: 156 and 160, 16,384: 174 and 166, 32,768: 221 and 182. All
// rows with one expert, which no router of several picks does: 640: 14 and 14,
// 8,192: 47 and 29, 16,384: 80 and 43.
constexpr int kNarrowTN = 32, kWideTN = 160;
bool narrow_tiles(int R, int E) { return R <= 32LL * E; }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return n;
}

template <bool kNv, int kTN, int kStages, int kSlots, typename OT>
cudaError_t run(const Maps& m, const Args& a, cudaStream_t st) {
  using C = Cfg<kTN, kStages, kSlots>;
  auto* kernel = fp4_gemm_kernel<kNv, kTN, kStages, kSlots, OT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  // at most this many tiles: every group with rows may end in a partial one
  const long long most = ((long long)a.R / kTN + (a.R < a.E ? a.R : a.E) + 1) * ((a.N + kBM - 1) / kBM);
  const int sms = sm_count() * (C::kNarrow ? 2 : 1);
  return launch_chained(kernel, dim3(unsigned(most < sms ? most : sms)), C::kThreads, C::kSmem, st, m, a);
}

template <bool kNv, typename OT>
cudaError_t run_tiles(const Maps& m, const Args& a, cudaStream_t st) {
  if (narrow_tiles(a.R, a.E)) return run<kNv, kNarrowTN, 3, 3, OT>(m, a, st);
  return run<kNv, kWideTN, 4, 4, OT>(m, a, st);
}

template <bool kNv>
cudaError_t run_out(int32_t dtype, const Maps& m, const Args& a, cudaStream_t st) {
  if (dtype == MOE_DT_BF16) return run_tiles<kNv, __nv_bfloat16>(m, a, st);
  if (dtype == MOE_DT_FP16) return run_tiles<kNv, __half>(m, a, st);
  return run_tiles<kNv, float>(m, a, st);
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
  // and the tiles are counted in 32 bits
  if (R < 0 || R > (1 << 30) || E < 1 || E > kMaxE || N < 1 || N > kMaxFpCols || K < 32 || K % 32 || K > kMaxFpCols ||
      (int64_t)N * K >= (1LL << 41) || (int64_t)R * N > (1LL << 40))
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
  Maps m;
  const int S = scale_stride(format == MOE_FP_NV, K);
  if (!byte_map(&m.wcodes, b_codes, K / 2, N, E, 3, kBKBytes, kBM) ||
      !byte_map(&m.tcodes, a_codes, K / 2, R, 1, 2, kBKBytes, kBoxRows) ||
      (!narrow_tiles(R, E) && !byte_map(&m.tall, a_codes, K / 2, R, 1, 2, kBKBytes, kWideTN)) ||
      !byte_map(&m.wscales, b_scales, S, N, E, 3, kSlotRow, kBM) ||
      !byte_map(&m.tscales, a_scales, S, R, 1, 2, kSlotRow, kBoxRows))
    return launched(cudaErrorInvalidValue);
  Args a{a_tensor_scale, b_tensor_scale, offsets, out, ws_at<WsHeader>(ws, 0), R, K, N, E,
         int((size_t(N) * size) % 16 == 0 && ptr_aligned(out, 16)), wait_cycles()};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launched(format == MOE_FP_NV ? run_out<true>(out_dtype, m, a, st) : run_out<false>(out_dtype, m, a, st));
}
