// Scores of a cache's pages for the step's queries, by which page selection chooses (choose.cu).
//
// score(row, KV head, page) = max over the heads h of  sum_d max(q_hd lo_d, q_hd hi_d), and since the larger of the two
// products is the one with hi where q is positive and with lo elsewhere,
//   sum_d max(q lo, q hi) = sum_d min(q, 0) lo + max(q, 0) hi :
// a matrix product of [min(q, 0) | max(q, 0)] with the pages' rows [lo | hi], which is how the bounds lie in memory.
//
//  * One work item is a query tile of one request and KV head and a run of its pages' tiles.  A query tile is 128 rows:
//    the heads of a token in a power of two of rows, so that they lie in one warp and their maximum is taken by
//    exchanges that halve the columns each time (a group of 12 heads uses 96 of the 128 rows).
//  * D = A.B^T (tcgen05, M = 128 query rows, N = 128 pages, K = 2 dims): the split queries lie in tensor memory, where
//    they stay for the item, so that shared memory is read for the pages alone (128 bytes a cycle at the tensor core's
//    full rate; with both operands there it would be twice as much as it has).  Two buffers of D in tensor memory.
//  * The pages' rows are gathered by page id, four at a time (TMA), 64 dims of 128 pages a stage, by sixteen warps into
//    a ring (a warp issues one gather after the other, ~40 ns each).  The next item's queries are loaded (TMA) while this one's products run.
//  * Scores are written as keys that have their order (choose.cuh), 0 for a page that does not exist.  For the error bound
//    the sum of |q| of every row is kept, and the largest |bound| of every tile of pages, taken from the ring by one warp
//    in the items of a request's last rows (which see all of its pages).
//  * What bounds it.  Decode: HBM.  Prompts: shared memory, 128 KB written and read a tile of 256 dims.
//  * Every mbarrier wait is bounded; a timeout records a code in the device status word, all roles leave their loops, copies
//    and MMAs in flight are drained, tensor memory is freed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "choose.cuh"
#include "window.cuh"

namespace qsa {
namespace {

using namespace window_detail;

template <int D>
struct ScoreCfg {
  static constexpr int kBlocks = 2 * D / 64;               // stages of a tile of pages
  static constexpr int kStageBytes = kScoreTile * 128;     // 64 dims of 128 pages
  static constexpr int kQBlocks = D / 64;
  static constexpr int kQBytes = kQBlocks * 128 * 128;
  static constexpr int kStages = D == 256 ? 9 : D == 128 ? 11 : 12;
  static constexpr int kThreads = 896;
  static constexpr int kGatherWarp0 = 12, kGatherWarps = 16;   // two a stage
  // registers per thread at launch, and after the split: the epilogue's two warpgroups, the gathers' four (the others keep
  // what they have)
  static constexpr int kLaunchRegs = 72, kEpilogueRegs = 104, kGatherRegs = 56;
  static_assert(256 * kEpilogueRegs + 128 * kLaunchRegs + 512 * kGatherRegs <= kThreads * kLaunchRegs, "register split");
  static constexpr int kRecords = 4;
  static constexpr int kSlots = 16;                        // > tiles between their gather and their scores
  static constexpr int kRingAt = kQBytes;
  static constexpr int kHereAt = kRingAt + kStages * kStageBytes;   // [kSlots][4] uint32: which pages exist
  static constexpr int kSumAt = kHereAt + kSlots * 16;     // [2][2][128] float: sums of |q|
  static constexpr int kCrossAt = kSumAt + 2048;           // [2][2][4][32] float: maxima of heads in several warps
  static constexpr int kRecAt = kCrossAt + 2048;
  static constexpr int kBarAt = kRecAt + kRecords * 64;
  // full, empty [stages]; dfull, dempty [2]; qfull, qempty, aready, adone, fin; recfull, recempty [records]
  static constexpr int kBars = 2 * kStages + 4 + 5 + 2 * kRecords;
  static constexpr int kTmemSlot = (kBarAt + 8 * kBars + 15) / 16 * 16;
  static constexpr int kSmem = kTmemSlot + 16;
  static_assert(kSmem <= kSmemLimit, "shared memory");
  static_assert(kStages / kBlocks + 4 < kSlots, "slots");
  static_assert(2 * D / 2 + 2 * kScoreTile <= 512, "tensor memory");
};

enum ScoreSite : int32_t {
  kPRecEmpty = 0x61, kPRecFull, kPQEmpty, kPQFull, kPStageEmpty, kPStageFull, kPDFull, kPDEmpty, kPAReady, kPADone
};

// A work item, written by the scheduler warp and read by every role.
struct Item {
  int32_t tiles;       // of pages (< 0: no more items)
  int32_t tile0;       // first of them
  int32_t req, kvh, row0, tokens;
  int32_t pages;       // of the request that its last row may choose
  int32_t last;        // the request's last rows
  int32_t first;       // the first run of pages
  int32_t pad[7];
};
static_assert(sizeof(Item) == 64, "item record");
__device__ __forceinline__ Item load_item(const Item* r) {
  Item x;
  const int4* s = reinterpret_cast<const int4*>(r);
  const int4 a = s[0], b = s[1];
  x.tiles = a.x; x.tile0 = a.y; x.req = a.z; x.kvh = a.w;
  x.row0 = b.x; x.tokens = b.y; x.pages = b.z; x.last = b.w;
  x.first = r->first;
  return x;
}

// Maxima over the GP lanes of a token, for 32 columns: each exchange halves the columns that a lane holds.  Afterwards a
// lane has 32 / GP columns, from (lane % GP) * 32 / GP on, in v[0] ...
template <int GP>
__device__ __forceinline__ void max_over_heads(float (&v)[32], int lane) {
  int n = 32;
#pragma unroll
  for (int d = GP / 2; d >= 1; d >>= 1) {
    n >>= 1;
    const bool up = lane & d;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      if (c < n) {
        const float send = up ? v[c] : v[c + n], keep = up ? v[c + n] : v[c];
        v[c] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, d));
      }
    }
  }
}
// Keys of a lane's N columns from col on (a multiple of N), to the keys of its token's row.  here: bit c of word k is
// whether the page of column 4 c + k exists.
template <int N>
__device__ __forceinline__ void store_keys(const float* v, const uint4& here, int col, uint32_t* to) {
  uint32_t k[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t word;
    if constexpr (N >= 4) {
      word = i % 4 == 0 ? here.x : i % 4 == 1 ? here.y : i % 4 == 2 ? here.z : here.w;
    } else {
      const int w = (col + i) & 3;
      word = w == 0 ? here.x : w == 1 ? here.y : w == 2 ? here.z : here.w;
    }
    k[i] = word >> ((col + i) >> 2) & 1u ? choose::key_of(v[i]) : 0u;
  }
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<uint4*>(to + i) = make_uint4(k[i], k[i + 1], k[i + 2], k[i + 3]);
  } else if constexpr (N == 2) {
    *reinterpret_cast<uint2*>(to) = make_uint2(k[0], k[1]);
  } else {
    *to = k[0];
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(ScoreCfg<D>::kThreads, 1)
    page_score_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmQ1,
                      const __grid_constant__ CUtensorMap tmQT, const __grid_constant__ ChooseParams p) {
  using C = ScoreCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const uint32_t b_full = base + C::kBarAt, b_empty = b_full + 8 * C::kStages;
  const uint32_t b_dfull = b_empty + 8 * C::kStages, b_dempty = b_dfull + 16;
  const uint32_t b_qfull = b_dempty + 16, b_qempty = b_qfull + 8, b_aready = b_qempty + 8, b_adone = b_aready + 8;
  const uint32_t b_fin = b_adone + 8, b_recfull = b_fin + 8, b_recempty = b_recfull + 8 * C::kRecords;
  uint32_t* const here = reinterpret_cast<uint32_t*>(smem + C::kHereAt);
  float* const sums = reinterpret_cast<float*>(smem + C::kSumAt);
  float* const cross = reinterpret_cast<float*>(smem + C::kCrossAt);
  Item* const recs = reinterpret_cast<Item*>(smem + C::kRecAt);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kTmemSlot);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* const status = p.status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((base & 1023u) != 0) {   // (uniform over the grid)
    if (threadIdx.x == 0) atomicCAS(status, 0, 0x100 | kWDrain);
    return;
  }
  constexpr int kReaders = 8 + 1 + 1 + 1 + C::kGatherWarps;   // of a record: epilogue, MMA, scan, queries, gathers
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(b_full + 8 * s, 2);
      mbar_init(b_empty + 8 * s, 2);                       // the MMA and the scan
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_dfull + 8 * i, 1);
      mbar_init(b_dempty + 8 * i, 8);
    }
    mbar_init(b_qfull, 1);
    mbar_init(b_qempty, 8);
    mbar_init(b_aready, 8);
    mbar_init(b_adone, 1);
    mbar_init(b_fin, 1);
    for (int r = 0; r < C::kRecords; ++r) {
      mbar_init(b_recfull + 8 * r, 1);
      mbar_init(b_recempty + 8 * r, kReaders);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot, tm_d = tmem + D;       // A: D columns (2 D values of 16 bits); D: 2 x 128

  auto wait = [&](uint32_t bar, uint32_t parity, int32_t site) { return wait_for(bar, parity & 1, abort_flag, p, site); };
  // the record of item `it`, for a whole warp
  auto next = [&](uint32_t it, Item& x) -> bool {
    const uint32_t r = it % C::kRecords;
    if (!__all_sync(0xffffffffu, wait(b_recfull + 8 * r, it / C::kRecords, kPRecFull))) return false;
    x = load_item(recs + r);
    __syncwarp();
    if (lane == 0) mbar_arrive(b_recempty + 8 * r);
    return x.tiles >= 0;
  };
  auto finish_role = [&]() {
    tc_fence_before();
    __syncthreads();
  };

  if (warp < 8) {
    regs_inc<C::kEpilogueRegs>();
    // ------------------------------------------------------------ splits the queries, writes the scores
    const int wg = warp >> 2, quarter = warp & 3, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int tok = row / p.head_rows, head = row - tok * p.head_rows;
    uint32_t jt = 0, turn = 0;
    bool bad = false;
    for (uint32_t it = 0;; ++it) {
      Item x;
      const bool more = next(it, x);
      if (named_bar_any(1, 256, !more || bad)) break;      // all leave together
      const bool live = head < p.group && tok < x.tokens;
      const bool warp_live = quarter * 32 / p.head_rows < x.tokens;   // (else the warp's rows are not looked at)
      // the queries: this warpgroup's half of the columns, min(q, 0) or max(q, 0)
      bad |= !wait(b_qfull, it, kPQFull);
      if (it > 0) bad |= !wait(b_adone, it - 1, kPADone);
      tc_fence_after();
      float sum = 0.0f;
      const int src = tok * p.group + head;
      // (the sum of |q| is shared between the halves: the even and the odd blocks; one block: its even and odd words)
#pragma unroll 1
      for (int b = 0; b < C::kQBlocks && warp_live; ++b) {
        uint32_t v[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint4 y = make_uint4(0u, 0u, 0u, 0u);
          if (live) y = ld_shared_v4(base + b * 16384 + src * 128 + ((c ^ (src & 7)) << 4));
          v[4 * c] = y.x;
          v[4 * c + 1] = y.y;
          v[4 * c + 2] = y.z;
          v[4 * c + 3] = y.w;
        }
        if (C::kQBlocks == 1 || (b & 1) == wg) {
          float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            if (C::kQBlocks == 1 && (c & 1) != 0) continue;
            const float2 y = choose::floats_of<T>(C::kQBlocks == 1 && wg == 1 ? v[c + 1] : v[c]);
            s0 += fabsf(y.x);
            s1 += fabsf(y.y);
          }
          sum += s0 + s1;
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = wg == 0 ? choose::best2<T, false>(v[c], 0u) : choose::best2<T, true>(v[c], 0u);
        tmem_st32(tmem + lanes + wg * (D / 2) + b * 32, v);
      }
      tc_wait_st();
      sums[(it & 1) * 256 + wg * 128 + row] = sum;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(b_aready);
        mbar_arrive(b_qempty);
      }
      if (x.first) {
        named_bar_sync(1, 256);
        if (threadIdx.x < x.tokens) {
          const float* const s = sums + (it & 1) * 256 + threadIdx.x * p.head_rows;
          uint32_t most = 0;                               // (bits of non-negative floats have their order, NaN above all)
          for (int h = 0; h < p.group; ++h) most = max(most, __float_as_uint(s[h] + s[128 + h]) & 0x7fffffffu);
          p.reach[(static_cast<int64_t>(x.row0) + threadIdx.x) * p.n_kvheads + x.kvh] = __uint_as_float(most);
        }
      }
      uint32_t* const keys = p.keys + ((static_cast<int64_t>(x.row0) + tok) * p.n_kvheads + x.kvh) * p.key_stride;
      for (int j = 0; j < x.tiles; ++j, ++jt) {
        bad |= !wait(b_dfull + 8 * (jt & 1), jt >> 1, kPDFull);
        tc_fence_after();
        const uint4 exist = *reinterpret_cast<const uint4*>(here + (jt % C::kSlots) * 4);
        if (!warp_live && p.head_rows <= 32) {
          __syncwarp();
          if (lane == 0) mbar_arrive(b_dempty + 8 * (jt & 1));
          continue;
        }
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          float v[32];
          tmem_ld32(tm_d + lanes + (jt & 1) * kScoreTile + wg * 64 + half * 32, v);
          tc_wait_ld();
          if (half == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_dempty + 8 * (jt & 1));
          }
          if (!live) {
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = -INFINITY;
          }
          const int col = wg * 64 + half * 32;             // of the tile
          uint32_t* const to = keys + (x.tile0 + j) * kScoreTile + col;
          const bool store = tok < x.tokens;
          switch (p.head_rows) {
            case 1:
              if (store) store_keys<32>(v, exist, col, to);
              break;
            case 2: {
              max_over_heads<2>(v, lane);
              const int c = (lane & 1) * 16;
              if (store) store_keys<16>(v, exist, col + c, to + c);
              break;
            }
            case 4: {
              max_over_heads<4>(v, lane);
              const int c = (lane & 3) * 8;
              if (store) store_keys<8>(v, exist, col + c, to + c);
              break;
            }
            case 8: {
              max_over_heads<8>(v, lane);
              const int c = (lane & 7) * 4;
              if (store) store_keys<4>(v, exist, col + c, to + c);
              break;
            }
            case 16: {
              max_over_heads<16>(v, lane);
              const int c = (lane & 15) * 2;
              if (store) store_keys<2>(v, exist, col + c, to + c);
              break;
            }
            case 32: {
              max_over_heads<32>(v, lane);
              if (store) store_keys<1>(v, exist, col + lane, to + lane);
              break;
            }
            default: {                                     // 64 or 128: two or four warps hold a token's heads
              max_over_heads<32>(v, lane);
              float* const m = cross + ((turn & 1) * 2 + wg) * 128;
              ++turn;
              m[quarter * 32 + lane] = v[0];
              named_bar_sync(2 + wg, 128);
              if (store && head < 32) {
                for (int w = 1; w < p.head_rows / 32; ++w) v[0] = fmaxf(v[0], m[(quarter + w) * 32 + lane]);
                store_keys<1>(v, exist, col + lane, to + lane);
              }
            }
          }
        }
      }
    }
    finish_role();
    return;
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer, tensor-memory owner
    constexpr uint32_t kIdesc = std::is_same<T, __half>::value ? idesc_f16_f32(128, kScoreTile, false, false)
                                                               : idesc_bf16_f32(128, kScoreTile, false, false);
    constexpr uint32_t kHi = sw128_desc_hi(1024);
    const uint32_t ring_lo = sw128_desc_lo(base + C::kRingAt, 16);
    RingPos st;
    uint32_t jt = 0;
    bool stop = false;
    for (uint32_t it = 0; !stop; ++it) {
      Item x;
      if (!next(it, x)) break;
      if (!__all_sync(0xffffffffu, wait(b_aready, it, kPAReady))) {
        stop = true;
        break;
      }
      for (int j = 0; j < x.tiles && !stop; ++j, ++jt) {
        if (jt >= 2 && !__all_sync(0xffffffffu, wait(b_dempty + 8 * (jt & 1), (jt >> 1) - 1, kPDEmpty))) {
          stop = true;
          break;
        }
        for (int b = 0; b < C::kBlocks; ++b) {
          if (!__all_sync(0xffffffffu, wait(b_full + 8 * st.st, st.par, kPStageFull))) {
            stop = true;
            break;
          }
          tc_fence_after();
          if (lane == 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_ta(tm_d + (jt & 1) * kScoreTile, tmem + b * 32 + k * 8,
                        ring_lo + st.st * (C::kStageBytes >> 4) + k * 2, kHi, kIdesc, b > 0 || k > 0 ? 1u : 0u);
            tc_commit(b_empty + 8 * st.st);
            if (b == C::kBlocks - 1) {
              tc_commit(b_dfull + 8 * (jt & 1));
              if (j == x.tiles - 1) tc_commit(b_adone);
            }
          }
          __syncwarp();
          ring_next(st, C::kStages);
        }
      }
    }
    if (lane == 0) {
      tc_commit(b_fin);
      drain(b_fin, 0, status, kDrainNs);
    }
    __syncwarp();
    finish_role();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
    return;
  } else if (warp == 9) {
    // ------------------------------------------------------------ scan: the largest |bound| of every tile of pages
    RingPos st;
    for (uint32_t it = 0;; ++it) {
      Item x;
      if (!next(it, x)) break;
      bool ok = true;
      for (int j = 0; j < x.tiles && ok; ++j) {
        uint32_t most = 0;                                 // two 16-bit magnitudes, in the upper halves of two words
        uint32_t most2 = 0;
        for (int b = 0; b < C::kBlocks && ok; ++b) {
          ok = __all_sync(0xffffffffu, wait(b_full + 8 * st.st, st.par, kPStageFull));
          if (ok && x.last) {
            const uint32_t at = base + C::kRingAt + st.st * C::kStageBytes + lane * 16;
#pragma unroll 8
            for (int i = 0; i < C::kStageBytes / 512; ++i) {
              const uint4 y = ld_shared_v4(at + i * 512);
              most = max(most, max(max(y.x & 0x7fff0000u, y.y & 0x7fff0000u), max(y.z & 0x7fff0000u, y.w & 0x7fff0000u)));
              most2 = max(most2, max(max(y.x << 17, y.y << 17), max(y.z << 17, y.w << 17)));
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(b_empty + 8 * st.st);
          ring_next(st, C::kStages);
        }
        most = max(most, most2 >> 1) >> 16;
        most = __reduce_max_sync(0xffffffffu, most);
        if (x.last && lane == 0) {
          const float2 f = choose::floats_of<T>(most);
          p.largest[(static_cast<int64_t>(x.req) * p.n_kvheads + x.kvh) * p.page_tiles + x.tile0 + j] = f.x;
        }
      }
      if (!ok) break;
    }
    finish_role();
    return;
  } else if (warp == 10) {
    // ------------------------------------------------------------ scheduler
    const int64_t first = blockIdx.x;
    uint32_t it = 0;
    auto put = [&](const Item& x) -> bool {
      const uint32_t r = it % C::kRecords;
      if (it >= C::kRecords && !__all_sync(0xffffffffu, wait(b_recempty + 8 * r, it / C::kRecords - 1, kPRecEmpty))) return false;
      if (lane == 0) {
        int4* const to = reinterpret_cast<int4*>(recs + r);
        to[0] = make_int4(x.tiles, x.tile0, x.req, x.kvh);
        to[1] = make_int4(x.row0, x.tokens, x.pages, x.last);
        recs[r].first = x.first;
        mbar_arrive(b_recfull + 8 * r);
      }
      __syncwarp();
      ++it;
      return true;
    };
    bool ok = !p.stall_first_item;
    for (int64_t n = first; n < p.n_items && ok; n += gridDim.x) {
      const int32_t unit = static_cast<int32_t>(n) / p.runs, run = static_cast<int32_t>(n) - unit * p.runs;
      const int32_t tile = unit / p.n_kvheads;
      Item x{};
      x.kvh = unit - tile * p.n_kvheads;
      // (numbers of tiles as in window_detail::first_tile)
      auto first_tile = [&](int32_t i) { return __ldg(p.pa.cu_seqlens_q + i) / p.tile_tokens + i; };
      int32_t lo = 0, hi = p.pa.n_requests - 1;
      while (lo < hi) {
        const int32_t step = (hi - lo + 32) / 32;
        const int32_t cand = lo + lane * step;
        const uint32_t m = __ballot_sync(0xffffffffu, cand <= hi && first_tile(cand) <= tile);
        const int l = m ? 31 - __clz(m) : 0;
        lo = lo + l * step;
        hi = min(hi, lo + step - 1);
      }
      x.req = lo;
      const int64_t r0 = __ldg(p.pa.cu_seqlens_q + lo), kv = __ldg(p.pa.kv_lens + lo);
      const int64_t r1 = min(static_cast<int64_t>(__ldg(p.pa.cu_seqlens_q + lo + 1)), p.n_rows);
      const int64_t t0 = static_cast<int64_t>(tile - first_tile(lo)) * p.tile_tokens;
      if (r0 < 0 || t0 < 0 || r0 + t0 >= r1) continue;
      x.row0 = static_cast<int32_t>(r0 + t0);
      x.tokens = static_cast<int32_t>(min(r1 - r0 - t0, static_cast<int64_t>(p.tile_tokens)));
      x.last = r0 + t0 + x.tokens == r1;
      const int64_t p_last = kv - (r1 - r0) + t0 + x.tokens - 1;
      if (p_last < 0) continue;
      const int32_t own = p.pa.page_shift >= 0 ? static_cast<int32_t>(p_last >> p.pa.page_shift)
                                               : static_cast<int32_t>(p_last) / p.pa.page_size;   // (p_last < kv)
      x.pages = min(own + 1, p.pa.pages_per_req);
      if (x.pages <= p.n_select) continue;                 // all of them are chosen
      x.first = run == 0;
      x.tile0 = run * p.run_tiles;
      x.tiles = min((x.pages + kScoreTile - 1) / kScoreTile - x.tile0, p.run_tiles);
      if (x.tiles <= 0) continue;
      ok = put(x);
    }
    Item end{};
    end.tiles = -1;
    if (ok) put(end);
    finish_role();
    return;
  } else if (warp == 11) {
    // ------------------------------------------------------------ queries
    if (lane == 0) {
      prefetch_tmap(&tmQ1);
      prefetch_tmap(&tmQT);
      prefetch_tmap(&tmB);
    }
    uint32_t loaded = 0;
    for (uint32_t it = 0;; ++it) {
      Item x;
      if (!next(it, x)) break;
      if (it > 0 && !__all_sync(0xffffffffu, wait(b_qempty, it - 1, kPQEmpty))) break;
      const uint32_t tok_bytes = static_cast<uint32_t>(p.group) * 128u;
      const bool whole = x.tokens == p.tile_tokens;
      if (lane == 0) mbar_arrive_expect_tx(b_qfull, static_cast<uint32_t>(x.tokens) * tok_bytes * C::kQBlocks);
      __syncwarp();
      const int loads = whole ? C::kQBlocks : x.tokens * C::kQBlocks;
      for (int i = lane; i < loads; i += 32) {
        const int b = i % C::kQBlocks, t = i / C::kQBlocks;
        tma_load_3d(base + b * 16384 + t * tok_bytes, whole ? &tmQT : &tmQ1, b * 64, x.kvh * p.group, x.row0 + t, b_qfull);
      }
      ++loaded;
    }
    if (*abort_flag && loaded > 0 && lane == 0) drain(b_qfull, (loaded - 1) & 1, status, kDrainNs);
    __syncwarp();
    finish_role();
    return;
  }
  // -------------------------------------------------------------- gathers: pairs of warps take the blocks in turn, each
  // half of a block's pages
  regs_dec<C::kGatherRegs>();
  const int gw = (warp - C::kGatherWarp0) >> 1, part = warp & 1;
  constexpr int kPairs = C::kGatherWarps / 2, kEvery = kPairs / C::kBlocks;   // tiles between two of a pair's
  const int block = gw % C::kBlocks, tile_turn = gw / C::kBlocks;
  uint32_t jt = 0, issued = 0;
  Item x{};
  uint32_t it = 0;
  int j = 0;
  bool more = next(it, x), stop = false;
  struct Rows {
    int32_t r[4];
    uint32_t here;
  };
  // page ids of the four pages of lane l (of 32) in tile t of item y
  auto look_up = [&](const Item& y, int t, int l) {
    Rows k;
    k.here = 0;
    const int32_t e0 = (y.tile0 + t) * kScoreTile + l * 4;
    const int32_t* const table = p.pa.page_table + static_cast<int64_t>(y.req) * p.pa.pages_per_req;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int32_t id = e0 + i < y.pages ? __ldg(table + e0 + i) : -1;
      const bool in = id >= 0 && id < p.pa.n_pages;
      k.r[i] = static_cast<int32_t>((in ? id : p.pa.n_pages) * p.n_kvheads + (in ? y.kvh : 0));   // (past the end: zeros)
      k.here |= (in ? 1u : 0u) << i;
    }
    return k;
  };
  // the pair's next tile from (it, x, j) on
  auto seek = [&]() {
    while (more) {
      if (j >= x.tiles) {
        ++it;
        j = 0;
        more = next(it, x);
        continue;
      }
      if (jt % kEvery == static_cast<uint32_t>(tile_turn)) return;
      ++j;
      ++jt;
    }
  };
  const int mine = part * 16 + (lane & 15);                // lanes 0-15 gather; all look up, for the pages that exist
  seek();
  Rows rows{};
  if (more) rows = look_up(x, j, part == 0 && block == 0 ? lane : mine);
  while (more) {
    const uint32_t tile = jt, n = tile * C::kBlocks + block, s = n % C::kStages;
    const Rows now = rows;
    if (n >= C::kStages && !__all_sync(0xffffffffu, wait(b_empty + 8 * s, n / C::kStages - 1, kPStageEmpty))) {
      stop = true;
      break;
    }
    if (block == 0 && part == 0) {
      uint32_t m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) m[i] = __ballot_sync(0xffffffffu, now.here >> i & 1u);
      if (lane == 0) *reinterpret_cast<uint4*>(here + (tile % C::kSlots) * 4) = make_uint4(m[0], m[1], m[2], m[3]);
    }
    if (lane == 0) mbar_arrive_expect_tx(b_full + 8 * s, C::kStageBytes / 2);
    __syncwarp();
    if (lane < 16)
      tma_gather4(base + C::kRingAt + s * C::kStageBytes + mine * 512, &tmB, block * 64, now.r[0], now.r[1], now.r[2],
                  now.r[3], b_full + 8 * s);
    issued = n + 1;
    ++j;
    ++jt;
    seek();
    if (more) rows = look_up(x, j, part == 0 && block == 0 ? lane : mine);
  }
  if (issued > 0 && lane == 0 && (stop || *abort_flag)) {
    // this warp's copies that may still be in flight: of the last ring
    const uint32_t last = issued - 1;
    for (uint32_t n = last; last - n < static_cast<uint32_t>(C::kStages); n -= kPairs) {
      drain(b_full + 8 * (n % C::kStages), (n / C::kStages) & 1, status, kDrainNs / 100);
      if (n < static_cast<uint32_t>(kPairs)) break;
    }
  }
  __syncwarp();
  finish_role();
}

template <int D, typename T>
cudaError_t launch_score_dim(const ChooseParams& p, const CUtensorMap& tb, const CUtensorMap& tq1, const CUtensorMap& tqt,
                             int grid, int which, cudaStream_t stream) {
  using C = ScoreCfg<D>;
  auto kern = page_score_kernel<D, T>;
  const cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(kern), C::kSmem, kOptScore + which);
  if (e != cudaSuccess) return e;
  // (the register shares add up to what the block is launched with: a kernel compiled to fewer would wait for ever)
  static const int regs = [&] {
    cudaFuncAttributes a{};
    return cudaFuncGetAttributes(&a, kern) == cudaSuccess ? a.numRegs : 0;
  }();
  if (regs < C::kLaunchRegs) return cudaErrorInvalidConfiguration;
  kern<<<grid, C::kThreads, C::kSmem, stream>>>(tb, tq1, tqt, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_page_score(const ChooseParams& p, bool fp16, int num_sms, cudaStream_t stream) {
  const CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;   // (16 bits are moved either way)
  const cuuint64_t d = static_cast<cuuint64_t>(p.head_dim);
  CUtensorMap tb{}, tq1{}, tqt{};
  const cuuint64_t b_dims[2] = {2 * d, static_cast<cuuint64_t>(p.pa.n_pages) * static_cast<cuuint64_t>(p.n_kvheads)};
  const cuuint64_t b_strides[1] = {4 * d};
  const cuuint32_t b_box[2] = {64, 1};
  CUresult r = encode_tensor_map(&tb, type, 2, p.bounds, b_dims, b_strides, b_box);
  const cuuint64_t q_dims[3] = {d, static_cast<cuuint64_t>(p.n_qheads), static_cast<cuuint64_t>(p.n_rows)};
  const cuuint64_t q_strides[2] = {d * 2, d * 2 * static_cast<cuuint64_t>(p.n_qheads)};
  const cuuint32_t q_box1[3] = {64, static_cast<cuuint32_t>(p.group), 1};
  const cuuint32_t q_boxt[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(p.tile_tokens)};
  if (r == CUDA_SUCCESS) r = encode_tensor_map(&tq1, type, 3, p.q, q_dims, q_strides, q_box1);
  if (r == CUDA_SUCCESS) r = encode_tensor_map(&tqt, type, 3, p.q, q_dims, q_strides, q_boxt);
  if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  const int grid = static_cast<int>(p.n_items < num_sms ? p.n_items : num_sms);
  if (fp16)
    return p.head_dim == 64    ? launch_score_dim<64, __half>(p, tb, tq1, tqt, grid, 0, stream)
           : p.head_dim == 128 ? launch_score_dim<128, __half>(p, tb, tq1, tqt, grid, 1, stream)
                               : launch_score_dim<256, __half>(p, tb, tq1, tqt, grid, 2, stream);
  return p.head_dim == 64    ? launch_score_dim<64, __nv_bfloat16>(p, tb, tq1, tqt, grid, 3, stream)
         : p.head_dim == 128 ? launch_score_dim<128, __nv_bfloat16>(p, tb, tq1, tqt, grid, 4, stream)
                             : launch_score_dim<256, __nv_bfloat16>(p, tb, tq1, tqt, grid, 5, stream);
}

}  // namespace qsa
