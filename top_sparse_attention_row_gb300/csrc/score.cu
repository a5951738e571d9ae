// Scores of a cache's pages for the step's queries, by which page selection chooses (select.cuh).
//
// score(row, KV head, page) = max over the heads h of  sum_d max(q_hd lo_d, q_hd hi_d), and since the larger of the two
// products is the one with hi where q is positive and with lo elsewhere,
//   sum_d max(q lo, q hi) = sum_d min(q, 0) lo + max(q, 0) hi :
// a matrix product of the pages' rows [lo | hi], which is how the bounds lie in memory, with [min(q, 0) | max(q, 0)].
//
//  * One work item is a query tile of one request and KV head (the heads of up to 128 / group tokens) and a run of its
//    pages' tiles.  D = pages x queries (tcgen05, M = 128 pages, N = the heads of the item's tokens, K = 2 dims), both
//    operands in shared memory, three buffers of D in tensor memory.  A thread of the epilogue has a page, so the maximum
//    over a token's heads is one over neighbouring columns, and 32 pages' keys are written side by side.
//    (The other way round, with the queries as M from tensor memory, an MMA of N = 128 takes 90 to 110 cycles where this
//    one takes 65, and the maxima go across lanes: 192 us of scores for 8192 prompt rows, 24/2 heads of 256 dims, where this takes 143.)
//  * The split queries of an item lie in shared memory until its products are done.  Eight warps have the next item's
//    queries in registers by then, and have summed |q| for the error bound.
//  * The pages' rows are gathered by page id, four at a time (TMA), 128 dims of 128 pages a stage, by four warps into a
//    ring, three stages at once: a warp issues one gather after the other, ~50 ns each.  (cp.async, 16 bytes a thread,
//    brought 30 bytes a cycle beside the building of the queries.)  A stage has eight MMAs, because a commit costs the
//    tensor core about two of them.
//  * Scores are written as keys that have their order (choose.cuh), 0 for a page that does not exist.  For the error bound
//    the largest |bound| of every 64 pages is taken from the ring by two warps, in the items of a request's last rows (which
//    see all of its pages).
//  * What bounds it.  Prompts: shared memory.  An MMA reads 8 KB in the 65 cycles it takes alone (126 of 128 bytes a cycle),
//    beside the gathers' writes and the queries', and a commit stands for two of them: ~4000 cycles a tile of 256 dims,
//    2048 for its MMAs (8192 rows at 24k, 24/2 heads: 143 us, 0.63 PFLOP/s).  Decode: HBM at half its rate (64 rows at
//    64k to 128k: 47 us, 4.1 TB/s).  Six stages of 32 KB an SM are more than its latency asks for.  Items are dealt out by
//    their numbers, a third of which have no rows, so the block with the most has 12 page tiles where the mean is 10.2; an
//    item is one tile of its queries, which are split anew for each into the one buffer that the item before it has
//    to leave; and a stage is free only when the scan has read all of it.
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

// QROWS: columns that an item's queries may have, 128, or 32 where the batch is mostly single tokens: the room goes to the
// ring then (64 tokens at 64k to 128k, 24/2 heads of 256 dims: 47 us of scores, with 128 columns 63).
template <int D, int QROWS>
struct ScoreCfg {
  static constexpr int kPer = D / 64;                      // stages of a tile of pages: 128 of 2 D dims each
  static constexpr int kStageBytes = kScoreTile * 256;
  static constexpr int kBlock = 128 * 128;                 // bytes of 64 dims of 128 rows
  static constexpr int kQBlock = QROWS * 128;              // of the queries
  static constexpr int kQBytes = 2 * D / 64 * kQBlock;     // the split queries
  static constexpr int kStages = QROWS == 32 ? 6 : D == 256 ? 3 : D == 128 ? 5 : 6;
  static constexpr int kThreads = 1024;
  static constexpr int kBuildWarp0 = 8, kMmaWarp = 16, kSchedulerWarp = 17, kScanWarp = 18, kGatherWarp0 = 20;
  static constexpr int kGatherWarps = 12, kStageWarps = 4;
  static constexpr int kChunks = QROWS * D / 8 / 256;      // 16-byte pieces of the queries a building thread has
  // registers per thread at launch, and after the split: epilogue and building warpgroups; the others
  static constexpr int kLaunchRegs = 64, kWideRegs = 80, kRoleRegs = 48;
  static_assert(512 * kWideRegs + 512 * kRoleRegs <= kThreads * kLaunchRegs, "register split");
  static constexpr int kRecords = 4;
  static constexpr int kSlots = 16;                        // > tiles between their gather and their scores
  static constexpr int kBuffers = 3;                       // of D, 128 columns each
  static constexpr int kRingAt = kQBytes;
  static constexpr int kHereAt = kRingAt + kStages * kStageBytes;   // [kSlots][4] uint32: which pages exist
  static constexpr int kSumAt = kHereAt + kSlots * 16;     // [2][128] float: sums of |q|
  static constexpr int kRecAt = kSumAt + 1024;
  static constexpr int kBarAt = kRecAt + kRecords * 64;
  // full, empty [stages]; dfull, dempty [buffers]; qready, adone, fin; recfull, recempty [records]
  static constexpr int kBars = 2 * kStages + 2 * kBuffers + 3 + 2 * kRecords;
  static constexpr int kTmemSlot = (kBarAt + 8 * kBars + 15) / 16 * 16;
  static constexpr int kSmem = kTmemSlot + 16;
  static_assert(kSmem <= kSmemLimit, "shared memory");
  static_assert(kStages / kPer + kBuffers + 2 < kSlots, "slots");
};

enum ScoreSite : int32_t {
  kPRecEmpty = 0x61, kPRecFull, kPStageEmpty, kPStageFull, kPDFull, kPDEmpty, kPQReady, kPADone
};

// A work item, written by the scheduler warp and read by every role.
struct Item {
  int32_t tiles;       // of pages (< 0: no more items)
  int32_t tile0;       // first of them
  int32_t req, kvh, row0, tokens;
  int32_t pages;       // of the request that its last row may choose
  int32_t flags;       // 1: the request's last rows; 2: the first run of pages
};
static_assert(sizeof(Item) == 32, "item record");
constexpr int32_t kLastRows = 1, kFirstRun = 2;
__device__ __forceinline__ Item load_item(const Item* r) {
  const int4* s = reinterpret_cast<const int4*>(r);
  const int4 a = s[0], b = s[1];
  return Item{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// The larger of two scores; NaN stays.
__device__ __forceinline__ float larger(float a, float b) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
  return a;
}
// Largest of v[0 .. N).
template <int N>
__device__ __forceinline__ float largest_of(const float* v) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = larger(m, v[i]);
  return m;
}

template <int D, typename T, int QROWS>
__global__ void __launch_bounds__(ScoreCfg<D, QROWS>::kThreads, 1) page_score_kernel(const __grid_constant__ CUtensorMap tmB,
                                                                               const __grid_constant__ ChooseParams p) {
  using C = ScoreCfg<D, QROWS>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const uint32_t b_full = base + C::kBarAt, b_empty = b_full + 8 * C::kStages;
  const uint32_t b_dfull = b_empty + 8 * C::kStages, b_dempty = b_dfull + 8 * C::kBuffers;
  const uint32_t b_qready = b_dempty + 8 * C::kBuffers, b_adone = b_qready + 8, b_fin = b_adone + 8;
  const uint32_t b_recfull = b_fin + 8, b_recempty = b_recfull + 8 * C::kRecords;
  uint32_t* const here = reinterpret_cast<uint32_t*>(smem + C::kHereAt);
  float* const sums = reinterpret_cast<float*>(smem + C::kSumAt);
  Item* const recs = reinterpret_cast<Item*>(smem + C::kRecAt);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kTmemSlot);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* const status = p.status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((base & 1023u) != 0) {   // (uniform over the grid)
    if (threadIdx.x == 0) atomicCAS(status, 0, 0x100 | kWDrain);
    return;
  }
  constexpr int kReaders = 8 + 8 + 1 + 2 + C::kGatherWarps;  // of a record: epilogue, build, MMA, scan, gathers
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(b_full + 8 * s, C::kStageWarps);
      mbar_init(b_empty + 8 * s, 3);                       // the MMA and the scan
    }
    for (int i = 0; i < C::kBuffers; ++i) {
      mbar_init(b_dfull + 8 * i, 1);
      mbar_init(b_dempty + 8 * i, 8);
    }
    mbar_init(b_qready, 8);
    mbar_init(b_adone, 1);
    mbar_init(b_fin, 1);
    for (int r = 0; r < C::kRecords; ++r) {
      mbar_init(b_recfull + 8 * r, 1);
      mbar_init(b_recempty + 8 * r, kReaders);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;

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
    // ------------------------------------------------------------ epilogue: two warpgroups share a tile's tokens
    regs_inc<C::kWideRegs>();
    const int wg = warp >> 2, quarter = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int g = p.group;
    const int64_t step = static_cast<int64_t>(p.n_kvheads) * p.key_stride;   // of a token's keys
    uint32_t buf = 0, turn = 0, slot = 0;
    for (uint32_t it = 0;; ++it) {
      Item x;
      if (!next(it, x)) break;
      uint32_t* const keys = p.keys + (static_cast<int64_t>(x.row0) * p.n_kvheads + x.kvh) * p.key_stride +
                             x.tile0 * kScoreTile + quarter * 32 + lane;
      bool ok = true;
      for (int j = 0; j < x.tiles; ++j) {
        ok = __all_sync(0xffffffffu, wait(b_dfull + 8 * buf, turn, kPDFull));
        if (!ok) break;
        tc_fence_after();
        const bool exists = here[slot * 4 + quarter] >> lane & 1u;
        uint32_t* const to = keys + j * kScoreTile;
        const uint32_t from = tmem + lanes + buf * 128;
        auto put = [&](int t, float m) { to[t * step] = exists ? choose::key_of(m) : 0u; };
        // sixteen columns at a time hold whole tokens where the group divides 16 (and reach past the tile's own columns
        // nowhere but into the next buffer's)
        const int columns = x.tokens * g;
        if (g == 1 || g == 2 || g == 4 || g == 8) {
          for (int c = wg * 16; c < columns; c += 32) {
            float v[16];
            tmem_ld16(from + c, v);
            tc_wait_ld();
            const int t = c / g;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (g == 1 && t + i < x.tokens) put(t + i, v[i]);
              if (g == 2 && i % 2 == 0 && t + i / 2 < x.tokens) put(t + i / 2, largest_of<2>(v + i));
              if (g == 4 && i % 4 == 0 && t + i / 4 < x.tokens) put(t + i / 4, largest_of<4>(v + i));
              if (g == 8 && i % 8 == 0 && t + i / 8 < x.tokens) put(t + i / 8, largest_of<8>(v + i));
            }
          }
        } else {
          for (int t = wg; t < x.tokens; t += 2) {
            float m = -INFINITY;
            for (int h0 = 0; h0 < g; h0 += 16) {
              float v[16];
              tmem_ld16(from + t * g + h0, v);
              tc_wait_ld();
#pragma unroll
              for (int h = 0; h < 16; ++h) m = h0 + h < g ? larger(m, v[h]) : m;
            }
            put(t, m);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_dempty + 8 * buf);
        if (++buf == C::kBuffers) {
          buf = 0;
          ++turn;
        }
        slot = (slot + 1) % C::kSlots;
      }
      if (!ok) break;
    }
    finish_role();
    return;
  }
  if (warp < 16) {
    // ------------------------------------------------------------ builds the split queries
    regs_inc<C::kWideRegs>();
    constexpr int kRowChunks = D / 8, kEvery = 256 / kRowChunks;   // 16-byte pieces of a row, rows between two of a thread's
    const int tid = threadIdx.x - 32 * C::kBuildWarp0, chunk = tid % kRowChunks, row0 = tid / kRowChunks;
    for (uint32_t it = 0;; ++it) {
      Item x;
      const bool more = next(it, x);
      if (named_bar_any(1, 256, *abort_flag != 0) || !more) break;   // all leave together
      const int rows = x.tokens * p.group;
      const T* const q = static_cast<const T*>(p.q) + (static_cast<int64_t>(x.row0) * p.n_qheads + x.kvh * p.group) * D + chunk * 8;
      uint4 v[C::kChunks];
#pragma unroll
      for (int i = 0; i < C::kChunks; ++i) {
        const int r = row0 + i * kEvery, t = r / p.group;
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) v[i] = __ldg(reinterpret_cast<const uint4*>(q + (static_cast<int64_t>(t) * p.n_qheads + (r - t * p.group)) * D));
      }
      if (x.flags & kFirstRun) {
#pragma unroll
        for (int i = 0; i < C::kChunks; ++i) {
          const float2 a = choose::floats_of<T>(v[i].x), b = choose::floats_of<T>(v[i].y), c = choose::floats_of<T>(v[i].z),
                       d = choose::floats_of<T>(v[i].w);
          float sum = ((fabsf(a.x) + fabsf(a.y)) + (fabsf(b.x) + fabsf(b.y))) + ((fabsf(c.x) + fabsf(c.y)) + (fabsf(d.x) + fabsf(d.y)));
#pragma unroll
          for (int o = kRowChunks / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (chunk == 0) sums[(it & 1) * 128 + row0 + i * kEvery] = sum;
        }
      }
      if (it > 0) wait(b_adone, it - 1, kPADone);          // (a wait that runs out shows at the next vote)
#pragma unroll
      for (int i = 0; i < C::kChunks; ++i) {
        const int r = row0 + i * kEvery;
        if (r < rows) {
          const uint32_t to = base + (chunk >> 3) * C::kQBlock + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
          const uint4 y = v[i];
          st_shared_v4(to, make_uint4(choose::best2<T, false>(y.x, 0u), choose::best2<T, false>(y.y, 0u),
                                      choose::best2<T, false>(y.z, 0u), choose::best2<T, false>(y.w, 0u)));
          st_shared_v4(to + C::kQBytes / 2, make_uint4(choose::best2<T, true>(y.x, 0u), choose::best2<T, true>(y.y, 0u),
                                                       choose::best2<T, true>(y.z, 0u), choose::best2<T, true>(y.w, 0u)));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_qready);
      if (x.flags & kFirstRun) {
        named_bar_sync(1, 256);
        if (tid < x.tokens) {
          const float* const s = sums + (it & 1) * 128 + tid * p.group;
          uint32_t most = 0;                               // (bits of non-negative floats have their order, NaN above all)
          for (int h = 0; h < p.group; ++h) most = max(most, __float_as_uint(s[h]) & 0x7fffffffu);
          p.reach[(static_cast<int64_t>(x.row0) + tid) * p.n_kvheads + x.kvh] = __uint_as_float(most);
        }
      }
    }
    finish_role();
    return;
  }
  regs_dec<C::kRoleRegs>();
  if (warp == C::kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer, tensor-memory owner
    constexpr uint32_t kIdesc = std::is_same<T, __half>::value ? idesc_f16_f32(128, 0, false, false)
                                                               : idesc_bf16_f32(128, 0, false, false);
    constexpr uint32_t kHi = sw128_desc_hi(1024);
    const uint32_t q_lo = sw128_desc_lo(base, 16), ring_lo = sw128_desc_lo(base + C::kRingAt, 16);
    if (lane == 0) {       // one thread issues; the others wait for it below
      RingPos st, d;
      uint32_t jt = 0;
      bool go = true;
      for (uint32_t it = 0; go; ++it) {
        const uint32_t r = it % C::kRecords;
        if (!wait(b_recfull + 8 * r, it / C::kRecords, kPRecFull)) break;
        const int32_t tiles = recs[r].tiles, columns = recs[r].tokens * p.group;
        mbar_arrive(b_recempty + 8 * r);
        if (tiles < 0 || !wait(b_qready, it, kPQReady)) break;
        const uint32_t idesc = kIdesc | static_cast<uint32_t>((columns + 15) / 16 * 2) << 17;   // N / 8
        for (int j = 0; j < tiles && go; ++j, ++jt) {
          if (jt >= C::kBuffers) go = wait(b_dempty + 8 * d.st, d.par ^ 1, kPDEmpty);
#pragma unroll
          for (int s = 0; s < C::kPer; ++s) {
            go = go && wait(b_full + 8 * st.st, st.par, kPStageFull);
            if (!go) break;
            tc_fence_after();
            const uint32_t a = ring_lo + st.st * (C::kStageBytes >> 4), b = q_lo + s * (2 * C::kQBlock >> 4);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              tc_mma_w(tmem + d.st * 128, a + (((k >> 2) * C::kBlock + (k & 3) * 32) >> 4), kHi,
                       b + (((k >> 2) * C::kQBlock + (k & 3) * 32) >> 4), kHi, idesc, s > 0 || k > 0 ? 1u : 0u);
            tc_commit(b_empty + 8 * st.st);
            ring_next(st, C::kStages);
          }
          if (go) {
            tc_commit(b_dfull + 8 * d.st);
            if (j == tiles - 1) tc_commit(b_adone);
            ring_next(d, C::kBuffers);
          }
        }
      }
      tc_commit(b_fin);
      drain(b_fin, 0, status, kDrainNs);
    }
    __syncwarp();
    finish_role();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
    return;
  } else if (warp == C::kScanWarp || warp == C::kScanWarp + 1) {
    // ------------------------------------------------------------ scan: the largest |bound| of every 64 pages
    const int part = warp - C::kScanWarp;
    RingPos st;
    for (uint32_t it = 0;; ++it) {
      Item x;
      if (!next(it, x)) break;
      const bool look = x.flags & kLastRows;
      bool ok = true;
      for (int j = 0; j < x.tiles && ok; ++j) {
        uint32_t most = 0, most2 = 0;                      // of pairs
        for (int s = 0; s < C::kPer && ok; ++s) {
          ok = __all_sync(0xffffffffu, wait(b_full + 8 * st.st, st.par, kPStageFull));
          if (ok && look) {
            const uint32_t at = base + C::kRingAt + st.st * C::kStageBytes + part * 8192 + lane * 16;
#pragma unroll 8
            for (int i = 0; i < 32; ++i) {                 // two blocks of 64 dims, 64 pages of each
              const uint4 y = ld_shared_v4(at + (i >> 4) * C::kBlock + (i & 15) * 512);
              most = choose::largest2<T>(most, y.x);
              most2 = choose::largest2<T>(most2, y.y);
              most = choose::largest2<T>(most, y.z);
              most2 = choose::largest2<T>(most2, y.w);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(b_empty + 8 * st.st);
          ring_next(st, C::kStages);
        }
        if (!look) continue;
        most = choose::largest2<T>(most, most2);
        most = __reduce_max_sync(0xffffffffu, max(most & 0xffffu, most >> 16));   // (as bits: NaN above all)
        const int32_t at = (x.tile0 + j) * 2 + part;
        if (lane == 0 && at < p.bound_tiles)
          p.largest[(static_cast<int64_t>(x.req) * p.n_kvheads + x.kvh) * p.bound_tiles + at] = choose::floats_of<T>(most).x;
      }
      if (!ok) break;
    }
    finish_role();
    return;
  } else if (warp == C::kSchedulerWarp) {
    // ------------------------------------------------------------ scheduler
    uint32_t it = 0;
    auto put = [&](const Item& x) -> bool {
      const uint32_t r = it % C::kRecords;
      if (it >= C::kRecords && !__all_sync(0xffffffffu, wait(b_recempty + 8 * r, it / C::kRecords - 1, kPRecEmpty))) return false;
      if (lane == 0) {
        int4* const to = reinterpret_cast<int4*>(recs + r);
        to[0] = make_int4(x.tiles, x.tile0, x.req, x.kvh);
        to[1] = make_int4(x.row0, x.tokens, x.pages, x.flags);
        mbar_arrive(b_recfull + 8 * r);
      }
      __syncwarp();
      ++it;
      return true;
    };
    bool ok = !p.stall_first_item;
    for (int64_t n = blockIdx.x; n < p.n_items && ok; n += gridDim.x) {
      const int32_t run = static_cast<int32_t>(n) / p.units, unit = static_cast<int32_t>(n) - run * p.units;
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
      x.flags = (r0 + t0 + x.tokens == r1 ? kLastRows : 0) | (run == 0 ? kFirstRun : 0);
      const int64_t p_last = kv - (r1 - r0) + t0 + x.tokens - 1;
      if (p_last < 0) continue;
      const int32_t own = p.pa.page_shift >= 0 ? static_cast<int32_t>(p_last >> p.pa.page_shift)
                                               : static_cast<int32_t>(p_last) / p.pa.page_size;   // (p_last < kv)
      x.pages = min(own + 1, p.pa.pages_per_req);
      if (x.pages <= p.n_select) continue;                 // all of them are chosen
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
  }
  // -------------------------------------------------------------- gathers: four warps a stage, each 32 of the pages
  constexpr int kGroups = C::kGatherWarps / C::kStageWarps;
  const int gw = warp - C::kGatherWarp0, part = gw % C::kStageWarps;
  uint32_t n = gw / C::kStageWarps, tile = 0, it = 0, issued = 0;   // stages: n, n + kGroups ..; tiles so far; items
  Item y{};                                                // of the next tile
  int k = 0;
  bool more = next(it, y), stop = false;
  if (lane == 0) prefetch_tmap(&tmB);
  // the page id of this lane's page in tile t of item z, or -1
  auto look_up = [&](const Item& z, int t) -> int32_t {
    const int32_t e = (z.tile0 + t) * kScoreTile + part * 32 + lane;
    const int32_t id = e < z.pages ? __ldg(p.pa.page_table + static_cast<int64_t>(z.req) * p.pa.pages_per_req + e) : -1;
    return id < p.pa.n_pages ? id : -1;
  };
  int32_t id_next = more ? look_up(y, 0) : -1;
  const int32_t past = static_cast<int32_t>(p.pa.n_pages) * p.n_kvheads;   // (the row past the end: zeros)
  while (!stop && more) {
    // this tile's ids are here; the next tile's are on their way while it is gathered
    const int32_t id = id_next, kvh = y.kvh;
    if (++k >= y.tiles) {
      k = 0;
      more = next(++it, y);
    }
    if (more) id_next = look_up(y, k);
    const uint32_t exist = __ballot_sync(0xffffffffu, id >= 0);
    const int32_t row = id >= 0 ? id * p.n_kvheads + kvh : past;
    int32_t r[4];                                          // lanes 0-7 and 8-15: the four pages of each gather
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __shfl_sync(0xffffffffu, row, (lane & 7) * 4 + i);
    for (; n < (tile + 1) * C::kPer; n += kGroups) {
      const uint32_t s = n % C::kStages;
      if (n >= C::kStages && !__all_sync(0xffffffffu, wait(b_empty + 8 * s, n / C::kStages - 1, kPStageEmpty))) {
        stop = true;
        break;
      }
      if (lane == 0) {
        here[(tile % C::kSlots) * 4 + part] = exist;       // (each group writes the same)
        mbar_arrive_expect_tx(b_full + 8 * s, C::kStageBytes / C::kStageWarps);
      }
      __syncwarp();
      if (lane < 16) {
        const int block = lane >> 3;
        tma_gather4(base + C::kRingAt + s * C::kStageBytes + block * C::kBlock + part * 4096 + (lane & 7) * 512, &tmB,
                    static_cast<int32_t>(n - tile * C::kPer) * 128 + block * 64, r[0], r[1], r[2], r[3], b_full + 8 * s);
      }
      issued = n + 1;
    }
    ++tile;
  }
  if (issued > 0 && lane == 0 && (stop || *abort_flag)) {
    // this warp's copies that may still be in flight: of the last ring
    const uint32_t last = issued - 1;
    for (uint32_t m = last; last - m < static_cast<uint32_t>(C::kStages); m -= kGroups) {
      drain(b_full + 8 * (m % C::kStages), (m / C::kStages) & 1, status, kDrainNs / 100);
      if (m < static_cast<uint32_t>(kGroups)) break;
    }
  }
  __syncwarp();
  finish_role();
}

template <int D, typename T, int QROWS>
cudaError_t launch_score_rows(const ChooseParams& p, const CUtensorMap& tb, int grid, int which, cudaStream_t stream) {
  using C = ScoreCfg<D, QROWS>;
  auto kern = page_score_kernel<D, T, QROWS>;
  const cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(kern), C::kSmem, kOptScore + which);
  if (e != cudaSuccess) return e;
  // (the register shares add up to what the block is launched with: a kernel compiled to fewer would wait for ever)
  static const int regs = [&] {
    cudaFuncAttributes a{};
    return cudaFuncGetAttributes(&a, kern) == cudaSuccess ? a.numRegs : 0;
  }();
  if (regs < C::kLaunchRegs) return cudaErrorInvalidConfiguration;
  kern<<<grid, C::kThreads, C::kSmem, stream>>>(tb, p);
  return cudaGetLastError();
}
template <int D, typename T>
cudaError_t launch_score_dim(const ChooseParams& p, const CUtensorMap& tb, int grid, int which, cudaStream_t stream) {
  return p.tile_tokens * p.group <= 32 ? launch_score_rows<D, T, 32>(p, tb, grid, 2 * which, stream)
                                       : launch_score_rows<D, T, 128>(p, tb, grid, 2 * which + 1, stream);
}

}  // namespace

cudaError_t launch_page_score(const ChooseParams& p, bool fp16, int num_sms, cudaStream_t stream) {
  const cuuint64_t d = static_cast<cuuint64_t>(p.head_dim);
  const cuuint64_t dims[2] = {2 * d, static_cast<cuuint64_t>(p.pa.n_pages) * static_cast<cuuint64_t>(p.n_kvheads)};
  const cuuint64_t strides[1] = {4 * d};
  const cuuint32_t box[2] = {64, 1};                       // (gathers of four rows; 16 bits are moved, whichever type)
  CUtensorMap tb{};
  if (encode_tensor_map(&tb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.bounds, dims, strides, box) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const int grid = static_cast<int>(p.n_items < num_sms ? p.n_items : num_sms);
  if (fp16)
    return p.head_dim == 64    ? launch_score_dim<64, __half>(p, tb, grid, 0, stream)
           : p.head_dim == 128 ? launch_score_dim<128, __half>(p, tb, grid, 1, stream)
                               : launch_score_dim<256, __half>(p, tb, grid, 2, stream);
  return p.head_dim == 64    ? launch_score_dim<64, __nv_bfloat16>(p, tb, grid, 3, stream)
         : p.head_dim == 128 ? launch_score_dim<128, __nv_bfloat16>(p, tb, grid, 4, stream)
                             : launch_score_dim<256, __nv_bfloat16>(p, tb, grid, 5, stream);
}

// Scores, then the choice by them.
cudaError_t launch_page_select(const ChooseParams& p, bool fp16, int num_sms, cudaStream_t stream) {
  const cudaError_t e = launch_page_score(p, fp16, num_sms, stream);
  if (e != cudaSuccess) return e;
  return p.head_dim == 64    ? launch_select_d64(p, fp16, num_sms, stream)
         : p.head_dim == 128 ? launch_select_d128(p, fp16, num_sms, stream)
                             : launch_select_d256(p, fp16, num_sms, stream);
}

}  // namespace qsa
