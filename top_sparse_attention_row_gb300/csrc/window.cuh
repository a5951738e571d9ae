// Attention with a sliding window and a few first tokens that stay visible, over a paged cache: prompt
// rows, prompt chunks and decode rows of one ragged batch in one kernel.
//
// Row r of request i stands at position p = kv_len - new + (r - cu[i]) and sees the positions j <= p with
// j > p - window (window 0: all of them) or j < n_sink:
//   S = scale q.k_j,  m = max S,  O = sum_j exp(S_j - m) v_j / l,  l = sum_j exp(S_j - m),  lse = m + ln l.
//
//  * One work unit is a query tile of one request and KV head -- 128 rows, the `group` query heads of
//    each of 128 / group consecutive tokens, so that every K and V row is read once for all of them.
//  * Units are dealt out in one of two ways.  Whole units: the grid has a block per unit, and the block on an
//    SM takes over the units of blocks that have not started (cluster launch control), so that the SMs stay
//    busy with units of unequal length and no counter in memory is needed.  A block holds one unit in advance,
//    and the longest of all heads go first, so that the last units go to the blocks that are free.  Equal shares: with few units for the SMs, the key tiles of all units
//    are laid end to end (each block sums the units' tiles when it starts) and cut into one equal run per block;
//    a block's first and last unit may be parts, whose normalised fp32 rows and log-sum-exps go to a workspace
//    and are joined by a second kernel.
//  * The keys a unit sees are the sinks and one range [lo, hi): both are laid side by side in a virtual
//    index v (position v below S0, v + shift from S0 on), which is cut into tiles of 128 keys.  A
//    window of 4096 costs 33 tiles whatever the context is; boxes that no row sees are not loaded.
//  * S = Q.K^T (tcgen05, M = 128 rows, N = 128 keys, both operands in shared memory) goes to one of two
//    tensor-memory buffers; the softmax overwrites it with P in 16 bits, which P.V takes as its A operand
//    from tensor memory; O stays in tensor memory (D columns).  S of tile j + 1 is issued before
//    P.V of tile j, so the tensor core works while the softmax does.
//  * Softmax: two warpgroups, each thread one row and half of the tile's keys; the two halves of a row
//    exchange their maxima through shared memory.  The running maximum is raised only when a tile
//    exceeds it by 2^8, so that O is seldom rescaled; O and l share it, the result is exact.  S, m, l and
//    O are fp32; P is rounded to 16 bits for the matrix product (half a step of a weight; see kLiftFp16 for
//    those far below the maximum), and l sums the unrounded weights.
//  * K and V are staged as 128-byte-swizzled 64-dim blocks of 128 keys in a ring that the MMA consumes in
//    the order K0 K1 V0 K2 V1 ...  Four producer warps issue TMA boxes of up to 64 keys (page sizes that
//    are multiples of 8), or gathers of four rows for other page sizes.
//  * 4-bit caches: four warps bring the codes and scales with cp.async some entries ahead into a staging
//    ring, and eight warps write them to the ring of stages as fp16: e2m1 times an e4m3 scale has six
//    significant bits, so that is exact; the caches' global scales multiply the logits and the output.
//    The MMAs run fp16 there (q is rounded to fp16, as for FP8 caches).
//  * Keys that no row of the unit sees (the rest of a page, positions that left the window, missing
//    pages) get weight 0 and V rows of zeros, so that whatever the cache holds there stays out.
//  * What bounds it.  Decode: HBM (128 rows over 1k to 8k keys, 24/2 heads of 256 dims, window 4096: 130 us, 5.7 TB/s;
//    the larger the batch the nearer).  Prompts of 256 dims: shared memory, 320 KB a tile = 2560 of ~2700 cycles,
//    where the tensor pipe needs 2048 (8192 rows at 24k, window 4096: 151 us, 1.37 PFLOP/s).  64 and 128 dims: the
//    softmax, ~2030 cycles a tile, of which the exponentials take 660, and ~6100 a unit (six requests of 1 to 2047
//    rows, 32/8 heads of 128 dims, window 1024: 57 us, 0.70 PFLOP/s).  4-bit caches: shared memory again, fp16 tiles
//    written and read (48 rows over 16k to 32k keys of 256 dims: 224 us, 2.9 TB/s of codes and scales).
//  * Every mbarrier wait is bounded (2 s, and more for very long units); a timeout records a code in the device status
//    word, all roles leave their loops, copies and MMAs in flight are drained, tensor memory is freed.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace qsa {

CUresult encode_tensor_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base,
                           const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box);

template <int D, bool FP4>
struct WinCfg {
  static constexpr int kStageDims = D < 128 ? D : 128;
  static constexpr int kNBS = kStageDims / 64;             // 64-dim blocks of a stage
  static constexpr int kSPT = D / kStageDims;              // stages of a K or V tile (one ring entry)
  static constexpr int kStageBytes = kWinTile * kStageDims * 2;
  // Rows of the query tile.  A 4-bit cache of 256 dims keeps 64: the other half of the tile's shared memory
  // holds a fourth ring stage and the copies ahead (the MMA's rows 64-127 then read other staged data, and
  // are not used).
  static constexpr int kRows = FP4 && D == 256 ? 64 : kWinTile;
  static constexpr int kQBlock = kRows * 128;              // bytes of a 64-dim block of the query tile
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kStages = FP4 ? (D == 64 ? 6 : 4) : (D == 256 ? 5 : D == 128 ? 6 : 12);
  static constexpr int kEntryBars = 16;                    // > entries in flight
  static constexpr int kRecords = 4;
  static constexpr int kBadSlots = FP4 ? 16 : 8;           // > tiles the producers may be ahead
  static constexpr int kThreads = FP4 ? 768 : 512;
  // registers per thread at launch, and after the split: softmax warpgroups; MMA and scheduler; copies; 4-bit
  // conversion
  static constexpr int kLaunchRegs = FP4 ? 80 : 128;
  static constexpr int kSoftmaxRegs = FP4 ? 128 : 168, kUtilRegs = FP4 ? 64 : 88, kProducerRegs = FP4 ? 72 : 88;
  static constexpr int kConvertRegs = 40;
  static_assert(256 * kSoftmaxRegs + 128 * (kUtilRegs + kProducerRegs) + (FP4 ? 256 * kConvertRegs : 0) <=
                    kThreads * kLaunchRegs,
                "register split within the launch's registers");
  static constexpr int kProducers = 4;
  static constexpr int kQWarps = FP4 ? 3 : 1;              // warps that write the query tile
  static constexpr int kDepth = D == 256 ? 3 : D == 128 ? 6 : 8;   // 4-bit entries staged
  static constexpr int kStaging = kWinTile * (D / 2 + D / 16);     // bytes of one
  // offsets
  static constexpr int kRing = kQBytes;
  static constexpr int kStagingAt = kRing + kStages * kStageBytes;
  static constexpr int kMaxAt = kStagingAt + (FP4 ? kDepth * kStaging : 0);   // [2][2][128] float
  static constexpr int kBadAt = kMaxAt + 2048;             // [kBadSlots][8] uint32
  static constexpr int kRecAt = kBadAt + kBadSlots * 32;   // [kRecords] Unit
  static constexpr int kBarAt = kRecAt + kRecords * 64;
  static constexpr int kTileBars = 8;                      // > tiles in flight
  // done[16] (by entry), kready[8], pvready[8], vlanded[8] (by tile), qfull, qempty, ofree, fin, next,
  // recfull/empty, staged/unstaged[kDepth] (4-bit caches)
  static constexpr int kBars = kEntryBars + 3 * kTileBars + 5 + 2 * kRecords + (FP4 ? 2 * kDepth : 0);
  static constexpr int kNextAt = (kBarAt + 8 * kBars + 15) / 16 * 16;   // answer of the launch control
  static constexpr int kShareAt = kNextAt + 16;            // Share
  static constexpr int kTagAt = kShareAt + 32;             // [kDepth] uint32 (4-bit caches)
  static constexpr int kTmemSlot = kTagAt + (FP4 ? 32 : 0);
  static constexpr int kSmem = kTmemSlot + 16;
  static_assert(kSmem <= kSmemLimit, "shared memory");
  static_assert(kStages / kSPT + 2 < kEntryBars, "entry barriers");
  static_assert(kStages / kSPT / 2 + 1 < kTileBars, "tile barriers");
  static_assert(kRows == kWinTile || FP4, "query rows");
};

namespace window_detail {

constexpr unsigned long long kDrainNs = 200000000ull;
constexpr float kRaise = 8.0f;          // log2 units by which a tile may exceed the running maximum
// Weights in fp16 are multiplied by 2^7 (l too, which lse undoes): at most 2^15 with kRaise, so that those far
// below the maximum do not fall out of fp16's range.  Below 2^-21 of the maximum they are rounded to whole 2^-31,
// below 2^-32 they are lost; unscaled, 6000 keys 18 nats below another one counted in l, but not in O.
constexpr float kLiftFp16 = 7.0f;       // (log2)
constexpr int32_t kShortUnit = 4;        // key tiles
constexpr float kLn2f = 0.6931471805599453f;
enum Site : int32_t {
  kWRecEmpty = 0x41, kWRecFull, kWQEmpty, kWQFull, kWStageEmpty, kWLanded, kWSFull, kWPvReady, kWPvDone,
  kWOFree, kWNext, kWStaged, kWUnstaged, kWDrain
};

__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Bounded wait for phase `parity` of a barrier.  False on timeout or abort.  (P: a kernel's parameters, with the limit
// and the status word.)
template <typename P>
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag, const P& p, int32_t site) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = now_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (now_ns() - t0 > p.wait_ns) {
      *abort_flag = 1;
      atomicCAS(p.status, 0, 0x100 | site);
      return false;
    }
  }
}
// Bounded wait that ignores the abort flag (copies and MMAs in flight finish before memory is given up).
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity, int32_t* status, unsigned long long ns) {
  const unsigned long long t0 = now_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (now_ns() - t0 > ns) {
      atomicCAS(status, 0, 0x100 | kWDrain);
      return;
    }
  }
}

// A work unit, written by the scheduler warp and read by every role.
struct Unit {
  int32_t tiles;       // key tiles of this unit (0: nothing to see, < 0: no more units)
  int32_t tile0;       // first of them
  int32_t req, kvh;
  int32_t part;        // slot of the partial result, -1: the unit is whole
  int32_t row0, tokens;
  int32_t p_first;     // position of the first token
  int32_t s0, shift;   // virtual index v: position v below s0, v + shift from s0 on
  int32_t lo, hi;      // positions some row sees: [lo, hi) and those below n_sink and hi
  // tiles of this unit, counted from tile0: [some0, some1) have only keys that some row sees, [all0, all1) only
  // keys that every row sees (the sinks' tiles count as neither)
  int32_t some0, some1, all0, all1;
};
static_assert(sizeof(Unit) == 64, "unit record");

__device__ __forceinline__ Unit load_unit(const Unit* u) {
  Unit r;
  const int4* s = reinterpret_cast<const int4*>(u);
  const int4 a = s[0], b = s[1], c = s[2], d = s[3];
  r.tiles = a.x; r.tile0 = a.y; r.req = a.z; r.kvh = a.w;
  r.part = b.x; r.row0 = b.y; r.tokens = b.z; r.p_first = b.w;
  r.s0 = c.x; r.shift = c.y; r.lo = c.z; r.hi = c.w;
  r.some0 = d.x; r.some1 = d.y; r.all0 = d.z; r.all1 = d.w;
  return r;
}

// Tiles before request i in the virtual tile numbering: cu / T + i leaves every request at least
// ceil(rows / T) numbers (at most one of them empty), and is increasing, so the owner of a number is
// found by search without any prefix sum of tile counts.
__device__ __forceinline__ int32_t first_tile(const WindowParams& p, int32_t i) {
  return __ldg(p.pa.cu_seqlens_q + i) / p.tile_tokens + i;
}
__device__ __forceinline__ int32_t tile_owner(const WindowParams& p, int32_t tile, int lane) {
  int32_t lo = 0, hi = p.pa.n_requests - 1;
  while (lo < hi) {
    const int32_t step = (hi - lo + 32) / 32;
    const int32_t cand = lo + lane * step;
    const uint32_t m = __ballot_sync(0xffffffffu, cand <= hi && first_tile(p, cand) <= tile);
    const int last = m ? 31 - __clz(m) : 0;
    lo = lo + last * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// The unit of virtual tile `tile`, which belongs to request `req`: all its key tiles, or tiles = -2 for a
// number without rows.  (kvh is left to the caller.)
__device__ __forceinline__ Unit make_unit(const WindowParams& p, int32_t req, int32_t tile) {
  Unit u{};
  u.req = req;
  u.part = -1;
  const int64_t r0 = __ldg(p.pa.cu_seqlens_q + req);
  int64_t r1 = __ldg(p.pa.cu_seqlens_q + req + 1);
  const int64_t kv = __ldg(p.pa.kv_lens + req);
  if (r1 > p.n_rows) r1 = p.n_rows;
  const int64_t t0 = static_cast<int64_t>(tile - (static_cast<int32_t>(r0) / p.tile_tokens + req)) * p.tile_tokens;
  if (r0 < 0 || t0 < 0 || r0 + t0 >= r1) {
    u.tiles = -2;
    return u;
  }
  const int64_t rows = r1 - r0;
  u.row0 = static_cast<int32_t>(r0 + t0);
  u.tokens = static_cast<int32_t>(rows - t0 < p.tile_tokens ? rows - t0 : p.tile_tokens);
  const int64_t p_first = kv - rows + t0;
  u.p_first = static_cast<int32_t>(p_first);
  const int64_t cap = static_cast<int64_t>(p.pa.pages_per_req) * p.pa.page_size;
  int64_t hi = p_first + u.tokens;
  if (hi > cap) hi = cap;
  if (hi < 0) hi = 0;
  int64_t lo = p.window > 0 ? p_first - p.window + 1 : 0;
  if (lo < 0) lo = 0;
  if (lo > hi) lo = hi;
  const int32_t grain = p.box > 0 ? p.box : 4;            // a power of two
  const int64_t lo_al = lo & ~static_cast<int64_t>(grain - 1);
  const int64_t sinks = p.n_sink < lo ? p.n_sink : lo;
  int64_t s0 = (sinks + grain - 1) & ~static_cast<int64_t>(grain - 1), shift = lo_al - s0;
  if (shift <= 0) {   // the sinks reach the window: one run from 0
    s0 = 0;
    shift = 0;
  }
  u.tiles = static_cast<int32_t>((hi - shift + kWinTile - 1) / kWinTile);   // hi - shift: the virtual length
  u.s0 = static_cast<int32_t>(s0);
  u.shift = static_cast<int32_t>(shift);
  u.lo = static_cast<int32_t>(lo);
  u.hi = static_cast<int32_t>(hi);
  // the window's run is v >= s0, positions from lo (every row: from the last row's) to hi (the first row's)
  const int64_t p_last = p_first + u.tokens - 1;
  int64_t lo_last = p.window > 0 ? p_last - p.window + 1 : 0;
  if (lo_last < lo) lo_last = lo;
  const int64_t run0 = lo - shift > s0 ? lo - shift : s0, all_from = lo_last - shift > run0 ? lo_last - shift : run0;
  const int64_t all_to = (p_first + 1 < hi ? p_first + 1 : hi) - shift;
  u.some0 = static_cast<int32_t>((run0 + kWinTile - 1) / kWinTile);
  u.some1 = static_cast<int32_t>((hi - shift) / kWinTile);
  u.all0 = static_cast<int32_t>((all_from + kWinTile - 1) / kWinTile);
  u.all1 = static_cast<int32_t>((all_to > 0 ? all_to : 0) / kWinTile);
  return u;
}
// Key tiles [a, b) of a unit.
__device__ __forceinline__ void cut(Unit& u, int32_t a, int32_t b) {
  u.tile0 = a;
  u.tiles = b - a;
  u.some0 -= a;
  u.some1 -= a;
  u.all0 -= a;
  u.all1 -= a;
}

// Listed units (chosen pages, shared prompts): a kernel before this one has written them, units [n_units] (in any
// order of tiles and KV heads) and their key tiles (-2: no unit).
__device__ __forceinline__ Unit listed_unit(const WindowParams& p, int32_t n) {
  Unit u = load_unit(static_cast<const Unit*>(p.units) + n);
  u.tiles = p.unit_tiles[n];
  return u;
}
// Chosen pages: a unit's keys are the positions of its pages, one page after the other (virtual index v: entry v / page
// size).  u.s0 holds their number, u.shift the unit's number.
__device__ __forceinline__ const PageEntry* unit_entries(const WindowParams& p, const Unit& u) {
  return p.entries + static_cast<int64_t>(u.shift) * p.list_cap;
}
// (a plain load: the kernel before, which writes the entries, may still run when this one starts, and only what nobody
// writes from then on may be read by non-coherent loads)
__device__ __forceinline__ PageEntry load_entry(const PageEntry* e) {
  const int4 x = *reinterpret_cast<const int4*>(e);
  return PageEntry{x.x, x.y, static_cast<uint32_t>(x.z), x.w};
}
__device__ __forceinline__ int32_t entry_of(const WindowParams& p, int32_t v) {
  return p.pa.page_shift >= 0 ? v >> p.pa.page_shift : v / p.pa.page_size;
}
// Whether some row of the unit sees key v: the last one that lists its page, if any.
__device__ __forceinline__ bool chosen_seen(const WindowParams& p, const Unit& u, int32_t v) {
  const int32_t e = entry_of(p, v);
  if (e >= u.s0) return false;
  const PageEntry x = load_entry(unit_entries(p, u) + e);
  return x.page * p.pa.page_size + (v - e * p.pa.page_size) <= u.p_first + 31 - __clz(x.rows);
}

// Equal shares: where a block's run of the units starts.  A unit counts as unit_cost for its beginning and end,
// then its tiles (at least one in all); a share that ends inside the former takes nothing of the unit.
struct Share {
  int64_t size;        // of a share, more than unit_cost
  int64_t left;        // of this block's
  int32_t kvh, tile;   // first unit
  int32_t offset;      // where the share starts in it
};
// Worked out by all threads of the block; `scratch` has room for 34 int64.  Ends with a barrier.
template <int THREADS, UnitSource SOURCE>
__device__ __forceinline__ void find_share(const WindowParams& p, int64_t* scratch, Share* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t heads = SOURCE == kWindowRows ? p.n_kvheads : 1;   // (listed units are of one head each)
  auto weight = [&](int32_t tile) -> int32_t {
    if (tile >= p.n_tiles) return 0;
    if constexpr (SOURCE != kWindowRows) {
      const int32_t t = p.unit_tiles[tile];
      return t == -2 ? 0 : max(t + p.unit_cost, 1);
    }
    int32_t lo = 0, hi = p.pa.n_requests - 1;             // the last request whose first tile is <= tile
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) >> 1;
      if (first_tile(p, mid) <= tile) lo = mid; else hi = mid - 1;
    }
    const int32_t t = make_unit(p, lo, tile).tiles;
    return t == -2 ? 0 : max(t + p.unit_cost, 1);
  };
  auto warp_sum = [&](int64_t v) -> int64_t {             // inclusive over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t w = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += w;
    }
    return v;
  };
  const int32_t w0 = weight(tid);
  int64_t mine = w0;
  for (int32_t t = tid + THREADS; t < p.n_tiles; t += THREADS) mine += weight(t);
  const int64_t in_warp = warp_sum(mine);
  if (lane == 31) scratch[warp] = in_warp;
  if (tid == 0) out->left = 0;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) total += scratch[w];
  __syncthreads();
  const int64_t all = total * heads, even = (all + p.shares - 1) / p.shares;
  const int64_t size = even > p.unit_cost ? even : p.unit_cost + 1;   // every share inside a unit has tiles of it
  const int64_t from = size * blockIdx.x;
  if (from < all) {                                       // uniform over the block
    const int32_t kvh = static_cast<int32_t>(from / total);
    const int64_t want = from - kvh * total;
    int64_t before = 0;
    for (int32_t c = 0; c < p.n_tiles; c += THREADS) {
      const int32_t w = c == 0 ? w0 : weight(c + tid);
      const int64_t incl = warp_sum(w);
      if (lane == 31) scratch[warp] = incl;
      __syncthreads();
      int64_t base = before;
#pragma unroll
      for (int k = 0; k < THREADS / 32; ++k) {
        if (k < warp) base += scratch[k];
        before += scratch[k];
      }
      if (w > 0 && base + incl - w <= want && want < base + incl) {
        out->size = size;
        out->left = size < all - from ? size : all - from;
        out->kvh = kvh;
        out->tile = c + tid;
        out->offset = static_cast<int32_t>(want - (base + incl - w));
      }
      __syncthreads();
      if (before > want) break;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int32_t position_of(const Unit& u, int32_t v) { return v >= u.s0 ? v + u.shift : v; }
__device__ __forceinline__ bool seen(const WindowParams& p, const Unit& u, int32_t pos) {
  return pos < u.hi && (pos >= u.lo || pos < p.n_sink);
}

// The ring entries of tile j of a unit with nt tiles.
__device__ __forceinline__ uint32_t k_entry(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ uint32_t v_entry(int j, int nt) { return j == nt - 1 ? 2 * j + 1 : 2 * j + 2; }
__device__ __forceinline__ uint32_t pack16(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  uint32_t r;
  memcpy(&r, &v, 4);
  return r;
}
__device__ __forceinline__ uint32_t pack16(float a, float b, __half) {
  const __half2 v = __floats2half2_rn(a, b);
  uint32_t r;
  memcpy(&r, &v, 4);
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_as_f16x2(uint32_t v) {
  const __half2 h = __floats2half2_rn(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  uint32_t r;
  memcpy(&r, &h, 4);
  return r;
}
// Two floats at a time (one instruction each).
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split_pair(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// One 32-byte store (the address is a multiple of 32).
__device__ __forceinline__ void st_global_v8(uint32_t* to, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
template <int N>
__device__ __forceinline__ void cp_async_zfill(uint32_t dst, const void* src, bool ok) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(ok ? N : 0)
                 : "memory");
}
// Arrives on `bar` once this thread's earlier cp.async copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// Two e2m1 codes (byte `k` of w) as fp16, times a pair of equal scales: exact.
__device__ __forceinline__ uint32_t e2m1_scaled(uint32_t w, int k, __half2 s) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3, c;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
      : "=r"(r)
      : "r"(w >> (8 * k)));
  __half2 h;
  memcpy(&h, &r, 4);
  h = __hmul2(h, s);
  memcpy(&r, &h, 4);
  return r;
}

}  // namespace window_detail

template <int D, typename T, bool FP4, UnitSource SOURCE>
__global__ void __launch_bounds__(WinCfg<D, FP4>::kThreads, 1)
    window_attention_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                            const __grid_constant__ CUtensorMap tmQ1, const __grid_constant__ CUtensorMap tmQT,
                            const __grid_constant__ WindowParams p) {
  using namespace window_detail;
  using C = WinCfg<D, FP4>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  // Ring entry e's MMAs are done (so its stages are free, and S of a K entry or O up to a V entry can be
  // read): at e % kEntryBars.  By tile, at tile % kTileBars: K is staged; V is staged and P written (one
  // wait for the P.V); V of a tile with unseen keys has landed and can be zeroed.
  const uint32_t b_done = base + C::kBarAt;
  const uint32_t b_kready = b_done + 8 * C::kEntryBars;
  const uint32_t b_pvready = b_kready + 8 * C::kTileBars;
  const uint32_t b_vlanded = b_pvready + 8 * C::kTileBars;
  const uint32_t b_qfull = b_vlanded + 8 * C::kTileBars;
  const uint32_t b_qempty = b_qfull + 8;
  const uint32_t b_ofree = b_qempty + 8;
  const uint32_t b_fin = b_ofree + 8;
  const uint32_t b_next = b_fin + 8;
  const uint32_t b_recfull = b_next + 8;
  const uint32_t b_recempty = b_recfull + 8 * C::kRecords;
  const uint32_t b_staged = b_recempty + 8 * C::kRecords;      // 4-bit caches: an entry's copies are staged, converted
  const uint32_t b_unstaged = b_staged + 8 * C::kDepth;
  float* const maxima = reinterpret_cast<float*>(smem + C::kMaxAt);
  uint32_t* const bad_keys = reinterpret_cast<uint32_t*>(smem + C::kBadAt);
  uint32_t* const tags = reinterpret_cast<uint32_t*>(smem + C::kTagAt);   // 4-bit caches: of the staged entries
  constexpr uint32_t kLastTag = 0xffffffffu;
  Unit* const recs = reinterpret_cast<Unit*>(smem + C::kRecAt);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kTmemSlot);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* const status = p.status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if ((base & 1023u) != 0) {   // the swizzle needs 1024-byte aligned tiles; uniform over the grid
    if (threadIdx.x == 0) {
      atomicCAS(status, 0, 0x100 | kWDrain);
      if (SOURCE != kSharedPrefix && p.shares > 0) p.joins[blockIdx.x] = JoinRecord{-1, 0, 0, 0, 0, 0, 0, 0};
    }
    return;
  }
  if (threadIdx.x == 0) {
    constexpr int kArrivals = FP4 ? 8 : C::kProducers * C::kSPT;   // of the warps that stage an entry
    for (int e = 0; e < C::kEntryBars; ++e) mbar_init(b_done + 8 * e, 1);
    for (int t = 0; t < C::kTileBars; ++t) {
      mbar_init(b_kready + 8 * t, kArrivals);
      mbar_init(b_pvready + 8 * t, kArrivals + 8);                 // and the softmax warps
      mbar_init(b_vlanded + 8 * t, kArrivals);
    }
    mbar_init(b_qfull, C::kQWarps);
    mbar_init(b_qempty, 1);
    mbar_init(b_ofree, 8);
    mbar_init(b_fin, 1);
    mbar_init(b_next, 1);
    for (int r = 0; r < C::kRecords; ++r) {
      mbar_init(b_recfull + 8 * r, 1);
      mbar_init(b_recempty + 8 * r, 8 + 1 + C::kProducers + 2);   // and warps 10 and 11
    }
    if constexpr (FP4) {
      for (int k = 0; k < C::kDepth; ++k) {
        mbar_init(b_staged + 8 * k, 128 + 1);                      // and the one that writes the tag
        mbar_init(b_unstaged + 8 * k, 8);
      }
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (!FP4 && warp == 12 && lane == 0) {
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    prefetch_tmap(&tmQ1);
    prefetch_tmap(&tmQT);
  }
  Share* const share = reinterpret_cast<Share*>(smem + C::kShareAt);
  if constexpr (SOURCE != kWindowRows) pdl_wait();   // the units are written, and what came before them
  if (p.shares > 0) find_share<C::kThreads, SOURCE>(p, reinterpret_cast<int64_t*>(smem + C::kMaxAt), share);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();                    // the join's launch overlaps (it waits for this grid's end)
  const uint32_t tmem = *tmem_slot;
  const uint32_t tm_o = tmem + 256;           // S buffers: columns 0-127 and 128-255; O: from 256

  auto wait_done = [&](uint32_t e, int32_t site) -> bool {
    return wait_for(b_done + 8 * (e % C::kEntryBars), (e / C::kEntryBars) & 1, abort_flag, p, site);
  };
  auto wait_tile = [&](uint32_t bars, uint32_t t, int32_t site) -> bool {
    return wait_for(bars + 8 * (t % C::kTileBars), (t / C::kTileBars) & 1, abort_flag, p, site);
  };
  auto finish_role = [&]() {
    tc_fence_before();
    __syncthreads();
  };

  if (warp < 8) {
    // ------------------------------------------------------------ softmax + epilogue
    regs_inc<C::kSoftmaxRegs>();
    const int wg = warp >> 2, w = warp & 3, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
    const float sc = p.scale_log2;
    const float raise = kRaise / sc;
    constexpr int kPart0 = SOURCE == kSharedPrefix ? 2 : 0;   // (see shared_unit)
    constexpr float kLift = FP4 || std::is_same<T, __half>::value ? kLiftFp16 : 0.0f;
    // (loops that run once a unit, or seldom, are not unrolled: their instructions would have to be fetched anew each
    // time)
    uint32_t it = 0, js = 0, eb = 0;          // records, tiles and ring entries so far
    bool bad = false;
    for (;; ++it) {
      const uint32_t rb = it % C::kRecords;
      bad |= !wait_for(b_recfull + 8 * rb, (it / C::kRecords) & 1, abort_flag, p, kWRecFull);
      // the two warps that share 32 rows leave together or not at all
      if (named_bar_any(1 + w, 64, bad || *abort_flag)) break;
      const Unit u = load_unit(recs + rb);
      __syncwarp();
      if (lane == 0) mbar_arrive(b_recempty + 8 * rb);
      if (u.tiles < 0) break;
      const int live_rows = u.tokens * p.group;
      const bool warp_live = w * 32 < live_rows;
      const int tok = row / p.group;
      const int32_t pos = u.p_first + tok;    // of this thread's row
      // positions this row sees: [row_lo, pos] and those below row_sink
      int32_t row_lo = SOURCE == kSharedPrefix ? u.lo : p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
      int32_t row_sink = min(p.n_sink, pos + 1);
      if (pos < 0) {
        row_lo = INT32_MAX;
        row_sink = 0;
      }
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < u.tiles; ++j) {
        const uint32_t jt = js + j, sb = jt & 1;
        const uint32_t tm_s = tmem + lanes + sb * 128 + wg * 64;
        const int32_t v0 = (u.tile0 + j) * kWinTile;
        // chosen pages: those that this half of the tile lies in (at most 8: whole 8s of keys), one a lane
        PageEntry mine{0, 0, 0, 0};
        const int32_t e0 = SOURCE == kChosenPages ? entry_of(p, v0 + wg * 64) : 0;
        if constexpr (SOURCE == kChosenPages) {
          if (lane < 8 && e0 + lane < u.s0) mine = load_entry(unit_entries(p, u) + e0 + lane);
        }
        bad |= !wait_done(eb + k_entry(j), kWSFull);
        tc_fence_after();
        const uint32_t* const holes = bad_keys + (jt % C::kBadSlots) * 8;
        bool any_hole = false;
        if constexpr (SOURCE != kChosenPages) {
          const uint4 h0 = *reinterpret_cast<const uint4*>(holes), h1 = *reinterpret_cast<const uint4*>(holes + 4);
          any_hole = (h0.x | h0.y | h0.z | h0.w | h1.x | h1.y | h1.z | h1.w) != 0;
        }
        if (warp_live) {
          float s[64];
          tmem_ld32(tm_s, s);
          tmem_ld32(tm_s + 32, s + 32);
          tc_wait_ld();
          // chosen pages: which sixteens of the columns some row of the warp sees (the tile's pages are those of all its
          // tokens, a warp's rows are of a few): the others are left out below, their weights are 0
          uint32_t live = 15u;
          if (j < u.all0 || j >= u.all1 || any_hole) {
            // the keys of this thread's half that its row sees, as bits
            const int32_t c0 = v0 + wg * 64;
            uint64_t keep = 0;
            if constexpr (SOURCE == kChosenPages) {
#pragma unroll 1
              for (int i = 0; i < 8; ++i) {
                const int32_t from = (e0 + i) * p.pa.page_size - c0;          // of the page's keys in this half
                if (from >= 64 || e0 + i >= u.s0) break;
                const int32_t page = __shfl_sync(0xffffffffu, mine.page, i);
                const uint32_t rows = __shfl_sync(0xffffffffu, mine.rows, i);
                const int32_t n = rows >> (tok & 31) & 1u ? min(pos + 1 - page * p.pa.page_size, p.pa.page_size) : 0;
                const int32_t a = max(from, 0), b = min(from + n, 64);
                if (b > a) keep |= (~0ull >> (64 - (b - a))) << a;
              }
            } else {
              const int32_t c_lo = row_lo == INT32_MAX ? 64 : max(max(row_lo - u.shift, u.s0) - c0, 0);
              const int32_t c_hi = pos >= 0 ? min(min(pos, u.hi - 1) - u.shift - c0, 63) : -1;
              const int32_t c_sink = min(min(row_sink, u.hi) - c0, 64);
              keep = c_sink >= 64 ? ~0ull : c_sink > 0 ? (1ull << c_sink) - 1 : 0ull;
              if (c_lo <= c_hi) keep |= (~0ull >> (63 - c_hi)) & (~0ull << c_lo);
            }
            if (any_hole) {
#pragma unroll 1
              for (int c = 0; c < 64; ++c) {
                const int key = wg * 64 + c;
                int word, bit;
                if constexpr (FP4) {
                  word = key >> 4;
                  bit = key & 15;
                } else if (p.box > 0) {
                  const int o = key / p.box * C::kNBS;
                  word = (o & 3) * 2;
                  bit = o >> 2;
                } else {
                  const int o = (key >> 2) * C::kNBS;
                  word = (o & 3) * 2 + ((key & 3) >> 1);
                  bit = (key & 1) * 16 + (o >> 2);
                }
                if ((holes[word] >> bit) & 1) keep &= ~(1ull << c);
              }
            }
            const uint32_t k0 = static_cast<uint32_t>(keep), k1 = static_cast<uint32_t>(keep >> 32);
            if constexpr (SOURCE == kChosenPages) {
              const uint32_t a0 = __reduce_or_sync(0xffffffffu, k0), a1 = __reduce_or_sync(0xffffffffu, k1);
              live = (a0 & 0xffffu ? 1u : 0u) | (a0 >> 16 ? 2u : 0u) | (a1 & 0xffffu ? 4u : 0u) | (a1 >> 16 ? 8u : 0u);
            }
#pragma unroll
            for (int h = 0; h < 64; h += 16) {
              if (SOURCE == kChosenPages && !(live >> (h / 16) & 1u)) continue;
#pragma unroll
              for (int c = h; c < h + 16; ++c) s[c] = (h < 32 ? k0 : k1) & (1u << (c & 31)) ? s[c] : -INFINITY;
            }
          }
          float t0 = -INFINITY, t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
#pragma unroll
          for (int h = 0; h < 64; h += 16) {
            if (SOURCE == kChosenPages && !(live >> (h / 16) & 1u)) continue;
#pragma unroll
            for (int c = h; c < h + 16; c += 4) {
              t0 = fmaxf(t0, s[c]);
              t1 = fmaxf(t1, s[c + 1]);
              t2 = fmaxf(t2, s[c + 2]);
              t3 = fmaxf(t3, s[c + 3]);
            }
          }
          float tile_max = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3));
          float* const mx = maxima + sb * 256;
          mx[wg * 128 + row] = tile_max;
          // (a warp whose wait ran out stays in step until the unit's end, so this barrier needs no vote)
          named_bar_sync(1 + w, 64);
          tile_max = fmaxf(tile_max, mx[(wg ^ 1) * 128 + row]);
          // (rows past the unit's hold anything: they must not make the warp rescale)
          const bool need = row < live_rows && (tile_max > m + raise || (m == -INFINITY && tile_max > -INFINITY));
          if (__any_sync(0xffffffffu, need)) {
            const float nm = need ? tile_max : m;
            const float f = m == -INFINITY ? 0.0f : fast_exp2((m - nm) * sc);
            if (j > 0) {
              bad |= !wait_done(eb + v_entry(j - 1, u.tiles), kWPvDone);
              tc_fence_after();
              const float g = need ? f : 1.0f;
#pragma unroll 1
              for (int c = 0; c < D / 2; c += 16) {
                float o[16];
                tmem_ld16(tm_o + lanes + wg * (D / 2) + c, o);
                tc_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] *= g;
                tmem_st16(tm_o + lanes + wg * (D / 2) + c, o);
              }
            }
            if (need) {
              l *= f;
              m = nm;
            }
          }
          const float neg = m == -INFINITY ? 0.0f : kLift - m * sc;
          const uint64_t sc2 = pair_of(sc, sc), neg2 = pair_of(neg, neg);
          uint64_t a0 = 0, a1 = 0;                 // sums of pairs
          uint32_t pk[32];
#pragma unroll
          for (int h = 0; h < 64; h += 16) {
            if (SOURCE == kChosenPages && !(live >> (h / 16) & 1u)) {
#pragma unroll
              for (int c = h; c < h + 16; c += 2) pk[c / 2] = 0u;
              continue;
            }
#pragma unroll
            for (int c = h; c < h + 16; c += 4) {
              float e0, e1, e2, e3;
              split_pair(fma_pair(pair_of(s[c], s[c + 1]), sc2, neg2), e0, e1);
              split_pair(fma_pair(pair_of(s[c + 2], s[c + 3]), sc2, neg2), e2, e3);
              e0 = fast_exp2(e0);
              e1 = fast_exp2(e1);
              e2 = fast_exp2(e2);
              e3 = fast_exp2(e3);
              a0 = add_pair(a0, pair_of(e0, e1));
              a1 = add_pair(a1, pair_of(e2, e3));
              if constexpr (FP4) {
                pk[c / 2] = pack16(e0, e1, __half{});
                pk[c / 2 + 1] = pack16(e2, e3, __half{});
              } else {
                pk[c / 2] = pack16(e0, e1, T{});
                pk[c / 2 + 1] = pack16(e2, e3, T{});
              }
            }
          }
          float l0, l1;
          split_pair(add_pair(a0, a1), l0, l1);
          l += l0 + l1;
          tmem_st32(tm_s, pk);
          tc_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_pvready + 8 * (jt % C::kTileBars));
      }
      // epilogue
      if (u.tiles > 0) {
        bad |= !wait_done(eb + 2 * u.tiles - 1, kWPvDone);
        tc_fence_after();
      }
      if (warp_live) {
        // the two halves' sums; the buffer of the other parity than the last tile's maxima
        float* const mx = maxima + ((js + u.tiles) & 1) * 256;
        mx[wg * 128 + row] = l;
        if (named_bar_any(1 + w, 64, bad)) break;
        l += mx[(wg ^ 1) * 128 + row];
      }
      const bool store = row < live_rows;
      const int64_t token = static_cast<int64_t>(u.row0) + tok;
      const int32_t head = u.kvh * p.group + (row - tok * p.group);
      const int64_t rh = token * p.n_qheads + head;
      const bool empty = l == 0.0f && m == -INFINITY;
      const float inv = empty ? 0.0f : p.v_mult / l;
      if (store && wg == 0) {
        constexpr float kUnlift = kLift > 0.0f ? 0x1p-7f : 1.0f;
        const float lse = empty ? -INFINITY : m * sc * kLn2f + logf(l * kUnlift);
        if (SOURCE == kSharedPrefix && u.part >= 0 && u.part < 2) p.first_lse[u.part * p.n_rows * p.n_qheads + rh] = lse;
        else if (u.part >= 0) p.part_lse[(u.part - kPart0) * kWinTile + row] = lse;
        else if (p.lse) p.lse[rh] = lse;
      }
      const uint32_t tm_row = tm_o + lanes + wg * (D / 2);
      if (warp_live && u.part >= 0) {
        float* const part = (SOURCE == kSharedPrefix && u.part < 2
                                 ? p.first_o + (u.part * p.n_rows * p.n_qheads + rh) * D
                                 : p.part_o + static_cast<int64_t>((u.part - kPart0) * kWinTile + row) * D) + wg * (D / 2);
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 32) {
          if (u.tiles == 0) break;
          float o[32];
          tmem_ld32(tm_row + c, o);
          tc_wait_ld();
          if (store && !empty) {
            uint32_t v[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(o[k] * inv);
#pragma unroll
            for (int k = 0; k < 32; k += 8) st_global_v8(reinterpret_cast<uint32_t*>(part) + c + k, v + k);
          }
        }
      }
      if (warp_live && u.part < 0) {
        uint32_t* const out = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + rh * D + wg * (D / 2));
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 32) {
          float o[32];
          if (u.tiles > 0) {
            tmem_ld32(tm_row + c, o);
            tc_wait_ld();
          }
          uint32_t v[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = empty ? 0u : pack16(o[2 * k] * inv, o[2 * k + 1] * inv, T{});
          if (!store) continue;
          // a thread writes its own row: 32-byte stores fill whole sectors
          if (p.out_32) {
            st_global_v8(out + c / 2, v);
            st_global_v8(out + c / 2 + 8, v + 8);
          } else {
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              *reinterpret_cast<uint4*>(out + c / 2 + k) = make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
          }
        }
      }
      if (u.tiles > 0) {      // O may be overwritten
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_ofree);
      }
      js += u.tiles;
      eb += 2 * u.tiles;
    }
    finish_role();
    return;
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer, tensor-memory owner
    regs_dec<C::kUtilRegs>();
    constexpr bool kF16 = FP4 || std::is_same<T, __half>::value;
    constexpr uint32_t kIdescQK = kF16 ? idesc_f16_f32(128, 128, false, false) : idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t kIdescPV = kF16 ? idesc_f16_f32(128, C::kStageDims, false, true)
                                       : idesc_bf16_f32(128, C::kStageDims, false, true);
    constexpr uint32_t kIdescPV2 = kF16 ? idesc_f16_f32(128, 256, false, true) : idesc_bf16_f32(128, 256, false, true);
    constexpr uint32_t kHi = sw128_desc_hi(1024);
    const uint32_t q_lo = sw128_desc_lo(base, 16);
    const uint32_t k_lo = sw128_desc_lo(base + C::kRing, 16);
    const uint32_t v_lo = sw128_desc_lo(base + C::kRing, 16384);
    uint32_t st = 0, entry = 0, js = 0, qit = 0;
    bool stop = false;
    // the stages of the next entry; st moves past them
    auto take_stages = [&](uint32_t* stage) {
#pragma unroll
      for (int h = 0; h < C::kSPT; ++h) {
        stage[h] = st;
        if (++st == C::kStages) st = 0;
      }
    };
    auto issue_qk = [&](uint32_t jt, bool last) -> bool {
      uint32_t stage[C::kSPT];
      take_stages(stage);
      if (!__all_sync(0xffffffffu, wait_tile(b_kready, jt, kWLanded))) return false;
      tc_fence_after();
      if (lane == 0) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int h = kk / (C::kStageDims / 16), kq = kk % (C::kStageDims / 16);
          const uint32_t b_off = (kq >> 2) * 16384 + (kq & 3) * 32;
          const uint32_t a_off = (kk >> 2) * C::kQBlock + (kk & 3) * 32;
          tc_mma_w(tmem + (jt & 1) * 128, q_lo + (a_off >> 4), kHi,
                   k_lo + stage[h] * (C::kStageBytes >> 4) + (b_off >> 4), kHi, kIdescQK, kk > 0 ? 1u : 0u);
        }
        tc_commit(b_done + 8 * (entry % C::kEntryBars));
        if (last) tc_commit(b_qempty);
      }
      __syncwarp();
      ++entry;
      return true;
    };
    for (uint32_t it = 0;; ++it) {
      const uint32_t rb = it % C::kRecords;
      if (!__all_sync(0xffffffffu, wait_for(b_recfull + 8 * rb, (it / C::kRecords) & 1, abort_flag, p,
                                            kWRecFull))) {
        stop = true;
        break;
      }
      const int nt = recs[rb].tiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(b_recempty + 8 * rb);
      if (nt < 0) break;
      if (nt == 0) continue;
      if (!__all_sync(0xffffffffu, wait_for(b_qfull, qit & 1, abort_flag, p, kWQFull))) {
        stop = true;
        break;
      }
      if (!issue_qk(js, nt == 1)) {
        stop = true;
        break;
      }
      for (int j = 0; j < nt; ++j) {
        const uint32_t jt = js + j;
        if (j + 1 < nt && !issue_qk(jt + 1, j + 2 == nt)) {
          stop = true;
          break;
        }
        uint32_t stage[C::kSPT];
        take_stages(stage);
        bool ok = wait_tile(b_pvready, jt, kWPvReady);
        if (j == 0) ok = ok && wait_for(b_ofree, (qit & 1) ^ 1, abort_flag, p, kWOFree);
        if (!__all_sync(0xffffffffu, ok)) {
          stop = true;
          break;
        }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t a0 = tmem + (jt & 1) * 128;
          if (C::kSPT == 2 && stage[0] + 1 == stage[C::kSPT - 1]) {
            // both halves of the dims lie one after the other: one MMA of N = 256 per 16 keys
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t a = a0 + (kk < 4 ? kk * 8 : 64 + (kk - 4) * 8);
              tc_mma_ta(tm_o, a, v_lo + stage[0] * (C::kStageBytes >> 4) + kk * (2048 >> 4), kHi, kIdescPV2,
                        j > 0 || kk > 0 ? 1u : 0u);
            }
          } else {
#pragma unroll
            for (int h = 0; h < C::kSPT; ++h) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                const uint32_t a = a0 + (kk < 4 ? kk * 8 : 64 + (kk - 4) * 8);
                tc_mma_ta(tm_o + h * 128, a, v_lo + stage[h] * (C::kStageBytes >> 4) + kk * (2048 >> 4), kHi,
                          kIdescPV, j > 0 || kk > 0 ? 1u : 0u);
              }
            }
          }
          tc_commit(b_done + 8 * (entry % C::kEntryBars));
        }
        __syncwarp();
        ++entry;
      }
      if (stop) break;
      js += nt;
      ++qit;
    }
    if (lane == 0) {
      tc_commit(b_fin);
      drain(b_fin, 0, status, stop ? kDrainNs : kWinWaitNs);
    }
    __syncwarp();
    finish_role();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
    return;
  } else if (warp < 12) {
    // ------------------------------------------------------------ scheduler (warp 9), query tile; warps 10
    // and 11: zero V rows (16-bit caches), a share of the query tile (4-bit caches)
    regs_dec<C::kUtilRegs>();
    if (!FP4 && warp > 9) {
      uint32_t js = 0, st0 = 0;          // tiles so far, the first stage of the next entry
      for (uint32_t it = 0;; ++it) {
        const uint32_t rb = it % C::kRecords;
        if (!__all_sync(0xffffffffu, wait_for(b_recfull + 8 * rb, (it / C::kRecords) & 1, abort_flag, p,
                                              kWRecFull)))
          break;
        const Unit u = load_unit(recs + rb);
        __syncwarp();
        if (lane == 0) mbar_arrive(b_recempty + 8 * rb);
        if (u.tiles < 0) break;
        bool ok = true;
        for (int j = 0; j < u.tiles; ++j) {
          // V of these tiles lands on this barrier, in every other tile the producers' copies do so on the
          // MMA's; a barrier per tile keeps its phases apart only if each is waited for, so whole tiles are
          // signed off by the producers here too
          const uint32_t jt = js + j;
          ok = __all_sync(0xffffffffu, wait_tile(b_vlanded, jt, kWLanded));
          if (!ok) break;
          if (j >= u.some0 && j < u.some1) continue;
          const uint32_t e = v_entry(j, u.tiles);
          for (int k = 0; k < kWinTile / 64; ++k) {
            const int row = k * 64 + (warp - 10) * 32 + lane;
            const int32_t v = (u.tile0 + j) * kWinTile + row;
            if (SOURCE == kChosenPages ? chosen_seen(p, u, v) : seen(p, u, position_of(u, v))) continue;
#pragma unroll
            for (int b = 0; b < D / 64; ++b) {
              const uint32_t st = (st0 + e * C::kSPT + b / C::kNBS) % C::kStages;
              const uint32_t at = base + C::kRing + st * C::kStageBytes + (b % C::kNBS) * 16384 + row * 128;
#pragma unroll
              for (int c = 0; c < 8; ++c) st_shared_v4(at + ((c ^ lane) & 7) * 16, make_uint4(0u, 0u, 0u, 0u));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          // in place of the producers' arrivals
          if (lane < C::kProducers * C::kSPT / 2) mbar_arrive(b_pvready + 8 * (jt % C::kTileBars));
        }
        if (!ok) break;
        js += u.tiles;
        st0 = (st0 + 2 * u.tiles * C::kSPT) % C::kStages;
      }
      finish_role();
      return;
    }
    uint32_t qit = 0;
    // Units: this block's own, then those of blocks that have not started.  The next one is asked for when the
    // softmax begins the present one, so that a block holds one unit in advance and the last units go to the
    // blocks that are free; after a short unit at once, so that its successor's loads need not wait.
    int32_t n = blockIdx.x, last_tiles = 0;
    uint32_t asked = 0;
    bool more = true;                        // no answer has said "none" yet
    auto ask = [&]() {
      if (lane == 0) {
        mbar_arrive_expect_tx(b_next, 16);
        clc_try_cancel(base + C::kNextAt, b_next);
      }
      __syncwarp();
    };
    auto answer = [&]() -> int32_t {
      const bool ok = mbar_try_wait(b_next, asked & 1) || wait_for(b_next, asked & 1, abort_flag, p, kWNext);
      ++asked;
      if (!__all_sync(0xffffffffu, ok)) {
        more = false;
        return -1;
      }
      const int32_t x = clc_answer(base + C::kNextAt);
      fence_proxy_async_smem();              // the next answer is written by the async proxy
      __syncwarp();
      more = x >= 0;
      return x;
    };
    // whole units: number n of the call.  A request's later tiles see more keys where there is no window: they go
    // first, of all heads
    auto whole_unit = [&](uint32_t n) -> Unit {
      if constexpr (SOURCE != kWindowRows) return listed_unit(p, p.n_tiles - 1 - static_cast<int32_t>(n));
      const uint32_t back = n / static_cast<uint32_t>(p.n_kvheads), kvh = n - back * static_cast<uint32_t>(p.n_kvheads);
      const int32_t tile = p.n_tiles - 1 - static_cast<int32_t>(back);
      Unit u = make_unit(p, tile_owner(p, tile, lane), tile);
      u.kvh = static_cast<int32_t>(kvh);
      return u;
    };
    // equal shares: the next unit of this block's run, whole or a part
    Share sh = *share;
    int64_t at = p.shares > 0 ? sh.size * blockIdx.x : 0;
    bool first_unit = true;
    JoinRecord join{-1, 0, 0, 0, 0, 0, 0, 0};
    // A unit's part goes to slot 2 block + {0, 1}, in the order in which the block has them.  Shared prompts: a row has
    // results of two units to be joined, so whole units are parts too (u.part as listed: 0 the prompt's, 1 the
    // request's own keys, by row and head, or -1 if there is but one), a first part goes to the same place, and one
    // that continues a unit of an earlier block to slot 2 + block.
    auto shared_unit = [&]() -> Unit {
      Unit u{};
      u.tiles = -1;
      const int32_t heads = SOURCE == kWindowRows ? p.n_kvheads : 1;
      while (sh.left > 0 && sh.kvh < heads) {
        const int32_t tile = sh.tile;
        if constexpr (SOURCE == kWindowRows) {
          u = make_unit(p, tile_owner(p, tile, lane), tile);
          u.kvh = sh.kvh;
        } else {
          u = listed_unit(p, tile);
        }
        if (++sh.tile == p.n_tiles) {
          sh.tile = 0;
          ++sh.kvh;
        }
        if (u.tiles == -2) {
          u.tiles = -1;
          continue;
        }
        const int32_t w = max(u.tiles + p.unit_cost, 1), off = sh.offset;
        sh.offset = 0;
        if (off >= w) {         // (row offsets that do not increase)
          u.tiles = -1;
          continue;
        }
        const int32_t take = sh.left < w - off ? static_cast<int32_t>(sh.left) : w - off;
        const int64_t end = at - off + w;
        const int32_t a = off > p.unit_cost ? off - p.unit_cost : 0, b = off + take - p.unit_cost;
        sh.left -= take;
        at += take;
        if (u.tiles == 0 ? off > 0 : b <= a) {
          u.tiles = -1;
          continue;
        }
        if constexpr (SOURCE == kSharedPrefix) {
          const bool goes_on = u.tiles > 0 && b < u.tiles;
          if (a > 0) u.part = 2 + static_cast<int32_t>(blockIdx.x);
          else if (goes_on && u.part < 0) u.part = 1;
          if (a == 0 && lane == 0)
            p.unit_joins[tile] = make_int2(static_cast<int32_t>(blockIdx.x),
                                           goes_on ? static_cast<int32_t>((end - 1) / sh.size - blockIdx.x) : 0);
          if (u.tiles > 0) cut(u, a, b);
        } else if (u.tiles > 0 && b - a < u.tiles) {
          u.part = static_cast<int32_t>(2 * blockIdx.x) + (first_unit ? 0 : 1);
          if (a == 0) {         // its later parts are the first ones of the blocks that follow
            int64_t last = (end - 1) / sh.size;
            if (last >= p.shares) last = p.shares - 1;   // (row offsets that do not increase)
            join = JoinRecord{u.part, static_cast<int32_t>(last - blockIdx.x), u.row0, u.tokens, u.kvh, 0, 0, 0};
          }
          cut(u, a, b);
        }
        first_unit = false;
        return u;
      }
      return u;
    };
    if (p.shares > 0) more = false;          // no block is taken over
    for (uint32_t it = 0;; ++it) {
      const uint32_t rb = it % C::kRecords, ph = (it / C::kRecords) & 1;
      Unit u;
      if (warp == 9) {
        if (p.stall_first_item && it == 0) break;
        if (p.shares > 0) {
          u = shared_unit();
        } else {
          u.tiles = -1;
          if (it > 0) {
            const uint32_t before = it - 1;
            if (last_tiles > kShortUnit &&
                !__all_sync(0xffffffffu, wait_for(b_recempty + 8 * (before % C::kRecords), (before / C::kRecords) & 1,
                                                  abort_flag, p, kWRecEmpty)))
              break;
            ask();
            n = answer();
          }
          while (n >= 0) {
            u = whole_unit(static_cast<uint32_t>(n));
            if (u.tiles >= 0) break;
            u.tiles = -1;              // a number without rows
            ask();
            n = answer();
          }
          last_tiles = u.tiles;
        }
        if (!__all_sync(0xffffffffu, wait_for(b_recempty + 8 * rb, ph ^ 1, abort_flag, p, kWRecEmpty))) break;
        if (lane == 0) {
          recs[rb] = u;
          mbar_arrive(b_recfull + 8 * rb);
        }
        __syncwarp();
      } else {
        if (!__all_sync(0xffffffffu, wait_for(b_recfull + 8 * rb, ph, abort_flag, p, kWRecFull))) break;
        u = load_unit(recs + rb);
        __syncwarp();
        if (lane == 0) mbar_arrive(b_recempty + 8 * rb);
      }
      if (u.tiles < 0) break;
      if (u.tiles == 0) continue;
      if (!__all_sync(0xffffffffu, wait_for(b_qempty, (qit & 1) ^ 1, abort_flag, p, kWQEmpty))) break;
      if constexpr (!FP4) {
        // a whole tile in one box per 64-dim block, a partial one token by token
        const bool full = u.tokens == p.tile_tokens;
        const uint32_t tok_bytes = static_cast<uint32_t>(p.group) * 128u;
        if (lane == 0) mbar_arrive_expect_tx(b_qfull, static_cast<uint32_t>(u.tokens) * tok_bytes * (D / 64));
        __syncwarp();
        const int loads = full ? D / 64 : u.tokens * (D / 64);
        for (int i = lane; i < loads; i += 32) {
          const int b = i % (D / 64), t = i / (D / 64);
          tma_load_3d(base + b * 16384 + t * tok_bytes, full ? &tmQT : &tmQ1, b * 64, u.kvh * p.group, u.row0 + t,
                      b_qfull);
        }
      } else {
        // rows to fp16 in the swizzled layout (generic stores)
        const int chunks = u.tokens * p.group * (D / 8);
        for (int i = (warp - 9) * 32 + lane; i < chunks; i += 32 * C::kQWarps) {
          const int r = i / (D / 8), c = i % (D / 8);
          const int64_t token = static_cast<int64_t>(u.row0) + r / p.group;
          const int32_t head = u.kvh * p.group + r % p.group;
          uint4 x = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + (token * p.n_qheads + head) * D +
                                                         c * 8));
          if constexpr (!std::is_same<T, __half>::value)
            x = make_uint4(bf16x2_as_f16x2(x.x), bf16x2_as_f16x2(x.y), bf16x2_as_f16x2(x.z), bf16x2_as_f16x2(x.w));
          st_shared_v4(base + (c >> 3) * C::kQBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4), x);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_qfull);
      }
      ++qit;
    }
    if (!FP4 && *abort_flag && qit > 0 && lane == 0) drain(b_qfull, (qit - 1) & 1, status, kDrainNs);
    __syncwarp();
    if (SOURCE != kSharedPrefix && warp == 9 && lane == 0 && p.shares > 0) p.joins[blockIdx.x] = join;
    if (warp == 9 && p.shares == 0 && (*abort_flag || p.stall_first_item)) {
      // the call is given up: blocks that have not started are taken off the grid, so that their waits do
      // not run out one after the other
      while (more) {
        ask();
        drain(b_next, asked & 1, status, kDrainNs);
        ++asked;
        more = clc_answer(base + C::kNextAt) >= 0;
        fence_proxy_async_smem();
        __syncwarp();
      }
    }
    finish_role();
    return;
  } else if constexpr (!FP4) {
    // ------------------------------------------------------------ K/V producers (TMA)
    regs_dec<C::kProducerRegs>();
    const int pw = warp - 12;
    const int per = p.box > 0 ? p.box : 4;                  // keys of one copy
    const int op = lane * 4 + pw;
    const int kb = op / C::kNBS * per, blk = op % C::kNBS;  // its first key and 64-dim block
    const bool active = op < kWinTile / per * C::kNBS;
    uint32_t st = 0, half = 0, js = 0, last_tile = 0;
    bool stop = false;
    struct Rows {   // physical rows of this lane's copy: slots of up to four keys
      int32_t r[4];
      bool wanted;
      uint32_t hole;
    };
    for (uint32_t it = 0; !stop; ++it) {
      const uint32_t rb = it % C::kRecords;
      if (!__all_sync(0xffffffffu, wait_for(b_recfull + 8 * rb, (it / C::kRecords) & 1, abort_flag, p,
                                            kWRecFull))) {
        stop = true;
        break;
      }
      const Unit u = load_unit(recs + rb);
      __syncwarp();
      if (lane == 0) mbar_arrive(b_recempty + 8 * rb);
      if (u.tiles < 0) break;
      // Where tile j's keys of this lane lie: a slot, or the row past the cache's end (which TMA fills
      // with zeros) where there is no page.
      auto locate = [&](int j) {
        Rows x{};
        if (!active) return x;
        const int32_t v = (u.tile0 + j) * kWinTile + kb;
        if constexpr (SOURCE == kChosenPages) {
          const int32_t e = entry_of(p, v);
          if (e < u.s0) {
            const PageEntry y = load_entry(unit_entries(p, u) + e);
            const int32_t o = v - e * p.pa.page_size;
            x.wanted = y.page * p.pa.page_size + o < u.p_first + u.tokens;
            x.r[0] = y.id * p.pa.page_size + o;
          }
          return x;
        }
        const int32_t pos = position_of(u, v);
        if (p.box > 0) {
          // a box is one run of positions inside one page
          x.wanted = pos < u.hi && (pos + per > u.lo || pos < p.n_sink);
          if (x.wanted) {
            const int64_t s = paged_slot(p.pa, u.req, INT32_MAX, pos);
            x.hole = s < 0;
            x.r[0] = s < 0 ? p.n_slots : static_cast<int32_t>(s);
          }
        } else {
          x.wanted = true;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool look = seen(p, u, pos + k);
            const int64_t s = look ? paged_slot(p.pa, u.req, INT32_MAX, pos + k) : -1;
            x.hole |= (look && s < 0 ? 1u : 0u) << k;
            x.r[k] = s < 0 ? p.n_slots * p.n_kvheads : static_cast<int32_t>(s) * p.n_kvheads + u.kvh;
          }
        }
        return x;
      };
      // K (is_v: V) of tile j
      auto issue = [&](const Rows& x, int j, bool is_v) -> bool {
        const uint32_t jt = js + j;
        last_tile = jt;
        const bool whole = j >= u.some0 && j < u.some1;
        const uint32_t bars = !is_v ? b_kready : whole ? b_pvready : b_vlanded;
        const uint32_t loads = __ballot_sync(0xffffffffu, x.wanted);
        const uint32_t bytes = __popc(loads) * per * 128;
#pragma unroll
        for (int h = 0; h < C::kSPT; ++h, ++half) {
          if (half >= C::kStages) {
            const uint32_t before = (half - C::kStages) / C::kSPT;   // the entry that held this stage
            if (!__all_sync(0xffffffffu, wait_done(before, kWStageEmpty))) return false;
          }
          if (h == 0 && !is_v) {
            uint32_t w0, w1 = 0;
            if (p.box > 0) {
              w0 = __ballot_sync(0xffffffffu, x.hole != 0);
            } else {
              w0 = (__ballot_sync(0xffffffffu, x.hole & 1) & 0xffffu) | (__ballot_sync(0xffffffffu, x.hole & 2) << 16);
              w1 = (__ballot_sync(0xffffffffu, x.hole & 4) & 0xffffu) | (__ballot_sync(0xffffffffu, x.hole & 8) << 16);
            }
            if (lane == 0)
              *reinterpret_cast<uint2*>(bad_keys + (jt % C::kBadSlots) * 8 + pw * 2) = make_uint2(w0, w1);
          }
          const uint32_t bar = bars + 8 * (jt % C::kTileBars);
          if (lane == 0) {
            if (bytes) mbar_arrive_expect_tx(bar, bytes); else mbar_arrive(bar);
            if (is_v && whole) mbar_arrive(b_vlanded + 8 * (jt % C::kTileBars));
          }
          __syncwarp();
          if (x.wanted) {
            const uint32_t dst = base + C::kRing + st * C::kStageBytes + blk * 16384 + kb * 128;
            const void* const tm = is_v ? static_cast<const void*>(&tmV) : static_cast<const void*>(&tmK);
            const int32_t d0 = h * 128 + blk * 64;
            if (p.box > 0) tma_load_3d(dst, tm, d0, u.kvh, x.r[0], bar);
            else tma_gather4(dst, tm, d0, x.r[0], x.r[1], x.r[2], x.r[3], bar);
          }
          if (++st == C::kStages) st = 0;
        }
        return true;
      };
      if (u.tiles == 0) continue;
      Rows k_next = locate(0);
      if (!issue(k_next, 0, false)) {
        stop = true;
        break;
      }
      Rows v_rows = k_next;
      if (u.tiles > 1) k_next = locate(1);
      for (int j = 0; j < u.tiles; ++j) {
        if (j + 1 < u.tiles && !issue(k_next, j + 1, false)) {
          stop = true;
          break;
        }
        if (!issue(v_rows, j, true)) {
          stop = true;
          break;
        }
        v_rows = k_next;
        if (j + 2 < u.tiles) k_next = locate(j + 2);
      }
      js += u.tiles;
    }
    if (stop && lane == 0) {
      // copies that may still be in flight: of the last tiles (a P.V barrier may also lack its softmax
      // arrivals; the limit is a thousand times what a copy takes)
      for (uint32_t t = last_tile > 5 ? last_tile - 5 : 0; t <= last_tile; ++t) {
        drain(b_kready + 8 * (t % C::kTileBars), (t / C::kTileBars) & 1, status, kDrainNs / 100);
        drain(b_pvready + 8 * (t % C::kTileBars), (t / C::kTileBars) & 1, status, kDrainNs / 100);
      }
    }
    __syncwarp();
    finish_role();
    return;
  } else {
    // A key's codes are kParts 16-byte parts.  Lanes convert neighbouring keys of one part, so the parts are
    // exchanged by the key's place: eight keys' loads then cover all banks.
    constexpr int kParts = D / 32;
    auto staged = [](int key, int part) -> uint32_t {
      return key * (D / 2) + ((part ^ (key / (8 / kParts) & (kParts - 1))) << 4);
    };
    if (warp < 16) {
      // ---------------------------------------------------------- 4-bit caches: copies into the staging ring
      regs_dec<C::kProducerRegs>();
      const int pw = warp - 12;                             // keys 32 pw .. 32 pw + 31 of every tile
      uint32_t n = 0, slot_at = 0, turn = 0, jt = 0;        // entries copied; n % kDepth, n / kDepth
      bool stop = false;
      const uint32_t row_codes = static_cast<uint32_t>(p.n_kvheads) * (D / 2);
      const uint32_t row_scales = static_cast<uint32_t>(p.n_kvheads) * (D / 16);
      for (uint32_t it = 0; !stop; ++it) {
        const uint32_t rb = it % C::kRecords;
        if (!__all_sync(0xffffffffu, wait_for(b_recfull + 8 * rb, (it / C::kRecords) & 1, abort_flag, p,
                                              kWRecFull))) {
          stop = true;
          break;
        }
        const Unit u = load_unit(recs + rb);
        __syncwarp();
        if (lane == 0) mbar_arrive(b_recempty + 8 * rb);
        if (u.tiles < 0) break;
        const uint8_t* const k_codes = p.k_codes + static_cast<int64_t>(u.kvh) * (D / 2) + lane % kParts * 16;
        const uint8_t* const v_codes = p.v_codes + static_cast<int64_t>(u.kvh) * (D / 2) + lane % kParts * 16;
        const uint8_t* const k_scale = p.k_scale + static_cast<int64_t>(u.kvh) * (D / 16);
        const uint8_t* const v_scale = p.v_scale + static_cast<int64_t>(u.kvh) * (D / 16);
        // The page of this lane's key in the next K tile is looked up one tile ahead, so that its load is not
        // waited for; V takes its K tile's slot.
        int32_t page = -1, offset = 0;
        bool look = false;
        auto look_up = [&](int tile) {
          const int32_t pos = position_of(u, (u.tile0 + tile) * kWinTile + pw * 32 + lane);
          look = seen(p, u, pos);
          page = -1;
          if (look) {
            const int32_t e = p.pa.page_shift >= 0 ? pos >> p.pa.page_shift : pos / p.pa.page_size;
            offset = pos - e * p.pa.page_size;
            if (e < p.pa.pages_per_req)
              page = __ldg(p.pa.page_table + static_cast<int64_t>(u.req) * p.pa.pages_per_req + e);
          }
        };
        auto copy = [&](int32_t slot, const uint8_t* codes, const uint8_t* scales, uint32_t tag) -> bool {
          if (n >= C::kDepth &&
              !__all_sync(0xffffffffu, wait_for(b_unstaged + 8 * slot_at, (turn & 1) ^ 1, abort_flag, p, kWUnstaged)))
            return false;
          const uint32_t to = base + C::kStagingAt + slot_at * C::kStaging;
#pragma unroll
          for (int i = 0; i < kParts; ++i) {
            const int key = i * (32 / kParts) + lane / kParts;
            const int32_t s = __shfl_sync(0xffffffffu, slot, key);
            cp_async_zfill<16>(to + staged(pw * 32 + key, lane % kParts),
                               codes + static_cast<uint64_t>(static_cast<uint32_t>(max(s, 0))) * row_codes, s >= 0);
          }
          cp_async_zfill<D / 16>(to + kWinTile * (D / 2) + (pw * 32 + lane) * (D / 16),
                                 scales + static_cast<uint64_t>(static_cast<uint32_t>(max(slot, 0))) * row_scales, slot >= 0);
          cp_async_arrive(b_staged + 8 * slot_at);
          if (pw == 0 && lane == 0) {
            tags[slot_at] = tag;
            mbar_arrive(b_staged + 8 * slot_at);
          }
          ++n;
          if (++slot_at == C::kDepth) {
            slot_at = 0;
            ++turn;
          }
          return true;
        };
        int32_t slot = -1;
        if (u.tiles > 0) look_up(0);
        for (int t = 0; t <= u.tiles && u.tiles > 0; ++t) {  // K of tile t, then V of tile t - 1
          const int32_t before = slot;
          if (t < u.tiles) {
            slot = page >= 0 && page < p.pa.n_pages ? page * p.pa.page_size + offset : -1;
            const uint32_t holes = __ballot_sync(0xffffffffu, look && slot < 0);
            if (lane == 0)
              *reinterpret_cast<uint2*>(bad_keys + (jt % C::kBadSlots) * 8 + pw * 2) = make_uint2(holes & 0xffffu, holes >> 16);
            ++jt;
            if (!copy(slot, k_codes, k_scale, 2 * (jt - 1))) {
              stop = true;
              break;
            }
            if (t + 1 < u.tiles) look_up(t + 1);
          }
          if (t > 0 && !copy(before, v_codes, v_scale, 2 * (t < u.tiles ? jt - 2 : jt - 1) + 1)) {
            stop = true;
            break;
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (!stop && n >= C::kDepth) {                        // (the tag's slot has been read)
        stop = !__all_sync(0xffffffffu, wait_for(b_unstaged + 8 * slot_at, (turn & 1) ^ 1, abort_flag, p, kWUnstaged));
      }
      if (!stop) {
        if (pw == 0 && lane == 0) {
          tags[slot_at] = kLastTag;
          mbar_arrive(b_staged + 8 * slot_at);
        }
        mbar_arrive(b_staged + 8 * slot_at);
      }
      __syncwarp();
      finish_role();
      return;
    }
    // ------------------------------------------------------------ 4-bit caches: conversion to fp16
    regs_dec<C::kConvertRegs>();
    const int wi = warp - 16;                               // keys 16 wi .. 16 wi + 15 of every tile
    uint32_t slot_at = 0, turn = 0;
    for (uint32_t n = 0;; ++n) {
      if (!__all_sync(0xffffffffu, wait_for(b_staged + 8 * slot_at, turn & 1, abort_flag, p, kWStaged))) break;
      const uint32_t tag = tags[slot_at];                   // 2 tile + 1 for V, of the call's tiles
      if (tag == kLastTag) break;
      const uint32_t half0 = n * C::kSPT;
      if (half0 + C::kSPT > C::kStages) {                   // the entry that held the last of the stages
        const uint32_t before = (half0 + C::kSPT - 1 - C::kStages) / C::kSPT;
        if (!__all_sync(0xffffffffu, wait_done(before, kWStageEmpty))) break;
      }
      const uint32_t from = base + C::kStagingAt + slot_at * C::kStaging;
      constexpr int kUnits = 16 * (D / 64);                 // (key, 64-dim block)
#pragma unroll 1
      for (int k = lane; k < kUnits; k += 32) {
        // neighbouring lanes take neighbouring keys: their rows differ in the swizzle, so that eight lanes'
        // stores cover all banks
        const int r = wi * 16 + k % 16, blk = k / 16;
        const uint4 c0 = ld_shared_v4(from + staged(r, 2 * blk));
        const uint4 c1 = ld_shared_v4(from + staged(r, 2 * blk + 1));
        const uint32_t sc4 = ld_shared_u32(from + kWinTile * (D / 2) + r * (D / 16) + blk * 4);
        const uint32_t s01 = e4m3x2_to_f16x2(static_cast<uint16_t>(sc4)), s23 = e4m3x2_to_f16x2(static_cast<uint16_t>(sc4 >> 16));
        __half2 sa, sb;
        memcpy(&sa, &s01, 4);
        memcpy(&sb, &s23, 4);
        const __half2 sc[4] = {__low2half2(sa), __high2half2(sa), __low2half2(sb), __high2half2(sb)};
        const uint32_t words[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        const uint32_t half = half0 + blk / C::kNBS;
        const uint32_t row = base + C::kRing + (half % C::kStages) * C::kStageBytes + (blk % C::kNBS) * 16384 + r * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          st_shared_v4(row + ((c ^ (r & 7)) << 4),
                       make_uint4(e2m1_scaled(words[c], 0, sc[c / 2]), e2m1_scaled(words[c], 1, sc[c / 2]),
                                  e2m1_scaled(words[c], 2, sc[c / 2]), e2m1_scaled(words[c], 3, sc[c / 2])));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive((tag & 1 ? b_pvready : b_kready) + 8 * ((tag >> 1) % C::kTileBars));
        mbar_arrive(b_unstaged + 8 * slot_at);
      }
      if (++slot_at == C::kDepth) {
        slot_at = 0;
        ++turn;
      }
    }
    __syncwarp();
    finish_role();
    return;
  }
}

// ---------------------------------------------------------------------------- host side
template <int D, typename T, bool FP4, UnitSource SOURCE = kWindowRows>
cudaError_t launch_window_instance(const WindowParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                                   const CUtensorMap& tq1, const CUtensorMap& tqt, int grid, int which,
                                   cudaStream_t stream) {
  using C = WinCfg<D, FP4>;
  auto kern = window_attention_kernel<D, T, FP4, SOURCE>;
  cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(kern), C::kSmem, kOptWindow + which);
  if (e != cudaSuccess) return e;
  // The warpgroups' register shares add up to kThreads x kLaunchRegs: a kernel compiled to fewer would wait
  // for registers that the block does not own.
  static const int regs = [&] {
    cudaFuncAttributes a{};
    return cudaFuncGetAttributes(&a, kern) == cudaSuccess ? a.numRegs : 0;
  }();
  if (regs < C::kLaunchRegs) return cudaErrorInvalidConfiguration;
  if constexpr (SOURCE == kWindowRows) {
    kern<<<grid, C::kThreads, C::kSmem, stream>>>(tk, tv, tq1, tqt, p);
    return cudaGetLastError();
  } else {   // starts while the kernel that lists the units runs
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tk, tv, tq1, tqt, p);
  }
}
template <int D>
cudaError_t launch_window_dim(const WindowParams& p, bool fp16, bool fp4, const CUtensorMap& tk,
                              const CUtensorMap& tv, const CUtensorMap& tq1, const CUtensorMap& tqt, int grid,
                              cudaStream_t stream) {
  constexpr int at = D == 64 ? 0 : D == 128 ? 4 : 8;
  if (fp4)
    return fp16 ? launch_window_instance<D, __half, true>(p, tk, tv, tq1, tqt, grid, at, stream)
                : launch_window_instance<D, __nv_bfloat16, true>(p, tk, tv, tq1, tqt, grid, at + 1, stream);
  return fp16 ? launch_window_instance<D, __half, false>(p, tk, tv, tq1, tqt, grid, at + 2, stream)
              : launch_window_instance<D, __nv_bfloat16, false>(p, tk, tv, tq1, tqt, grid, at + 3, stream);
}
// Listed units.
template <int D>
cudaError_t launch_listed_dim(const WindowParams& p, bool fp16, bool prefix, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tq1, const CUtensorMap& tqt, int grid, cudaStream_t stream) {
  constexpr int at = D == 64 ? 12 : D == 128 ? 16 : 20;
  if (prefix)
    return fp16 ? launch_window_instance<D, __half, false, kSharedPrefix>(p, tk, tv, tq1, tqt, grid, at, stream)
                : launch_window_instance<D, __nv_bfloat16, false, kSharedPrefix>(p, tk, tv, tq1, tqt, grid, at + 1, stream);
  return fp16 ? launch_window_instance<D, __half, false, kChosenPages>(p, tk, tv, tq1, tqt, grid, at + 2, stream)
              : launch_window_instance<D, __nv_bfloat16, false, kChosenPages>(p, tk, tv, tq1, tqt, grid, at + 3, stream);
}
// one translation unit per head dim, for each of the two kinds
cudaError_t launch_window_d64(const WindowParams&, bool, bool, const CUtensorMap&, const CUtensorMap&,
                              const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
cudaError_t launch_window_d128(const WindowParams&, bool, bool, const CUtensorMap&, const CUtensorMap&,
                               const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
cudaError_t launch_window_d256(const WindowParams&, bool, bool, const CUtensorMap&, const CUtensorMap&,
                               const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
cudaError_t launch_listed_d64(const WindowParams&, bool, bool, const CUtensorMap&, const CUtensorMap&,
                               const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
cudaError_t launch_listed_d128(const WindowParams&, bool, bool, const CUtensorMap&, const CUtensorMap&,
                               const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);
cudaError_t launch_listed_d256(const WindowParams&, bool, bool, const CUtensorMap&, const CUtensorMap&,
                               const CUtensorMap&, const CUtensorMap&, int, cudaStream_t);

}  // namespace qsa
