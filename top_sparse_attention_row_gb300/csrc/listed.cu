// Listed units of attention (window.cuh): what a call over chosen pages or behind shared prompts consists of, worked out
// by a small kernel before the attention kernel, and the join of shared prompts' rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "window.cuh"

namespace qsa {
namespace {

using window_detail::Unit;

// Tiles before request (group) i: first row / tile tokens + i, as in window_detail::first_tile.
__device__ __forceinline__ int32_t request_tile(const ListParams& p, int32_t i) {
  return __ldg(p.pa.cu_seqlens_q + i) / p.tile_tokens + i;
}
__device__ __forceinline__ int32_t group_begin(const ListParams& p, int32_t g) {
  return min(max(__ldg(p.cu_groups + g), 0), p.pa.n_requests);
}
__device__ __forceinline__ int32_t group_tile(const ListParams& p, int32_t g) {
  return __ldg(p.pa.cu_seqlens_q + group_begin(p, g)) / p.tile_tokens + g;
}
// The last i in [0, n) with first(i) <= x (first does not decrease); 0 where there is none.  By whole warps.
template <typename F>
__device__ __forceinline__ int32_t last_at_most(int32_t n, int32_t x, int lane, F first) {
  int32_t lo = 0, hi = n - 1;
  while (lo < hi) {
    const int32_t step = (hi - lo + 32) / 32;
    const int32_t cand = lo + lane * step;
    const uint32_t m = __ballot_sync(0xffffffffu, cand <= hi && first(cand) <= x);
    const int last = m ? 31 - __clz(m) : 0;
    lo = lo + last * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}
struct Rows {
  int32_t row0, tokens;
  int64_t p_first;
};
// Rows of tile number `tile` of request req; tokens = 0 for a number without rows.
__device__ __forceinline__ Rows tile_rows(const ListParams& p, int32_t req, int32_t tile) {
  const int64_t r0 = __ldg(p.pa.cu_seqlens_q + req);
  int64_t r1 = __ldg(p.pa.cu_seqlens_q + req + 1);
  if (r1 > p.n_rows) r1 = p.n_rows;
  const int64_t t0 = static_cast<int64_t>(tile - request_tile(p, req)) * p.tile_tokens;
  Rows x{0, 0, 0};
  if (r0 < 0 || t0 < 0 || r0 + t0 >= r1) return x;
  x.row0 = static_cast<int32_t>(r0 + t0);
  x.tokens = static_cast<int32_t>(r1 - r0 - t0 < p.tile_tokens ? r1 - r0 - t0 : p.tile_tokens);
  x.p_first = __ldg(p.pa.kv_lens + req) - (r1 - r0) + t0;
  return x;
}
__device__ __forceinline__ void store_unit(Unit* to, const Unit& u) {
  int4* const t = reinterpret_cast<int4*>(to);
  t[0] = make_int4(u.tiles, u.tile0, u.req, u.kvh);
  t[1] = make_int4(u.part, u.row0, u.tokens, u.p_first);
  t[2] = make_int4(u.s0, u.shift, u.lo, u.hi);
  t[3] = make_int4(u.some0, u.some1, u.all0, u.all1);
}

// ---------------------------------------------------------------------------- chosen pages
// A block lists the unit of one query tile and KV head: the pages that some of its tokens list and can see a position
// of, in increasing order, each once, with the tokens that list it.  Neighbouring tokens list much the same pages, so
// the unit reads little more than one token's.  The tokens of a page are gathered as bits of a map over the
// request's pages in shared memory, which makes repeats and the order of the lists immaterial.
constexpr int kListThreads = 256;

__global__ void __launch_bounds__(kListThreads) list_pages_kernel(const __grid_constant__ ListParams p) {
  extern __shared__ uint32_t map[];
  __shared__ int32_t counts[kListThreads / 32];
  __shared__ int32_t partial, last_page;   // first entry that some row does not see whole; the last entry's page
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  const int32_t f = blockIdx.x, tile = f / p.n_kvheads, kvh = f - tile * p.n_kvheads;
  const int32_t req = last_at_most(p.pa.n_requests, tile, lane, [&](int32_t i) { return request_tile(p, i); });
  const Rows x = tile_rows(p, req, tile);
  if (x.tokens == 0) {
    if (tid == 0) p.unit_tiles[f] = -2;
    return;
  }
  const int32_t ps = p.pa.page_size;
  const int64_t p_last = x.p_first + x.tokens - 1;
  const int64_t mine = p_last < 0 ? 0 : p_last / ps + 1;
  const int32_t n = static_cast<int32_t>(mine < p.pa.pages_per_req ? mine : p.pa.pages_per_req);
  for (int32_t e = tid; e < n; e += kListThreads) map[e] = 0;
  if (tid == 0) {
    partial = INT32_MAX;
    last_page = -1;
  }
  __syncthreads();
  const int32_t* const lists = p.pages + (static_cast<int64_t>(x.row0) * p.n_kvheads + kvh) * p.n_select;
  for (int64_t i = tid; i < static_cast<int64_t>(x.tokens) * p.n_select; i += kListThreads) {
    const int32_t t = static_cast<int32_t>(i / p.n_select), k = static_cast<int32_t>(i - static_cast<int64_t>(t) * p.n_select);
    const int32_t e = __ldg(lists + static_cast<int64_t>(t) * p.n_kvheads * p.n_select + k);
    if (e >= 0 && e < n && static_cast<int64_t>(e) * ps <= x.p_first + t) atomicOr(map + e, 1u << t);
  }
  __syncthreads();
  const int32_t* const table = p.pa.page_table + static_cast<int64_t>(req) * p.pa.pages_per_req;
  PageEntry* const out = p.entries + static_cast<int64_t>(f) * p.list_cap;
  const uint32_t full = x.tokens == 32 ? 0xffffffffu : (1u << x.tokens) - 1u;
  int32_t base = 0, whole = 0;             // entries so far; this thread's that lie before the first row's position
  for (int32_t c = 0; c < n; c += kListThreads) {
    const int32_t e = c + tid;
    const uint32_t rows = e < n ? map[e] : 0u;
    const int32_t id = rows ? __ldg(table + e) : -1;
    const bool in = id >= 0 && id < p.pa.n_pages;
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    if (lane == 0) counts[warp] = __popc(m);
    __syncthreads();
    int32_t at = base + __popc(m & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kListThreads / 32; ++w) {
      if (w < warp) at += counts[w];
      base += counts[w];
    }
    if (in) {
      *reinterpret_cast<int4*>(out + at) = make_int4(e, id, static_cast<int32_t>(rows), 0);
      const bool before = static_cast<int64_t>(e + 1) * ps <= x.p_first + 1;
      whole += before;
      if (!before || rows != full) atomicMin(&partial, at);
      atomicMax(&last_page, e);
    }
    __syncthreads();
  }
  whole = __reduce_add_sync(0xffffffffu, whole);
  if (lane == 0) counts[warp] = whole;
  __syncthreads();
  if (tid != 0) return;
  whole = 0;
  for (int w = 0; w < kListThreads / 32; ++w) whole += counts[w];
  Unit u{};
  if (base > 0) {
    const int64_t tail = p_last + 1 - static_cast<int64_t>(last_page) * ps;
    const int64_t keys = static_cast<int64_t>(base - 1) * ps + (tail < ps ? tail : ps);
    u.tiles = static_cast<int32_t>((keys + kWinTile - 1) / kWinTile);
  }
  u.req = req;
  u.kvh = kvh;
  u.part = -1;
  u.row0 = x.row0;
  u.tokens = x.tokens;
  u.p_first = static_cast<int32_t>(x.p_first);
  u.s0 = base;
  u.shift = f;
  u.some1 = static_cast<int32_t>(static_cast<int64_t>(whole) * ps / kWinTile);
  u.all1 = static_cast<int32_t>(static_cast<int64_t>(min(partial, whole)) * ps / kWinTile);
  store_unit(static_cast<Unit*>(p.units) + f, u);
  p.unit_tiles[f] = u.tiles;
}

// ---------------------------------------------------------------------------- shared prompts
// What a group shares: the positions below prefix_len that all of its requests with rows have as past, by the page table of
// the first of these (a request without rows may have no pages any more).
struct Group {
  int32_t number, table, row0, rows, shared;
};
// By whole warps.  Sharing pays where it saves more key tiles than it costs: the requests' tiles each read the shared keys
// on their own, or the fewer tiles of the group's rows do, and cost about 5 key tiles each (query tile, first softmax,
// output in fp32, join) and one more for every tile of a request, whose output is joined too.
__device__ __forceinline__ Group make_group(const ListParams& p, int32_t g, int lane) {
  Group x{g, 0, 0, 0, 0};
  const int32_t begin = group_begin(p, g), end = max(group_begin(p, g + 1), begin);
  x.row0 = __ldg(p.pa.cu_seqlens_q + begin);
  x.rows = __ldg(p.pa.cu_seqlens_q + end) - x.row0;
  int32_t past = INT32_MAX, first = INT32_MAX;
  uint32_t tiles = 0;
  for (int32_t i = begin + lane; i < end; i += 32) {
    const int32_t fresh = __ldg(p.pa.cu_seqlens_q + i + 1) - __ldg(p.pa.cu_seqlens_q + i);
    if (fresh <= 0) continue;
    past = min(past, max(__ldg(p.pa.kv_lens + i), 0) - fresh);
    first = min(first, i);
    tiles += (fresh + p.tile_tokens - 1) / p.tile_tokens;
  }
  past = __reduce_min_sync(0xffffffffu, past);
  first = __reduce_min_sync(0xffffffffu, first);
  const int64_t own = __reduce_add_sync(0xffffffffu, tiles);
  const int64_t cap = static_cast<int64_t>(p.pa.pages_per_req) * p.pa.page_size;
  int64_t shared = min(past, __ldg(p.prefix_lens + g));
  if (shared > cap) shared = cap;
  const int64_t all = (x.rows + p.tile_tokens - 1) / p.tile_tokens, key_tiles = (shared + kWinTile - 1) / kWinTile;
  if (x.row0 >= 0 && shared > 0 && (own - all) * key_tiles > 5 * all + own) x.shared = static_cast<int32_t>(shared);
  if (first < end) x.table = first;                        // (else nothing is shared: no request has rows)
  return x;
}

constexpr int kPrefixWarps = 4;   // of a block

__global__ void __launch_bounds__(kPrefixWarps * 32) list_prefix_kernel(const __grid_constant__ ListParams p) {
  const int lane = threadIdx.x & 31;
  pdl_launch_dependents();
  const int32_t tiles = p.n_tiles / p.n_kvheads;
  const int32_t t_first = (static_cast<int32_t>(blockIdx.x) * kPrefixWarps + (threadIdx.x >> 5)) * p.run;
  Group group{-1, 0, 0, 0, 0};
  for (int32_t t = t_first; t < min(t_first + p.run, tiles); ++t) {
    Unit u{};
    u.tiles = -2;
    OwnUnit own{0, -1, 0, 0};
    if (t < p.prefix_tiles) {
      // a tile of a group's rows: all of them see all of the shared keys
      const int32_t g = last_at_most(p.n_groups, t, lane, [&](int32_t i) { return group_tile(p, i); });
      if (g != group.number) group = make_group(p, g, lane);
      const int64_t t0 = static_cast<int64_t>(t - group_tile(p, g)) * p.tile_tokens;
      const int64_t rows = min(static_cast<int64_t>(group.rows), p.n_rows - group.row0);
      if (group.shared > 0 && t0 >= 0 && t0 < rows) {
        u.req = group.table;
        u.part = 0;
        u.row0 = group.row0 + static_cast<int32_t>(t0);
        u.tokens = static_cast<int32_t>(rows - t0 < p.tile_tokens ? rows - t0 : p.tile_tokens);
        u.p_first = group.shared;
        u.hi = group.shared;
        u.tiles = (group.shared + kWinTile - 1) / kWinTile;
        u.some1 = u.all1 = group.shared / kWinTile;
      }
    } else {
      // a tile of a request's rows: the keys behind the shared ones
      const int32_t number = t - p.prefix_tiles;
      const int32_t req = last_at_most(p.pa.n_requests, number, lane, [&](int32_t i) { return request_tile(p, i); });
      const Rows x = tile_rows(p, req, number);
      if (x.tokens > 0) {
        int64_t shared = 0;
        if (p.n_groups > 0) {
          const int32_t g = last_at_most(p.n_groups, req, lane, [&](int32_t i) { return group_begin(p, i); });
          if (group_begin(p, g) <= req && req < group_begin(p, g + 1)) {
            if (g != group.number) group = make_group(p, g, lane);
            shared = group.shared;
            if (shared > 0) own = OwnUnit{group.row0, group_tile(p, g) * p.n_kvheads, 0, 0};
          }
        }
        own.row0 = x.row0;
        own.tokens = x.tokens;
        const int64_t cap = static_cast<int64_t>(p.pa.pages_per_req) * p.pa.page_size;
        const int64_t hi = max(min(x.p_first + x.tokens, cap), static_cast<int64_t>(0)), lo = min(shared, hi);
        const int64_t shift = lo & ~static_cast<int64_t>(p.grain - 1);
        u.req = req;
        u.part = shared > 0 ? 1 : -1;
        u.row0 = x.row0;
        u.tokens = x.tokens;
        u.p_first = static_cast<int32_t>(x.p_first);
        u.shift = static_cast<int32_t>(shift);
        u.lo = static_cast<int32_t>(lo);
        u.hi = static_cast<int32_t>(hi);
        u.tiles = static_cast<int32_t>((hi - shift + kWinTile - 1) / kWinTile);
        const int64_t first = (lo - shift + kWinTile - 1) / kWinTile;
        u.some0 = u.all0 = static_cast<int32_t>(first);
        u.some1 = static_cast<int32_t>((hi - shift) / kWinTile);
        const int64_t all = min(x.p_first + 1, hi) - shift;      // keys that the first row sees too
        u.all1 = static_cast<int32_t>((all > 0 ? all : 0) / kWinTile);
      }
    }
    for (int32_t h = lane; h < p.n_kvheads; h += 32) {
      const int32_t f = t * p.n_kvheads + h;
      u.kvh = h;
      p.unit_tiles[f] = u.tiles;
      p.unit_joins[f] = make_int2(0, -1);   // (for a call that is given up)
      if (u.tiles >= 0) store_unit(static_cast<Unit*>(p.units) + f, u);
      if (t >= p.prefix_tiles) {
        OwnUnit o = own;
        if (o.prefix_unit >= 0) o.prefix_unit += h;
        p.own[f - p.prefix_tiles * p.n_kvheads] = o;
      }
    }
  }
}

// Joins the results of a row: of the shared keys and of its own, each of which may have several parts.  With L_s a
// part's log-sum-exp and O_s its normalised output, lse = ln sum exp(L_s) and O = sum exp(L_s - lse) O_s.  W warps take a
// row and divide its parts: one where there are many rows (of two or three parts each), four where few rows have a part in
// many blocks and the latency of one part after the other would count.  The parts are added in a fixed order.  A part that
// is NaN makes the row NaN.
constexpr int kJoinWarps = 8;
constexpr int64_t kJoinFewRows = 16384;
template <int D, typename T, int W>
__global__ void __launch_bounds__(kJoinWarps * 32)
    join_prefix_kernel(const __grid_constant__ WindowParams p, const OwnUnit* own_units, int32_t prefix_units) {
  constexpr int kPer = D / 32, kRows = kJoinWarps / W;
  __shared__ float sums[W > 1 ? kJoinWarps : 1][W > 1 ? D : 1];
  pdl_wait();   // first thing in every thread: the grid must not end before the attention kernel has
  const OwnUnit own = own_units[blockIdx.x];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp % W, rows = own.tokens * p.group;
  const int32_t unit = prefix_units + static_cast<int32_t>(blockIdx.x), kvh = unit % p.n_kvheads;
  const int64_t all_rows = p.n_rows * p.n_qheads;
  if (rows == 0) return;
  const int2 b = p.unit_joins[unit];
  for (int first = blockIdx.y * kRows; first < rows; first += gridDim.y * kRows) {   // (uniform over the block)
    const int row = first + warp / W;
    const bool live = row < rows;
    const int tok = live ? row / p.group : 0;
    const int64_t token = static_cast<int64_t>(own.row0) + tok;
    const int64_t rh = token * p.n_qheads + kvh * p.group + (row - tok * p.group);
    // (many rows) Most have two results that are whole: these are on their way while it is looked up whether that is so.
    float l0 = -INFINITY, l1 = -INFINITY, x0[kPer], x1[kPer];
    if (W == 1 && live && own.prefix_unit >= 0) {
      l0 = p.first_lse[rh];
      l1 = p.first_lse[all_rows + rh];
#pragma unroll
      for (int k = 0; k < kPer; k += 2) {
        const float2 y0 = *reinterpret_cast<const float2*>(p.first_o + rh * D + lane * kPer + k);
        const float2 y1 = *reinterpret_cast<const float2*>(p.first_o + (all_rows + rh) * D + lane * kPer + k);
        x0[k] = y0.x;
        x0[k + 1] = y0.y;
        x1[k] = y1.x;
        x1[k + 1] = y1.y;
      }
    }
    // parts: [0, split) of the shared keys, then of the row's own; slots and rows of those after the first ones
    int2 a = make_int2(0, -1);
    int32_t a_row = 0;
    if (own.prefix_unit >= 0) {
      const int32_t ahead = static_cast<int32_t>(token) - own.group_row0, tile = ahead / p.tile_tokens;
      const int32_t from = own.prefix_unit + tile * p.n_kvheads;
      if (ahead >= 0 && from < prefix_units) {             // (offsets that do not increase)
        a = p.unit_joins[from];
        a_row = (ahead - tile * p.tile_tokens) * p.group + (row - tok * p.group);
      }
    }
    const int split = a.y + 1, all = split + b.y + 1;
    // nothing to join: given up; written by the attention kernel
    const int parts = !live || all == 0 || (split == 0 && all == 1) ? 0 : all;
    auto place = [&](int s, int64_t* whole) -> int64_t {   // of a part: row of the first parts, or of the others
      *whole = s == 0 && split > 0 ? rh : s == split ? all_rows + rh : -1;
      return s < split ? static_cast<int64_t>(a.x + s) * kWinTile + a_row
                       : static_cast<int64_t>(b.x + s - split) * kWinTile + row;
    };
    auto lse_of = [&](int s) {
      int64_t whole;
      const int64_t other = place(s, &whole);
      return whole >= 0 ? p.first_lse[whole] : p.part_lse[other];
    };
    float m = -INFINITY, total = 0.0f;
    float acc[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] = 0.0f;
    const bool two = W == 1 && split == 1 && parts == 2;   // (uniform over the warp)
    if (two) {
      m = fmaxf(l0, l1);
      // a part that saw nothing of this row wrote no output: whatever is there stays out
      const float w0 = l0 == -INFINITY ? 0.0f : __expf(l0 - m), w1 = l1 == -INFINITY ? 0.0f : __expf(l1 - m);
      total = lane == 0 ? w0 + w1 : 0.0f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = (l0 == -INFINITY ? 0.0f : w0 * x0[k]) + (l1 == -INFINITY ? 0.0f : w1 * x1[k]);
    } else {
      for (int s = lane; s < parts; s += 32) m = fmaxf(m, lse_of(s));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    for (int s0 = 0; s0 < parts && !two; s0 += 32) {
      const float l = s0 + lane < parts ? lse_of(s0 + lane) : -INFINITY;
      const float w = l == -INFINITY ? 0.0f : __expf(l - m);
      total += w;
      // a part that saw nothing of this row wrote no output: whatever is there stays out
      const uint32_t saw = __ballot_sync(0xffffffffu, l != -INFINITY);
#pragma unroll 4
      for (int i = mine; i < min(parts - s0, 32); i += W) {
        const float ws = __shfl_sync(0xffffffffu, w, i);
        int64_t whole;
        const int64_t other = place(s0 + i, &whole);
        const float* const src = (whole >= 0 ? p.first_o + whole * D : p.part_o + other * D) + lane * kPer;
#pragma unroll
        for (int k = 0; k < kPer; k += 2) {
          const float2 x = *reinterpret_cast<const float2*>(src + k);
          if (saw >> i & 1) {
            acc[k] += ws * x.x;
            acc[k + 1] += ws * x.y;
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const float inv = m == -INFINITY ? 0.0f : 1.0f / total;
    if constexpr (W > 1) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) sums[warp][lane * kPer + k] = acc[k];
      __syncthreads();
      if (mine == 0) {
#pragma unroll
        for (int w = 1; w < W; ++w) {
#pragma unroll
          for (int k = 0; k < kPer; ++k) acc[k] += sums[warp + w][lane * kPer + k];
        }
      }
      __syncthreads();
    }
    if (mine != 0 || parts == 0) continue;
    uint32_t* const out = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + rh * D + lane * kPer);
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k) out[k] = window_detail::pack16(acc[2 * k] * inv, acc[2 * k + 1] * inv, T{});
    if (lane == 0 && p.lse) p.lse[rh] = total == 0.0f ? -INFINITY : m + logf(total);
  }
}

template <int D, typename T, int W>
cudaError_t launch_join_prefix_warps(const WindowParams& p, const ListParams& l, cudaStream_t stream) {
  const int32_t prefix_units = l.prefix_tiles * l.n_kvheads;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // as many blocks as the units have rows on average (a block of a unit with more goes over them)
  const int64_t units = (l.n_tiles - prefix_units) / l.n_kvheads, tokens = p.n_rows > units ? (p.n_rows + units - 1) / units : 1;
  cfg.gridDim = dim3(static_cast<unsigned>(l.n_tiles - prefix_units),
                     static_cast<unsigned>((tokens * p.group + kJoinWarps / W - 1) / (kJoinWarps / W)));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_prefix_kernel<D, T, W>, p, static_cast<const OwnUnit*>(l.own), prefix_units);
}
template <int D, typename T>
cudaError_t launch_join_prefix_dim(const WindowParams& p, const ListParams& l, cudaStream_t stream) {
  return p.n_rows * p.n_qheads <= kJoinFewRows ? launch_join_prefix_warps<D, T, 4>(p, l, stream)
                                               : launch_join_prefix_warps<D, T, 1>(p, l, stream);
}

}  // namespace

cudaError_t launch_list_pages(const ListParams& p, cudaStream_t stream) {
  const cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(list_pages_kernel), kMaxChoosePages * 4, kOptListPages);
  if (e != cudaSuccess) return e;
  list_pages_kernel<<<static_cast<unsigned>(p.n_tiles), kListThreads, static_cast<size_t>(p.pa.pages_per_req) * 4, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_list_prefix(ListParams p, cudaStream_t stream) {
  // a warp that lists several tiles reads its group's lengths once; few tiles are listed side by side
  const int32_t tiles = p.n_tiles / p.n_kvheads;
  p.run = tiles <= 2048 ? 1 : 4;
  const int32_t per = kPrefixWarps * p.run;
  list_prefix_kernel<<<static_cast<unsigned>((tiles + per - 1) / per), kPrefixWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_join_prefix(const WindowParams& p, const ListParams& l, int head_dim, bool fp16, cudaStream_t stream) {
  if (fp16)
    return head_dim == 64    ? launch_join_prefix_dim<64, __half>(p, l, stream)
           : head_dim == 128 ? launch_join_prefix_dim<128, __half>(p, l, stream)
                             : launch_join_prefix_dim<256, __half>(p, l, stream);
  return head_dim == 64    ? launch_join_prefix_dim<64, __nv_bfloat16>(p, l, stream)
         : head_dim == 128 ? launch_join_prefix_dim<128, __nv_bfloat16>(p, l, stream)
                           : launch_join_prefix_dim<256, __nv_bfloat16>(p, l, stream);
}

}  // namespace qsa
