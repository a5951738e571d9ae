// Page tables and slot maps of a serving step, built on the GPU from the requests' lengths.
//
// Request i holds past[i] cached tokens and brings new[i] tokens.  With P(x) = min(ceil(x / page
// size), pages per request) it needs need[i] = P(past + new) - P(past) fresh pages, which it takes
// from the free list at head + need[0] + .. + need[i-1].  Row r of the step belongs to the request
// with cu[i] <= r < cu[i+1] (cu = exclusive sums of new), has position past[i] + r - cu[i], and is
// written to slot page * page size + position mod page size.
//
// The work is two prefix sums over the requests and two searches through them (one per fresh page,
// one per row); the data is a few bytes per request, page and row, so the call is bound by launch
// and memory latency (64 decode requests 5.6 us).  One kernel does all of it: a single cluster of up to 8 CTAs,
// each of which repeats the prefix sums over all requests in its own shared memory (two loads per request) and
// then takes its share of the fresh pages and of the rows; with many rows those 8 SMs' searches are what takes the time
// (256 prompt chunks of up to 2048 rows 12.7 us).  The cluster barrier orders every read of
// the free-list head before its one write, and of the lengths before kv_lens, so head and lengths may be
// updated in place and a captured step replays.
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace qsa {
namespace {

constexpr int kThreadsPlan = 1024;
constexpr int kRowsPerThread = 4;

// a / d, ceil(a / d) for a >= 0 by a shift where d is a power of two (shift >= 0)
__device__ __forceinline__ int64_t div_floor(int64_t a, int32_t d, int32_t shift) {
  return shift >= 0 ? a >> shift : static_cast<int64_t>(static_cast<uint64_t>(a) / static_cast<uint32_t>(d));
}
__device__ __forceinline__ int32_t pages_of(const PagePlanParams& p, int64_t tokens) {
  const int64_t n = div_floor(tokens + p.page_size - 1, p.page_size, p.page_shift);
  return static_cast<int32_t>(n < p.pages_per_req ? n : p.pages_per_req);
}
__device__ __forceinline__ int32_t saturate(int64_t v) {
  return static_cast<int32_t>(v < INT32_MAX ? v : INT32_MAX);
}

// First i in [0, n) with sums[i + 1] > x; sums is non-decreasing and sums[n] > x.
__device__ __forceinline__ int32_t owner_of(const int32_t* sums, int32_t n, int32_t x) {
  int32_t lo = 0, hi = n - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi) >> 1;
    if (sums[mid + 1] > x) hi = mid; else lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ int64_t warp_inclusive(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

__global__ void __launch_bounds__(kThreadsPlan, 1) page_plan_kernel(const PagePlanParams p) {
  extern __shared__ int32_t sm[];
  int32_t* const cu = sm;                             // [n + 1] exclusive sums of new rows
  int32_t* const first = cu + p.n_requests + 1;       // [n + 1] exclusive sums of fresh pages
  int32_t* const past = first + p.n_requests + 1;     // [n]
  __shared__ int64_t warp_rows[32], warp_pages[32];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank());
  const int32_t n = p.n_requests;
  const int64_t n_free = p.n_free;
  int64_t head = __ldcg(p.free_head);
  head = head < 0 ? 0 : head > n_free ? n_free : head;

  // Prefix sums, 1024 requests at a time, in 64 bits (the lengths of a bad batch may add up past 32).
  int64_t rows_before = 0, pages_before = 0;
  for (int32_t c0 = 0; c0 < n; c0 += kThreadsPlan) {
    const int32_t i = c0 + tid;
    int64_t pi = 0, ni = 0;
    int32_t need = 0;
    if (i < n) {
      pi = max(__ldcg(p.past_lens + i), 0);
      ni = max(__ldcg(p.new_lens + i), 0);
      need = pages_of(p, pi + ni) - pages_of(p, pi);
    }
    const int64_t r = warp_inclusive(ni, lane), g = warp_inclusive(need, lane);
    if (lane == 31) {
      warp_rows[warp] = r;
      warp_pages[warp] = g;
    }
    __syncthreads();
    const int64_t wr = warp_rows[lane], wg = warp_pages[lane];   // 32 warps' totals
    const int64_t sr = warp_inclusive(wr, lane), sg = warp_inclusive(wg, lane);
    const int64_t r0 = rows_before + __shfl_sync(0xffffffffu, sr - wr, warp);
    const int64_t g0 = pages_before + __shfl_sync(0xffffffffu, sg - wg, warp);
    rows_before += __shfl_sync(0xffffffffu, sr, 31);
    pages_before += __shfl_sync(0xffffffffu, sg, 31);
    if (i < n) {
      const int64_t end = r0 + r;
      past[i] = static_cast<int32_t>(pi);
      cu[i + 1] = static_cast<int32_t>(end < p.max_rows ? end : p.max_rows);
      first[i + 1] = saturate(g0 + g);
      if (rank == 0) p.cu_seqlens_q[i + 1] = cu[i + 1];
      if (p.cluster == 1) p.kv_lens[i] = saturate(pi + ni);     // (this thread alone has read the lengths)
    }
    __syncthreads();   // the totals are overwritten by the next round
  }
  if (tid == 0) {
    cu[0] = 0;
    first[0] = 0;
    if (rank == 0) p.cu_seqlens_q[0] = 0;
  }
  // Every CTA of the cluster has read the free-list head before it is written (it may be the same word).
  if (p.cluster > 1) cluster_sync_all(); else __syncthreads();
  if (rank == 0 && tid == 0) {
    const int64_t wanted = head + pages_before;
    *p.free_head_out = static_cast<int32_t>(wanted < n_free ? wanted : n_free);
    if (p.shortfall) *p.shortfall = wanted > n_free ? saturate(wanted - n_free) : 0;
  }

  const int64_t stride = static_cast<int64_t>(p.cluster) * kThreadsPlan;
  const int64_t self = static_cast<int64_t>(rank) * kThreadsPlan + tid;
  // kv_lens may be past_lens or new_lens: where several CTAs read those, it is written behind the barrier
  if (p.cluster > 1) {
    for (int64_t i = self; i < n; i += stride)
      p.kv_lens[i] = saturate(static_cast<int64_t>(past[i]) + max(__ldcg(p.new_lens + i), 0));
  }
  // Fresh page k of the step goes to its request's next table entry (-1 past the end of the list).
  const int32_t n_fresh = first[n];
  for (int64_t k = self; k < n_fresh; k += stride) {
    const int32_t i = owner_of(first, n, static_cast<int32_t>(k));
    const int32_t entry = pages_of(p, past[i]) + static_cast<int32_t>(k - first[i]);
    const int64_t at = head + k;
    p.page_table[static_cast<int64_t>(i) * p.pages_per_req + entry] =
        at < n_free ? __ldg(p.free_pages + at) : -1;
  }
  if (p.positions == nullptr && p.slots == nullptr) return;

  // Rows: each thread finds the request of its first row and walks on from there.
  const int32_t live = cu[n];
  const bool vec = p.vec_rows != 0;
  for (int64_t r0 = self * kRowsPerThread; r0 < p.max_rows; r0 += stride * kRowsPerThread) {
    int32_t pos[kRowsPerThread], slot[kRowsPerThread];
    int32_t i = r0 < live ? owner_of(cu, n, static_cast<int32_t>(r0)) : n;
#pragma unroll
    for (int k = 0; k < kRowsPerThread; ++k) {
      const int64_t r = r0 + k;
      pos[k] = slot[k] = -1;
      if (r >= live) continue;
      while (cu[i + 1] <= r) ++i;
      const int64_t x = static_cast<int64_t>(past[i]) + (r - cu[i]);
      if (x > INT32_MAX) continue;
      pos[k] = static_cast<int32_t>(x);
      const int64_t e = div_floor(x, p.page_size, p.page_shift);
      if (e >= p.pages_per_req) continue;
      // a page taken in this call is read from the free list, an older one from the table
      const int32_t held = pages_of(p, past[i]);
      int32_t page = -1;
      if (e < held) {
        page = p.page_table[static_cast<int64_t>(i) * p.pages_per_req + e];
      } else {
        const int64_t at = head + first[i] + (e - held);
        if (at < n_free) page = __ldg(p.free_pages + at);
      }
      if (page < 0 || (p.n_pages > 0 && page >= p.n_pages)) continue;
      const int64_t s = static_cast<int64_t>(page) * p.page_size + (x - e * p.page_size);
      if (s <= INT32_MAX) slot[k] = static_cast<int32_t>(s);
    }
    if (vec && r0 + kRowsPerThread <= p.max_rows) {
      if (p.positions) *reinterpret_cast<int4*>(p.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      if (p.slots) *reinterpret_cast<int4*>(p.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int k = 0; k < kRowsPerThread; ++k) {
        if (r0 + k >= p.max_rows) break;
        if (p.positions) p.positions[r0 + k] = pos[k];
        if (p.slots) p.slots[r0 + k] = slot[k];
      }
    }
  }
}

}  // namespace

int page_plan_smem_bytes(int32_t n_requests) { return (3 * n_requests + 2) * 4; }

cudaError_t launch_page_plan(PagePlanParams p, cudaStream_t stream) {
  const int smem = page_plan_smem_bytes(p.n_requests);
  cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(page_plan_kernel),
                              page_plan_smem_bytes(kPlanMaxRequests), kOptPlan);
  if (e != cudaSuccess) return e;
  // A CTA for every 2048 rows or requests, at most the portable cluster size.
  const int64_t rows = p.positions || p.slots ? p.max_rows : 0;
  const int64_t work = rows > p.n_requests ? rows : p.n_requests;
  p.cluster = 1;
  while (p.cluster < 8 && static_cast<int64_t>(p.cluster) * 2048 < work) p.cluster *= 2;
  if (p.cluster == 1) {
    page_plan_kernel<<<1, kThreadsPlan, smem, stream>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.cluster));
  cfg.blockDim = dim3(kThreadsPlan);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, page_plan_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qsa
