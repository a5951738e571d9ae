// Bounds of a cache's pages, from which pages are chosen (score.cu, select.cuh).
//
// For every page that the step's rows reach, the smallest and the largest value of each key dim over the page's filled
// rows, lo and hi.  For a query q every key of the page has q.k <= sum_d max(q_d lo_d, q_d hi_d).
// A page's rows are read once, 16 bytes a thread, and reduced in packed 16-bit minima and maxima, which are exact.  The
// step's new rows lie in few pages, so latency bounds it: the search for a page's request, the lengths, the page id and the
// rows follow one another (64 decode rows, 2 heads of 256 dims: 4.9 us; 8619 prompt rows of four requests, 9 MB: 4.8 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "choose.cuh"
#include "internal.h"
#include "paged.cuh"

namespace qsa {
namespace {

using choose::best2;

constexpr int kBoundsThreads = 256;

// Numbers of pages before request i: cu / page size + 2 i leaves room for every page that its new rows lie in, and
// grows with i, so the owner of a number is found by search without a prefix sum.
__device__ __forceinline__ int64_t first_page(const PagedAddr& pa, int32_t i) {
  const int64_t cu = __ldg(pa.cu_seqlens_q + i);
  return (cu > 0 ? cu / pa.page_size : 0) + 2 * static_cast<int64_t>(i);
}
__device__ __forceinline__ int32_t page_owner(const PagedAddr& pa, int64_t page, int lane) {
  int32_t lo = 0, hi = pa.n_requests - 1;
  while (lo < hi) {
    const int32_t step = (hi - lo + 32) / 32;
    const int32_t cand = lo + lane * step;
    const uint32_t m = __ballot_sync(0xffffffffu, cand <= hi && first_page(pa, cand) <= page);
    const int last = m ? 31 - __clz(m) : 0;
    lo = lo + last * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

template <int D, typename T>
__global__ void __launch_bounds__(kBoundsThreads) page_bounds_kernel(const __grid_constant__ BoundsParams p) {
  constexpr int kCols = D / 8, kRows = kBoundsThreads / kCols;   // threads across a row, rows at a time
  __shared__ uint4 part[2][kRows][kCols];
  const int col = threadIdx.x % kCols, group = threadIdx.x / kCols, lane = threadIdx.x & 31;
  const int64_t pages = first_page(p.pa, p.pa.n_requests);
  for (int64_t item = blockIdx.x; item < pages * p.n_kvheads; item += gridDim.x) {
    const int64_t number = item / p.n_kvheads;
    const int32_t kvh = static_cast<int32_t>(item - number * p.n_kvheads);
    const int32_t req = page_owner(p.pa, number, lane);
    const int64_t kv = __ldg(p.pa.kv_lens + req);
    const int64_t fresh = static_cast<int64_t>(__ldg(p.pa.cu_seqlens_q + req + 1)) - __ldg(p.pa.cu_seqlens_q + req);
    const int64_t past = kv > fresh ? kv - fresh : 0;
    const int64_t nth = number - first_page(p.pa, req);   // (< 0 before the first request's rows, where they do not begin at 0)
    const int64_t e = past / p.pa.page_size + nth, start = e * p.pa.page_size;
    // (uniform over the block)
    if (nth < 0 || fresh <= 0 || start >= kv || e >= p.pa.pages_per_req) continue;
    const int32_t page = __ldg(p.pa.page_table + static_cast<int64_t>(req) * p.pa.pages_per_req + e);
    if (page < 0 || page >= p.pa.n_pages) continue;
    const int32_t filled = static_cast<int32_t>(kv - start < p.pa.page_size ? kv - start : p.pa.page_size);
    const T* const src = static_cast<const T*>(p.k_cache) +
                         (static_cast<int64_t>(page) * p.pa.page_size * p.n_kvheads + kvh) * D + col * 8;
    uint4 lo{}, hi{};
    auto take = [&](const uint4& x) {
      lo.x = best2<T, false>(lo.x, x.x);
      lo.y = best2<T, false>(lo.y, x.y);
      lo.z = best2<T, false>(lo.z, x.z);
      lo.w = best2<T, false>(lo.w, x.w);
    };
    auto take_hi = [&](const uint4& x) {
      hi.x = best2<T, true>(hi.x, x.x);
      hi.y = best2<T, true>(hi.y, x.y);
      hi.z = best2<T, true>(hi.z, x.z);
      hi.w = best2<T, true>(hi.w, x.w);
    };
    // (a group without rows of its own repeats the last one)
    const int32_t last = filled - 1;
    lo = hi = __ldg(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(min(group, last)) * p.n_kvheads * D));
#pragma unroll 8
    for (int32_t r = group + kRows; r <= last; r += kRows) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(r) * p.n_kvheads * D));
      take(x);
      take_hi(x);
    }
    part[0][group][col] = lo;
    part[1][group][col] = hi;
    __syncthreads();
    if (threadIdx.x < 2 * kCols) {
      const bool is_hi = threadIdx.x >= kCols;
      const int c = threadIdx.x % kCols;
      lo = hi = part[is_hi][0][c];
#pragma unroll 8
      for (int r = 1; r < kRows; ++r) {
        if (is_hi) take_hi(part[1][r][c]);
        else take(part[0][r][c]);
      }
      T* const out = static_cast<T*>(p.bounds) + ((static_cast<int64_t>(page) * p.n_kvheads + kvh) * 2 + is_hi) * D;
      *reinterpret_cast<uint4*>(out + c * 8) = is_hi ? hi : lo;
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_page_bounds(const BoundsParams& p, bool fp16, int num_sms, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(num_sms) * 8);
  auto go = [&](auto kern) {
    kern<<<grid, kBoundsThreads, 0, stream>>>(p);
    return cudaGetLastError();
  };
  if (fp16)
    return p.head_dim == 64    ? go(page_bounds_kernel<64, __half>)
           : p.head_dim == 128 ? go(page_bounds_kernel<128, __half>)
                               : go(page_bounds_kernel<256, __half>);
  return p.head_dim == 64    ? go(page_bounds_kernel<64, __nv_bfloat16>)
         : p.head_dim == 128 ? go(page_bounds_kernel<128, __nv_bfloat16>)
                             : go(page_bounds_kernel<256, __nv_bfloat16>);
}

}  // namespace qsa
