// Bounds of a cache's pages, and the choice of pages by them.
//
// Bounds: for every page that the step's rows reach, the smallest and the largest value of each key dim over the
// page's filled rows, lo and hi.  For a query q every key of the page has q.k <= sum_d max(q_d lo_d, q_d hi_d).
// A page's rows are read once, 16 bytes a thread, and reduced in packed 16-bit minima and maxima, which are exact.
//
// Choice: the score of a page is the largest of that bound over the query heads that share the KV head.  A row takes
// its first and last pages and, of the others up to its own, those with the highest scores (choose.cuh).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>
#include <type_traits>

#include "choose.cuh"
#include "internal.h"
#include "paged.cuh"

namespace qsa {
namespace {

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  using type = __nv_bfloat162;
};
template <>
struct Pair<__half> {
  using type = __half2;
};
// (NaN stays)
template <typename T, bool MAX>
__device__ __forceinline__ uint32_t best2(uint32_t a, uint32_t b) {
  typename Pair<T>::type x, y;
  memcpy(&x, &a, 4);
  memcpy(&y, &b, 4);
  x = MAX ? __hmax2_nan(x, y) : __hmin2_nan(x, y);
  memcpy(&a, &x, 4);
  return a;
}
template <typename T>
__device__ __forceinline__ float2 floats_of(uint32_t a) {
  typename Pair<T>::type x;
  memcpy(&x, &a, 4);
  if constexpr (std::is_same<T, __half>::value) return __half22float2(x);
  else return __bfloat1622float2(x);
}

// ---------------------------------------------------------------------------- bounds
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
    const int64_t e = past / p.pa.page_size + (number - first_page(p.pa, req)), start = e * p.pa.page_size;
    if (fresh <= 0 || start >= kv || e >= p.pa.pages_per_req) continue;    // (uniform over the block)
    const int32_t page = __ldg(p.pa.page_table + static_cast<int64_t>(req) * p.pa.pages_per_req + e);
    if (page < 0 || page >= p.pa.n_pages) continue;
    const int32_t filled = static_cast<int32_t>(kv - start < p.pa.page_size ? kv - start : p.pa.page_size);
    const T* const src = static_cast<const T*>(p.k_cache) +
                         (static_cast<int64_t>(page) * p.pa.page_size * p.n_kvheads + kvh) * D + col * 8;
    uint4 lo, hi;
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

// ---------------------------------------------------------------------------- choice
// fp32 sums of products that are exact in fp32, however they are grouped: the error stays below 2^-16 of the sum of
// the magnitudes, which is at most the sum of |q| times the largest bound.
constexpr float kScoreError = 0x1p-16f;

// Exact score of a page for `group` heads (whole warps): each lane takes D / 32 dims.
template <int D, typename T>
__device__ __forceinline__ double exact_score(const T* q, const T* bounds, int group, int lane) {
  constexpr int kPer = D / 32;
  float lo[kPer], hi[kPer];
#pragma unroll
  for (int c = 0; c < kPer; c += 2) {
    uint32_t a, b;
    memcpy(&a, bounds + lane * kPer + c, 4);
    memcpy(&b, bounds + D + lane * kPer + c, 4);
    const float2 x = floats_of<T>(a), y = floats_of<T>(b);
    lo[c] = x.x;
    lo[c + 1] = x.y;
    hi[c] = y.x;
    hi[c + 1] = y.y;
  }
  double best = -INFINITY;
  bool nan = false;
  for (int h = 0; h < group; ++h) {
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < kPer; c += 2) {
      uint32_t a;
      memcpy(&a, q + static_cast<int64_t>(h) * D + lane * kPer + c, 4);
      const float2 x = floats_of<T>(a);
      s += static_cast<double>(x.x) * (x.x > 0.0f ? hi[c] : lo[c]);
      s += static_cast<double>(x.y) * (x.y > 0.0f ? hi[c + 1] : lo[c + 1]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    nan |= s != s;
    best = s > best ? s : best;
  }
  return nan ? __longlong_as_double(0x7ff8000000000000ll) : best;
}

constexpr int kChooseThreads = 256;

// One block a row and KV head.
template <int D, typename T>
__global__ void __launch_bounds__(kChooseThreads) page_select_kernel(const __grid_constant__ ChooseParams p) {
  using namespace choose;
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t scratch[Team<kChooseThreads>::kScratch];
  Team<kChooseThreads> team(scratch);
  const int lane = team.lane, warp = team.warp;
  const int64_t row = blockIdx.x / p.n_kvheads;
  const int32_t kvh = static_cast<int32_t>(blockIdx.x - row * p.n_kvheads);
  if (row >= __ldg(p.pa.cu_seqlens_q + p.pa.n_requests)) return;
  const int32_t req = paged_request_of_row(p.pa, row, lane);
  const int64_t pos = static_cast<int64_t>(__ldg(p.pa.kv_lens + req)) - __ldg(p.pa.cu_seqlens_q + req + 1) + row;
  int32_t* const out = p.out + static_cast<int64_t>(blockIdx.x) * p.n_select;
  const int64_t mine = pos < 0 ? -1 : pos / p.pa.page_size;
  const int32_t n = static_cast<int32_t>(mine + 1 < p.pa.pages_per_req ? mine + 1 : p.pa.pages_per_req);
  const T* const q = static_cast<const T*>(p.q) + (row * p.n_qheads + static_cast<int64_t>(kvh) * p.group) * D;
  const T* const bounds = static_cast<const T*>(p.bounds) + static_cast<int64_t>(kvh) * 2 * D;
  const int32_t* const table = p.pa.page_table + static_cast<int64_t>(req) * p.pa.pages_per_req;
  constexpr int kPer = D / 32;
  uint32_t largest = 0;                                    // |q| summed, the largest bound: as bits
  float reach = 0.0f;
  for (int h = warp; h < p.group; h += Team<kChooseThreads>::kWarps) {
    float s = 0.0f;
    for (int c = 0; c < kPer; ++c) s += fabsf(static_cast<float>(q[static_cast<int64_t>(h) * D + lane * kPer + c]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    reach = s > reach || s != s ? s : reach;
  }
  for (int32_t e = warp; e < n; e += Team<kChooseThreads>::kWarps) {
    const int32_t page = __ldg(table + e);
    uint32_t key = 0;
    if (page >= 0 && page < p.pa.n_pages) {
      const T* const b = bounds + static_cast<int64_t>(page) * p.n_kvheads * 2 * D;
      float best = -INFINITY;
      bool nan = false;
      for (int h = 0; h < p.group; ++h) {
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
          const int d = lane * kPer + c;
          const float x = static_cast<float>(q[static_cast<int64_t>(h) * D + d]);
          const float lo = static_cast<float>(b[d]), hi = static_cast<float>(b[D + d]);
          s += x * (x > 0.0f ? hi : lo);
          largest = max(largest, max(__float_as_uint(lo) & 0x7fffffffu, __float_as_uint(hi) & 0x7fffffffu));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        nan |= s != s;
        best = fmaxf(best, s);
      }
      key = e < p.n_first || e > mine - p.n_last ? kChosen : nan ? kNan : key_of(best);
    }
    if (lane == 0) keys[e] = key;
  }
  __syncthreads();
  // (bits of non-negative floats have their order, NaN above all)
  reach = __uint_as_float(team.max(__float_as_uint(reach))) * __uint_as_float(team.max(largest));
  const float eps = reach < 0x1p126f ? reach * kScoreError : INFINITY;
  choose::choose(team, keys, n, p.n_select, eps,
                 [&](int32_t e) { return exact_score<D>(q, bounds + static_cast<int64_t>(__ldg(table + e)) * p.n_kvheads * 2 * D, p.group, lane); },
                 out);
}

template <int D, typename T>
cudaError_t launch_select_dim(const ChooseParams& p, cudaStream_t stream, int which) {
  auto kern = page_select_kernel<D, T>;
  const cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(kern), kMaxChoosePages * 4, kOptChoose + which);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(p.n_rows * p.n_kvheads), kChooseThreads, static_cast<size_t>(p.pa.pages_per_req) * 4, stream>>>(p);
  return cudaGetLastError();
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

cudaError_t launch_page_select(const ChooseParams& p, bool fp16, cudaStream_t stream) {
  if (fp16)
    return p.head_dim == 64    ? launch_select_dim<64, __half>(p, stream, 0)
           : p.head_dim == 128 ? launch_select_dim<128, __half>(p, stream, 1)
                               : launch_select_dim<256, __half>(p, stream, 2);
  return p.head_dim == 64    ? launch_select_dim<64, __nv_bfloat16>(p, stream, 3)
         : p.head_dim == 128 ? launch_select_dim<128, __nv_bfloat16>(p, stream, 4)
                             : launch_select_dim<256, __nv_bfloat16>(p, stream, 5);
}

}  // namespace qsa
