// The choice of pages by their scores: the score of a page is the largest bound of q.k over the query heads that share the
// KV head (score.cu).  A row takes its first and last pages and, of the others up to its own, those with the highest scores
// (choose.cuh).
#pragma once

#include "choose.cuh"
#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace qsa {

using choose::floats_of;

// The tensor core's error of a score, as a part of the sum of |q| times the largest bound (which is no less than the sum of the
// products' magnitudes).  Products are exact in fp32; 2 D / 16 times, sixteen of them and the sum so far are added and cut
// to 24 bits, which takes off up to 2^-23 of the magnitudes each time: D 2^-26, and half as much again for the alignment
// within the sixteen.  Measured: up to 2^-18.3 of the magnitudes for 256 dims whose bounds lie anywhere from 2^-12 to 2^12,
// and at most 2^-21.1 of what this bound is a part of (2^-17).
template <int D>
constexpr float kScoreError = D * 0x1p-25f;

// s + x as the nearest float and what is left of it (Knuth's two-sum): exact.
__device__ __forceinline__ float two_sum(float s, float x, float* rest) {
  const float t = s + x, z = t - s;
  *rest = (s - (t - z)) + (x - z);
  return t;
}

// One head's score in two floats (whole warps; each lane has D / 32 dims).
template <int PER>
__device__ __forceinline__ uint64_t two_float_key(const float (&x)[PER], const float (&lo)[PER], const float (&hi)[PER]) {
  float s = 0.0f, rest = 0.0f, r;
#pragma unroll
  for (int c = 0; c < PER; ++c) {
    s = two_sum(s, __fmul_rn(x[c], x[c] > 0.0f ? hi[c] : lo[c]), &r);
    rest += r;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s = two_sum(s, __shfl_xor_sync(0xffffffffu, s, o), &r);
    rest += __shfl_xor_sync(0xffffffffu, rest, o);
    rest += r;
  }
  s = two_sum(s, rest, &r);
  return choose::key_of(s, r);
}
template <int PER, typename T>
__device__ __forceinline__ void load_dims(const T* p, float (&x)[PER]) {
  uint32_t w[PER / 2];
  if constexpr (PER == 8) {
    const uint4 y = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = y.x;
    w[1] = y.y;
    w[2] = y.z;
    w[3] = y.w;
  } else if constexpr (PER == 4) {
    const uint2 y = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = y.x;
    w[1] = y.y;
  } else {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
#pragma unroll
  for (int c = 0; c < PER; c += 2) {
    const float2 y = floats_of<T>(w[c / 2]);
    x[c] = y.x;
    x[c + 1] = y.y;
  }
}

// The key of a page's score for `group` heads, to compare scores that the products' fp32 sums cannot part (by whole
// warps; each lane takes D / 32 dims).  A product of two 16-bit values is exact in fp32; sums are kept in two floats,
// whose error is below 2^-44 of the sum of the magnitudes, for the heads that come within fp32's error of the largest:
// eight heads' fp32 sums are taken at a time, with exchanges that halve them.  Doubles would do too, but this GPU adds
// few of them (two a cycle and SM: 230 us of 468 for 8192 prompt rows), so they are left to scores that floats cannot hold
// (`wide`): all pages of a row over whose pages a bound is not finite, for one (one infinity in a prompt of 24k: 89 ms in
// place of 0.2 for 8192 rows; one in the context of one of 64 decode rows: 3.6 ms in place of 0.06).  reach: sum of |q| times the largest bound.
template <int D, typename T>
__device__ __forceinline__ uint64_t exact_key(const T* q, const T* bounds, int group, int lane, float reach, bool wide) {
  constexpr int kPer = D / 32, kHeads = 8;
  float lo[kPer], hi[kPer];
  load_dims<kPer>(bounds + lane * kPer, lo);
  load_dims<kPer>(bounds + D + lane * kPer, hi);
  q += lane * kPer;
  uint64_t best = 0;
  if (wide) {
    for (int h = 0; h < group; ++h) {
      float x[kPer];
      load_dims<kPer>(q + static_cast<int64_t>(h) * D, x);
      double s = 0.0;
#pragma unroll
      for (int c = 0; c < kPer; ++c) s += static_cast<double>(x[c]) * (x[c] > 0.0f ? hi[c] : lo[c]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const uint64_t key = choose::key_of(s);
      best = key > best ? key : best;
    }
    return best;
  }
  const float margin = reach * 0x1p-18f;                   // twice the error of a sum of 13 roundings
  float most = -INFINITY;
  for (int h0 = 0; h0 < group; h0 += kHeads) {
    float v[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      float x[kPer];
      load_dims<kPer>(q + static_cast<int64_t>(min(h0 + h, group - 1)) * D, x);
      v[h] = 0.0f;
#pragma unroll
      for (int c = 0; c < kPer; ++c) v[h] = fmaf(x[c], x[c] > 0.0f ? hi[c] : lo[c], v[h]);
    }
    // lane l comes out with the sum of head h0 + l / 4
    int n = kHeads;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (o >= 4) {
        n >>= 1;
        const bool up = lane & o;
#pragma unroll
        for (int c = 0; c < kHeads / 2; ++c) {
          if (c < n) {
            const float send = up ? v[c] : v[c + n], keep = up ? v[c + n] : v[c];
            v[c] = keep + __shfl_xor_sync(0xffffffffu, send, o);
          }
        }
      } else {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
      }
    }
    float m = v[0];
#pragma unroll
    for (int o = 16; o >= 4; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    most = fmaxf(most, m);
    const uint32_t near = __ballot_sync(0xffffffffu, (lane & 3) == 0 && h0 + lane / 4 < group && v[0] >= most - margin);
    for (uint32_t left = near; left; left &= left - 1) {
      float x[kPer];
      load_dims<kPer>(q + static_cast<int64_t>(h0 + (__ffs(left) - 1) / 4) * D, x);
      const uint64_t key = two_float_key<kPer>(x, lo, hi);
      best = key > best ? key : best;
    }
  }
  return best;
}

// A team of threads takes a row and KV head: a warp where there are many, else a block.  A lane has N of its pages' keys.
// (Blocks of four warps: a row whose close scores are summed anew takes several times as long as the others, and holds up
// few of them.)
constexpr int kWarpTeams = 4;
template <int D, typename T, int TEAM, int N>
__global__ void __launch_bounds__(TEAM == 32 ? 32 * kWarpTeams : TEAM, TEAM == 32 && N <= 16 ? 8 : 1)
    page_select_kernel(const __grid_constant__ ChooseParams p) {
  using namespace choose;
  constexpr int kTeams = TEAM == 32 ? kWarpTeams : 1;
  __shared__ uint32_t scratch[TEAM == 32 ? 1 : Team<TEAM>::kScratch];
  pdl_wait();
  Team<TEAM> team(scratch);
  const int lane = team.lane;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kTeams + (TEAM == 32 ? threadIdx.x >> 5 : 0), row = item / p.n_kvheads;
  const int32_t kvh = static_cast<int32_t>(item - row * p.n_kvheads);
  if (row >= p.n_rows || row >= __ldg(p.pa.cu_seqlens_q + p.pa.n_requests)) return;
  const int32_t req = paged_request_of_row(p.pa, row, lane);
  if (row < __ldg(p.pa.cu_seqlens_q + req)) return;        // before the first request
  const int64_t pos = static_cast<int64_t>(__ldg(p.pa.kv_lens + req)) - __ldg(p.pa.cu_seqlens_q + req + 1) + row;
  int32_t* const out = p.out + item * p.n_select;
  const int64_t mine = pos < 0 ? -1 : pos / p.pa.page_size;
  const int32_t n = static_cast<int32_t>(mine + 1 < p.pa.pages_per_req ? mine + 1 : p.pa.pages_per_req);
  const int32_t* const table = p.pa.page_table + static_cast<int64_t>(req) * p.pa.pages_per_req;
  Keys<TEAM, N> keys(team, n);
  const int32_t to = min(keys.from + (n + TEAM - 1) / TEAM * 32, n);   // end of this warp's run
  float reach = 0.0f, eps = 0.0f;
  bool wide = false;
  if (n <= p.n_select) {                                   // every page that exists (no scores have been taken)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int32_t e = keys.place(team, j), page = e < to ? __ldg(table + e) : -1;
      keys.k[j] = page >= 0 && page < p.pa.n_pages ? kChosen : 0u;
    }
  } else {
    // (plain loads of what the score kernel writes, which may still run when this one starts: non-coherent ones are for
    // what nobody writes from then on)
    const uint32_t* const src = p.keys + item * p.key_stride;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int32_t e = keys.place(team, j);
      keys.k[j] = e < to ? src[e] : 0u;
    }
    // (bits of non-negative floats have their order, NaN above all)
    uint32_t most = 0;
    const float* const largest = p.largest + (static_cast<int64_t>(req) * p.n_kvheads + kvh) * p.bound_tiles;
    for (int32_t i = lane; i * kBoundTile < n; i += 32) most = max(most, __float_as_uint(largest[i]));
    const float q_sum = p.reach[item], bound = __uint_as_float(__reduce_max_sync(0xffffffffu, most));
    reach = q_sum * bound;
    // beyond these, sums overflow or products lose bits in fp32 (NaN fails all comparisons)
    wide = !(reach < 0x1p126f && reach > 0x1p-80f && q_sum > 0x1p-100f && bound > 0x1p-100f);
    // sums of zeros are exact (0 times infinity or NaN is none: those scores are taken anew)
    const bool zeros = (q_sum == 0.0f && bound < INFINITY) || (bound == 0.0f && q_sum < INFINITY);
    eps = zeros ? 0.0f : wide ? INFINITY : reach * kScoreError<D>;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int32_t e = keys.place(team, j);
      if (keys.k[j] != 0 && (e < p.n_first || e > mine - p.n_last)) keys.k[j] = kChosen;
    }
  }
  const T* const q = static_cast<const T*>(p.q) + (row * p.n_qheads + static_cast<int64_t>(kvh) * p.group) * D;
  const T* const bounds = static_cast<const T*>(p.bounds) + static_cast<int64_t>(kvh) * 2 * D;
  choose::choose(team, keys, p.n_select, eps,
                 [&](int32_t e) -> uint64_t {
                   const int32_t page = __ldg(table + e);
                   if (page < 0 || page >= p.pa.n_pages) return 0;   // (has no key, unless the scores were given up)
                   return exact_key<D>(q, bounds + static_cast<int64_t>(page) * p.n_kvheads * 2 * D, p.group, lane, reach, wide);
                 },
                 out);
}

template <int D, typename T, int TEAM, int N>
cudaError_t launch_select_team(const ChooseParams& p, cudaStream_t stream) {
  constexpr int kTeams = TEAM == 32 ? kWarpTeams : 1;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // starts while the scores are taken
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>((p.n_rows * p.n_kvheads + kTeams - 1) / kTeams));
  cfg.blockDim = dim3(TEAM == 32 ? 32 * kWarpTeams : TEAM);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, page_select_kernel<D, T, TEAM, N>, p);
}
// A team's size.  A warp does a row of up to 1024 pages with a fraction of a block's instructions and without its barriers,
// but takes longer; a block is for few rows and for longer lists.  Whole calls, us, warps / blocks, 24/2 heads of 256 dims:
// one row of 512 pages 20.7 / 15.6, 64 rows 47.9 / 33.3, 400 rows 115 / 106, 600 rows 51.3 / 53.1, 8192 rows 208 / 411;
// 1000 rows of 110 pages 33.3 / 55.1; 300 rows of 938 pages 135 / 127, 4000 rows 220 / 279.  (Both with the choice's steps
// written out; with one loop and a plain emission 8192 rows take 196.)
template <int D, typename T>
cudaError_t launch_select_type(const ChooseParams& p, int num_sms, cudaStream_t stream) {
  const int32_t n = p.pa.pages_per_req;
  const int64_t rows = p.n_rows * p.n_kvheads;
  const int64_t per_sm = rows / num_sms;
  if (n <= 128 && per_sm >= 2) return launch_select_team<D, T, 32, 4>(p, stream);
  if (n <= 512 && per_sm >= 8) return launch_select_team<D, T, 32, 16>(p, stream);
  if (n <= 1024 && per_sm >= 16) return launch_select_team<D, T, 32, 32>(p, stream);
  if (n <= 2048) return launch_select_team<D, T, 256, 8>(p, stream);
  return n <= 8192 ? launch_select_team<D, T, 1024, 8>(p, stream) : launch_select_team<D, T, 1024, 32>(p, stream);
}
template <int D>
cudaError_t launch_select_dim(const ChooseParams& p, bool fp16, int num_sms, cudaStream_t stream) {
  return fp16 ? launch_select_type<D, __half>(p, num_sms, stream) : launch_select_type<D, __nv_bfloat16>(p, num_sms, stream);
}

}  // namespace qsa
