// The k best of a list of scores, decided as the exact scores decide (page selection, choose.cu).
//
// Scores come in fp32 with an error of at most eps each.  Let t be the k-th largest of them.  The k-th largest exact
// score is then within eps of t, so an entry above t + 2 eps belongs to the k best and one below t - 2 eps does not;
// where the entries between are more than the places left, their exact scores (64 bits) decide, equal ones by their
// place in the list.  (eps = 0: scores that are equal are so exactly.)
//
// Scores are held as unsigned keys that have their order, 0 for entries that cannot be chosen and kChosen for those
// that are in any case.  The k-th key is found by halving the range of keys and counting; the search ends as soon as a
// value parts the k best from the others, after log2(entries) + 3 or so counts.  The exact scores are taken in two
// steps, their upper and their lower halves, so that they need no more room than the keys, however many there are.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

namespace qsa {
namespace choose {

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

constexpr uint32_t kChosen = 0xffffffffu;
constexpr uint32_t kNan = 0xfffffffeu;      // a score that is NaN stands above all others

__device__ __forceinline__ uint32_t key_of(float s) {
  if (s != s) return kNan;
  const uint32_t b = __float_as_uint(s + 0.0f);            // (-0 becomes 0)
  return b >> 31 ? ~b : b | 0x80000000u;                   // infinities: 0x007fffff and 0xff800000
}
__device__ __forceinline__ float score_of(uint32_t key) {
  return __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key);
}
// A score in two floats, hi + lo with hi the nearest float: ordered like (hi, lo).
__device__ __forceinline__ uint64_t key_of(float hi, float lo) {
  return static_cast<uint64_t>(key_of(hi)) << 32 | key_of(lo);
}
__device__ __forceinline__ uint64_t key_of(double s) {
  if (s != s) return static_cast<uint64_t>(kNan) << 32;
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(s + 0.0));
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

// The threads that work on one list: a warp, or a whole block.
template <int THREADS>
struct Team {
  static constexpr int kWarps = THREADS / 32;
  static constexpr int kScratch = 4 * kWarps;              // uint32 of shared memory
  uint32_t* red;
  int lane, warp;
  int turn = 0;
  __device__ __forceinline__ Team(uint32_t* scratch)
      : red(scratch), lane(threadIdx.x & 31), warp(THREADS == 32 ? 0 : threadIdx.x >> 5) {}
  __device__ __forceinline__ void sync() {
    if constexpr (THREADS == 32) __syncwarp();
    else __syncthreads();
  }
  // (two halves of the scratch in turn: one barrier a call)
  __device__ __forceinline__ uint32_t sum(uint32_t v) {
    v = __reduce_add_sync(0xffffffffu, v);
    if constexpr (THREADS > 32) {
      uint32_t* const r = red + turn * kWarps;
      turn ^= 1;
      if (lane == 0) r[warp] = v;
      __syncthreads();
      v = __reduce_add_sync(0xffffffffu, lane < kWarps ? r[lane] : 0u);
    }
    return v;
  }
  __device__ __forceinline__ uint32_t max(uint32_t v) {
    v = __reduce_max_sync(0xffffffffu, v);
    if constexpr (THREADS > 32) {
      uint32_t* const r = red + turn * kWarps;
      turn ^= 1;
      if (lane == 0) r[warp] = v;
      __syncthreads();
      v = __reduce_max_sync(0xffffffffu, lane < kWarps ? r[lane] : 0u);
    }
    return v;
  }
};

// Keys [n] in shared memory, each warp of the team owns a run of them (whole 32s).
template <int THREADS>
struct Run {
  int32_t from, to;
  __device__ __forceinline__ Run(const Team<THREADS>& t, int32_t n) {
    const int32_t per = ((n + THREADS - 1) / THREADS) * 32;
    from = t.warp * per;
    to = from + per < n ? from + per : n;
  }
};

template <int THREADS, typename F>
__device__ __forceinline__ uint32_t count_if(Team<THREADS>& t, const uint32_t* keys, int32_t n, F f) {
  const Run<THREADS> run(t, n);
  uint32_t c = 0;
  for (int32_t i = run.from + t.lane; i < run.to; i += 32) c += f(keys[i]) ? 1u : 0u;
  return t.sum(c);
}

// The k-th largest key (k >= 1, at least k keys are not 0, fewer than k are kChosen).
template <int THREADS>
__device__ __forceinline__ uint32_t kth_largest(Team<THREADS>& t, const uint32_t* keys, int32_t n, uint32_t k) {
  const Run<THREADS> run(t, n);
  uint32_t top = 0, low = 0xffffffffu;
  for (int32_t i = run.from + t.lane; i < run.to; i += 32) {
    const uint32_t x = keys[i];
    if (x != kChosen && x > top) top = x;
    if (x != 0 && x < low) low = x;
  }
  uint32_t hi = t.max(top), lo = ~t.max(~low);             // the answer is in [lo, hi]
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    const uint32_t c = count_if(t, keys, n, [&](uint32_t x) { return x >= mid; });
    if (c >= k) lo = mid; else hi = mid - 1;
    if (c == k) {                                          // mid parts them: the smallest key from it on
      low = 0xffffffffu;
      for (int32_t i = run.from + t.lane; i < run.to; i += 32) low = keys[i] >= mid && keys[i] < low ? keys[i] : low;
      return ~t.max(~low);
    }
  }
  return lo;
}

// Writes the places of the keys above `bar`, and of the first `equal` ones equal to it, in order; then -1.
template <int THREADS>
__device__ __forceinline__ void emit(Team<THREADS>& t, const uint32_t* keys, int32_t n, uint32_t bar, uint32_t equal,
                                     int32_t k, int32_t* out) {
  const Run<THREADS> run(t, n);
  uint32_t above = 0, same = 0;                            // in the runs before this warp's
  if constexpr (THREADS > 32) {
    uint32_t a = 0, s = 0;
    for (int32_t i = run.from + t.lane; i < run.to; i += 32) {
      a += keys[i] > bar;
      s += keys[i] == bar;
    }
    a = __reduce_add_sync(0xffffffffu, a);
    s = __reduce_add_sync(0xffffffffu, s);
    uint32_t* const r = t.red + 2 * Team<THREADS>::kWarps;
    if (t.lane == 0) {
      r[2 * t.warp] = a;
      r[2 * t.warp + 1] = s;
    }
    __syncthreads();
    above = __reduce_add_sync(0xffffffffu, t.lane < t.warp ? r[2 * t.lane] : 0u);
    same = __reduce_add_sync(0xffffffffu, t.lane < t.warp ? r[2 * t.lane + 1] : 0u);
  }
  const uint32_t before = (1u << t.lane) - 1u;
  for (int32_t i = run.from; i < run.to; i += 32) {
    const uint32_t x = i + t.lane < run.to ? keys[i + t.lane] : 0u;
    const bool in = i + t.lane < run.to;
    const uint32_t a = __ballot_sync(0xffffffffu, in && x > bar), s = __ballot_sync(0xffffffffu, in && x == bar);
    const uint32_t my_above = above + __popc(a & before), my_same = same + __popc(s & before);
    const uint32_t place = my_above + (my_same < equal ? my_same : equal);
    if (in && (x > bar || (x == bar && my_same < equal)) && place < static_cast<uint32_t>(k))
      out[place] = i + t.lane;
    above += __popc(a);
    same += __popc(s);
  }
  // the last warp has counted them all
  if (t.warp == Team<THREADS>::kWarps - 1) {
    const uint32_t all = above + (same < equal ? same : equal);
    for (int32_t i = static_cast<int32_t>(all) + t.lane; i < k; i += 32) out[i] = -1;
  }
}

// Chooses the k best of keys [n] (shared memory, changed by the call) and writes their places in order, then -1.
// exact(i), called by whole warps, is the 64-bit key of entry i's score.
template <int THREADS, typename Exact>
__device__ __forceinline__ void choose(Team<THREADS>& t, uint32_t* keys, int32_t n, int32_t k, float eps, Exact exact,
                                       int32_t* out) {
  const uint32_t want = static_cast<uint32_t>(k);
  if (count_if(t, keys, n, [](uint32_t x) { return x != 0; }) <= want) {
    emit(t, keys, n, 0u, 0u, k, out);
    return;
  }
  if (count_if(t, keys, n, [](uint32_t x) { return x == kChosen; }) >= want) {
    emit(t, keys, n, kChosen, want, k, out);
    return;
  }
  const uint32_t bar = kth_largest(t, keys, n, want);
  const float s = score_of(bar), e2 = 2.0f * eps;
  uint32_t lo = 1u, hi = kNan;                             // no bound on the error: all may belong
  if (bar != kNan && isfinite(s) && isfinite(e2)) {
    lo = key_of(__fsub_rd(s, e2));
    hi = key_of(__fadd_ru(s, e2));
  }
  const uint32_t sure = count_if(t, keys, n, [&](uint32_t x) { return x > hi; });
  const uint32_t open = count_if(t, keys, n, [&](uint32_t x) { return x >= lo && x <= hi; });
  if (sure + open == want) {
    emit(t, keys, n, lo - 1u, 0u, k, out);
    return;
  }
  if (eps == 0.0f) {                                       // they are equal
    emit(t, keys, n, bar, want - sure, k, out);
    return;
  }
  const Run<THREADS> run(t, n);
  t.sync();                                                // the keys have been read by all
  for (int32_t i = run.from; i < run.to; i += 32) {
    const uint32_t x = i + t.lane < run.to ? keys[i + t.lane] : 0u;
    uint32_t y = x > hi ? kChosen : 0u;
    for (uint32_t m = __ballot_sync(0xffffffffu, x >= lo && x <= hi); m; m &= m - 1) {
      const int j = __ffs(m) - 1;
      const uint64_t v = exact(i + j);
      if (t.lane == j) y = static_cast<uint32_t>(v >> 32);
    }
    if (i + t.lane < run.to) keys[i + t.lane] = y;
  }
  t.sync();
  const uint32_t upper = kth_largest(t, keys, n, want);
  uint32_t over = count_if(t, keys, n, [&](uint32_t x) { return x > upper; });
  if (over + count_if(t, keys, n, [&](uint32_t x) { return x == upper; }) == want) {
    emit(t, keys, n, upper, want - over, k, out);
    return;
  }
  t.sync();
  for (int32_t i = run.from; i < run.to; i += 32) {
    const uint32_t x = i + t.lane < run.to ? keys[i + t.lane] : 0u;
    uint32_t y = x > upper ? kChosen : 0u;
    for (uint32_t m = __ballot_sync(0xffffffffu, x == upper && i + t.lane < run.to); m; m &= m - 1) {
      const int j = __ffs(m) - 1;
      const uint64_t v = exact(i + j);
      // (0 and kChosen stay free: the last of the 64 bits is left out)
      if (t.lane == j) y = 1u + (static_cast<uint32_t>(v) >> 1);
    }
    if (i + t.lane < run.to) keys[i + t.lane] = y;
  }
  t.sync();
  const uint32_t lower = kth_largest(t, keys, n, want);
  over = count_if(t, keys, n, [&](uint32_t x) { return x > lower; });
  emit(t, keys, n, lower, want - over, k, out);
}

}  // namespace choose
}  // namespace qsa
