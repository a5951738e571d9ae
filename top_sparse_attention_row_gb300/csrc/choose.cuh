// The k best of a list of scores, decided as the exact scores decide (page selection, select.cuh).
//
// Scores come in fp32 with an error of at most eps each.  Let t be the k-th largest of them.  The k-th largest exact
// score is then within eps of t, so an entry above t + 2 eps belongs to the k best and one below t - 2 eps does not;
// where the entries between are more than the places left, their exact scores (64 bits) decide, equal ones by their
// place in the list.  (eps = 0: scores that are equal are so exactly.)
//
// Scores are held as unsigned keys that have their order, 0 for entries that cannot be chosen and kChosen for those
// that are in any case.  The k-th key is found by halving the range of keys and counting; the search ends as soon as a
// value parts the k best from the others: after about ten counts where scores are well spread, more where one lies far from
// the rest, 32 where equal scores straddle the last place.  The exact scores are taken in two
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
// The larger of |a|'s and |b|'s halves (a is not negative; NaN stays).
template <typename T>
__device__ __forceinline__ uint32_t largest2(uint32_t a, uint32_t b) { return best2<T, true>(a, b & 0x7fff7fffu); }
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

// The keys of a list, in registers: each warp of the team has a run of it, in which a lane has every 32nd entry.  Entries past
// the list's end have key 0, which nothing below counts.
template <int THREADS, int N>
struct Keys {
  uint32_t k[N];
  int32_t from;                                            // first entry of the warp's run
  __device__ __forceinline__ Keys(const Team<THREADS>& t, int32_t n) : from(t.warp * ((n + THREADS - 1) / THREADS) * 32) {}
  // entry j of this lane
  __device__ __forceinline__ int32_t place(const Team<THREADS>& t, int j) const { return from + j * 32 + t.lane; }
  template <typename F>
  __device__ __forceinline__ uint32_t count(Team<THREADS>& t, F f) const {
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) c += f(k[j]) ? 1u : 0u;
    return t.sum(c);
  }
  // two counts in one sum, of 16 bits each (THREADS N entries at most)
  template <typename F, typename G>
  __device__ __forceinline__ uint2 count(Team<THREADS>& t, F f, G g) const {
    static_assert(THREADS * N < 65536, "counts of 16 bits");
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) c += (f(k[j]) ? 1u : 0u) + (g(k[j]) ? 65536u : 0u);
    c = t.sum(c);
    return make_uint2(c & 0xffffu, c >> 16);
  }
};

// The want-th largest key (want >= 1, at least so many keys are not 0, fewer are kChosen).
template <int THREADS, int N>
__device__ __forceinline__ uint32_t kth_largest(Team<THREADS>& t, const Keys<THREADS, N>& keys, uint32_t want) {
  uint32_t top = 0, low = 0xffffffffu;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const uint32_t x = keys.k[j];
    top = x != kChosen ? max(top, x) : top;
    low = x != 0 ? min(low, x) : low;
  }
  uint32_t hi = t.max(top), lo = ~t.max(~low);             // the answer is in [lo, hi]
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    const uint32_t c = keys.count(t, [&](uint32_t x) { return x >= mid; });
    if (c >= want) lo = mid; else hi = mid - 1;
    if (c == want) {                                       // mid parts them: the smallest key from it on
      low = 0xffffffffu;
#pragma unroll
      for (int j = 0; j < N; ++j) low = keys.k[j] >= mid ? min(low, keys.k[j]) : low;
      return ~t.max(~low);
    }
  }
  return lo;
}

// What the warps before this one counted (`part`: 0 or 1, each once a list).
template <int THREADS>
__device__ __forceinline__ uint32_t before_warp(Team<THREADS>& t, uint32_t mine, int part) {
  if constexpr (THREADS == 32) return 0u;
  mine = __reduce_add_sync(0xffffffffu, mine);
  uint32_t* const r = t.red + (2 + part) * Team<THREADS>::kWarps;
  if (t.lane == 0) r[t.warp] = mine;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, t.lane < t.warp ? r[t.lane] : 0u);
}

// Writes the places of the keys above `bar`, and of the first `equal` ones equal to it, in order; then -1.  Changes the keys.
template <int THREADS, int N>
__device__ __forceinline__ void emit(Team<THREADS>& t, Keys<THREADS, N>& keys, uint32_t bar, uint32_t equal, int32_t k,
                                     int32_t* out) {
  const uint32_t before = (1u << t.lane) - 1u;
  if (equal != 0) {                                        // (rare) the first of the equal ones to kChosen, the others to 0
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) mine += keys.k[j] == bar;
    uint32_t same = before_warp(t, mine, 0);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint32_t s = __ballot_sync(0xffffffffu, keys.k[j] == bar);
      if (keys.k[j] == bar) keys.k[j] = same + __popc(s & before) < equal ? kChosen : 0u;
      same += __popc(s);
    }
    bar = min(bar, kChosen - 1u);
  }
  uint32_t mine = 0;
  if constexpr (THREADS > 32) {
#pragma unroll
    for (int j = 0; j < N; ++j) mine += keys.k[j] > bar;
  }
  uint32_t above = before_warp(t, mine, 1);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const bool in = keys.k[j] > bar;
    const uint32_t a = __ballot_sync(0xffffffffu, in), place = above + __popc(a & before);
    if (in && place < static_cast<uint32_t>(k)) out[place] = keys.place(t, j);
    above += __popc(a);
  }
  // the last warp has counted them all
  if (t.warp == Team<THREADS>::kWarps - 1) {
    for (int32_t i = static_cast<int32_t>(above) + t.lane; i < k; i += 32) out[i] = -1;
  }
}

// Replaces the keys from lo to hi by value(place), a function of whole warps, those above by kChosen, those below by 0.
template <int THREADS, int N, typename F>
__device__ __forceinline__ void refine(Team<THREADS>& t, Keys<THREADS, N>& keys, uint32_t lo, uint32_t hi, F value) {
  uint32_t open = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const uint32_t x = keys.k[j];
    if (x >= lo && x <= hi) open |= 1u << j;
    keys.k[j] = x > hi ? kChosen : 0u;
  }
  while (true) {
    const uint32_t lanes = __ballot_sync(0xffffffffu, open != 0);
    if (lanes == 0) break;
    const int l = __ffs(lanes) - 1, j = __ffs(__shfl_sync(0xffffffffu, open, l)) - 1;
    const uint32_t y = value(keys.from + j * 32 + l);
    if (t.lane == l) {
      open &= open - 1;
#pragma unroll
      for (int i = 0; i < N; ++i) keys.k[i] = i == j ? y : keys.k[i];
    }
  }
}

// Chooses the k best of the keys (changed by the call) and writes their places in order, then -1.
// exact(i), called by whole warps, is the 64-bit key of entry i's score.
template <int THREADS, int N, typename Exact>
__device__ __forceinline__ void choose(Team<THREADS>& t, Keys<THREADS, N>& keys, int32_t k, float eps, Exact exact,
                                       int32_t* out) {
  static_assert(N <= 32, "a lane's entries as bits");
  const uint32_t want = static_cast<uint32_t>(k);
  const uint2 n = keys.count(t, [](uint32_t x) { return x != 0; }, [](uint32_t x) { return x == kChosen; });
  uint32_t bar = 0u, equal = 0u;                           // (all there are)
  if (n.y >= want) {
    bar = kChosen;
    equal = want;
  } else if (n.x > want) {
    // by the scores, then by the upper halves of the exact ones that are close, then by their lower halves (one loop, so that
    // its code is there once: written out three times it did not stay in the instruction cache)
#pragma unroll 1
    for (int stage = 0;; ++stage) {
      bar = kth_largest(t, keys, want);
      uint32_t lo = bar, hi = bar;
      if (stage == 0 && eps != 0.0f) {
        const float s = score_of(bar), e2 = 2.0f * eps;
        const bool bounded = bar != kNan && isfinite(s) && isfinite(e2);
        lo = bounded ? key_of(__fsub_rd(s, e2)) : 1u;      // no bound on the error: all may belong
        hi = bounded ? key_of(__fadd_ru(s, e2)) : kNan;
      }
      const uint2 m = keys.count(t, [&](uint32_t x) { return x > hi; }, [&](uint32_t x) { return x >= lo; });
      if (m.y == want) {
        bar = lo - 1u;
        break;
      }
      equal = want - m.x;
      if (stage == 2 || eps == 0.0f) break;                // they are equal
      equal = 0u;
      // (0 and kChosen stay free: the last of the 64 bits is left out)
      refine(t, keys, lo, hi, [&](int32_t i) {
        const uint64_t x = exact(i);
        return stage == 0 ? static_cast<uint32_t>(x >> 32) : 1u + (static_cast<uint32_t>(x) >> 1);
      });
    }
  }
  emit(t, keys, bar, equal, k, out);
}

}  // namespace choose
}  // namespace qsa
