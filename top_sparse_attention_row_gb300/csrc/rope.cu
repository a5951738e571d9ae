// Rotary positions, and the write of new K/V rows into the cache, as they are or in 4 bits.
//
// Pair (a, b) of a head at position x turns by the angle x * theta_i: a' = m (a cos - b sin),
// b' = m (b cos + a sin).  The pairs are dims (i, i + rot/2) in the half layout and (2i, 2i + 1) in the
// interleaved one.  theta_i comes as a step: the fraction of a full turn per token, as a 64-bit
// fixed-point number.  x * step modulo 2^64, one integer product, is then that step's angle as a fraction of
// a turn at any 31-bit position (theta_i * x in fp32 is off by 2^-24 of the whole angle, 0.06 rad at a
// million; the steps themselves are made in doubles, 2^-53 turns per token).  Its upper half, as a signed
// number of half turns, is rounded to fp32 (2^-25 half turns) and goes to sincospi.
//
// The operator reads and writes every element once and does a handful of operations on each, so it is
// bound by memory (8192 rows of 24 q, 2 k and 2 v heads of 256 dims 42.6 us, 5.5 TB/s: 81 % of the measured copy
// rate).  A thread owns one 16-dim unit (8 pairs) of a row: it computes its 8 sines and cosines once and applies them
// to that unit of every head of its share, with 16-byte loads and stores.  Calls with few rows give each thread
// fewer heads, so that enough threads run.
//
// 4-bit rows: a block of 16 dims is stored as 16 e2m1 codes (two in a byte, the even dim in the low
// half) and one e4m3 scale s = e4m3(max|x| / (6 g)), g being the cache's fp32 scale; a code is
// e2m1((x / g) / s), both rounded to nearest, ties to even.  The rotated values are quantised from fp32.
// 8192 rows of 2 + 2 heads of 256 dims take 11.5 us, where their 38 MB need 5.6: a thread's loads, maximum, scale and
// codes follow one another, two heads deep.
// Codes and scales fall as the formula says, ties (x = border times scales: common, since all have few bits)
// and values next to them included: see quantise8.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "internal.h"

namespace qsa {
namespace {

constexpr int kRopeThreads = 128;

__device__ __forceinline__ float2 unpack2(uint32_t v, __nv_bfloat16) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t v, __half) {
  __half2 h;
  memcpy(&h, &v, 4);
  return __half22float2(h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  uint32_t r;
  memcpy(&r, &h, 4);
  return r;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  uint32_t r;
  memcpy(&r, &h, 4);
  return r;
}
// (plain loads: q may be rotated in place)
// The two 8-element halves of a unit at elements `a` and `b`; b = a + 8 where `joined`, and one 32-byte access
// then takes both where the rows allow it.
template <typename T>
__device__ __forceinline__ void load_halves(const void* base, int64_t row, int a, int b, bool joined, uint4& ra, uint4& rb) {
  const T* const p = static_cast<const T*>(base) + row;
  if (joined) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(ra.x), "=r"(ra.y), "=r"(ra.z), "=r"(ra.w), "=r"(rb.x), "=r"(rb.y), "=r"(rb.z), "=r"(rb.w)
                 : "l"(p + a)
                 : "memory");
  } else {
    ra = *reinterpret_cast<const uint4*>(p + a);
    rb = *reinterpret_cast<const uint4*>(p + b);
  }
}
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 t = unpack2(w[k], T{});
    f[2 * k] = t.x;
    f[2 * k + 1] = t.y;
  }
}
template <typename T>
__device__ __forceinline__ void store_halves(void* base, int64_t row, int a, int b, bool joined, const float* f) {
  T* const p = static_cast<T*>(base) + row;
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = pack2(f[2 * k], f[2 * k + 1], T{});
  if (joined) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + a), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(p + a) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(p + b) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Sine and cosine of the angle at position `pos`, times the magnitude.
__device__ __forceinline__ void angle_of(const RopeParams& p, int i, int32_t pos, float& c, float& s) {
  const uint64_t turn = static_cast<uint64_t>(static_cast<uint32_t>(pos)) * p.steps[i];
  const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
  sincospif(half_turns, &s, &c);
  c *= p.magnitude;
  s *= p.sin_sign;   // the magnitude, negative for the transpose
}

// Eight values as e2m1 codes, nearest with ties to even, four bits each from the lowest on.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// The values of eight codes.
__device__ __forceinline__ void e2m1x8_values(uint32_t w, float* v) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 t = unpack2(h[k], __half{});
    v[2 * k] = t.x;
    v[2 * k + 1] = t.y;
  }
}
__device__ __forceinline__ uint8_t e4m3_of(float a) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(a));
  return static_cast<uint8_t>(r);
}
__device__ __forceinline__ float e4m3_value(uint8_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(c)));
  return unpack2(r, __half{}).x;
}
__device__ __forceinline__ float amax8(const float* f) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int k = 1; k < 8; ++k) m = fmaxf(m, fabsf(f[k]));
  return m;
}

__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 split_pair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Quotients of f by the divisor d (few bits), r being 1 / d to within some ulp.  The product p = f r is corrected
// by its residual: f - p d is exact in fp32, so p + (f - p d) r is the quotient to 2^-44 of itself before its one
// rounding.  That decides as the exact quotient does, ties included: a border between two codes or scales has at
// most 5 bits, so border times d is a float, another float f is at least 2^-24 of it away, and the quotient's
// neighbourhood that rounds to the border is narrower (half a step, by more than 2^-28 of the border).
// (Infinities and products that overflow must not come here.)

// Eight dims of a block whose scales are d: code words.  (NaN is converted to 6.)
__device__ __forceinline__ uint32_t quantise8(const float* f, float d, float r) {
  float v[8];
  const uint64_t d2 = pair_of(-d, -d), r2 = pair_of(r, r);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const uint64_t x = pair_of(f[k], f[k + 1]), p = mul_pair(x, r2);
    const float2 q = split_pair(fma_pair(fma_pair(p, d2, x), r2, p));
    v[k] = copysignf(q.x, f[k]);             // (-0 has come out as 0)
    v[k + 1] = copysignf(q.y, f[k + 1]);
  }
  return r > 0.0f ? e2m1x8(v) : 0u;
}
// The scale of a block with the largest magnitude m, in the cache's units.  A block of NaN alone has none: its scale
// is e4m3's NaN, so that reads show it, and its codes are 0.
__device__ __forceinline__ uint8_t scale_code(float m) {
  constexpr float kSixth = 1.0f / 6.0f;
  const float t = fminf(m, 4096.0f);         // (past 6 x 448 all are alike)
  const float p = t * kSixth, q = fmaf(fmaf(-6.0f, p, t), kSixth, p);
  return e4m3_of(m == m ? q : m);
}

// The two 8-dim halves of a K or V unit (dims da.. and db..) into the 4-bit cache row `cell`; ma and mb
// are the largest magnitudes of the 16-dim blocks that the halves lie in (ONE: the same block).  f and the
// magnitudes are in units of `unit` = 1 / inv, both exact.
template <typename T, bool ONE>
__device__ __forceinline__ void write_fp4(const RopeParams& p, bool is_v, int64_t row, int32_t kvh, int64_t cell, int da,
                                          int db, float unit, float inv, float ma, float mb, float* f) {
  auto reciprocal = [&](float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return s > 0.0f ? r * inv : 0.0f;
  };
  const uint8_t ca = scale_code(ma * inv), cb = ONE ? ca : scale_code(mb * inv);
  const float sa = e4m3_value(ca), sb = ONE ? sa : e4m3_value(cb);
  const float ra = reciprocal(sa), rb = ONE ? ra : reciprocal(sb);
  // beside the largest scale stand infinities and values far past the largest code: kept at 8 times the scale
  auto limit = [&](float* x, uint8_t code) {
    if (code != 0x7E) return;
    const float most = 8.0f * 448.0f * unit;
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = fminf(fmaxf(x[k], -most), most);      // (NaN becomes -most)
  };
  limit(f, ca);
  limit(f + 8, cb);
  const uint32_t wa = quantise8(f, sa * unit, ra), wb = quantise8(f + 8, sb * unit, rb);
  uint8_t* const codes = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + cell * (p.head_dim / 2);
  uint8_t* const scales = (is_v ? p.v_scale : p.k_scale) + cell * (p.head_dim / 16);
  if constexpr (ONE) {
    *reinterpret_cast<uint2*>(codes + da / 2) = make_uint2(wa, wb);
    scales[da / 16] = ca;
  } else {
    *reinterpret_cast<uint32_t*>(codes + da / 2) = wa;
    *reinterpret_cast<uint32_t*>(codes + db / 2) = wb;
    // one lane writes each block's scale: the one that holds the block's first dim
    if ((da & 15) == 0) scales[da / 16] = ca;
    if ((db & 15) == 0) scales[db / 16] = cb;
  }
  void* const seen = is_v ? p.v_seen : p.k_seen;
  if (seen) {
    const float g = is_v ? p.v_global : p.k_global;
    e2m1x8_values(wa, f);
    e2m1x8_values(wb, f + 8);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f[k] *= sa * g;
      f[k + 8] *= sb * g;
    }
    store_halves<T>(seen, (row * p.n_kvheads + kvh) * p.head_dim, da, db, db == da + 8 && p.wide_seen, f);
  }
}

// Aligned rows: thread = (row, 16-dim unit); blockIdx.y is a share of the heads (q, then k, then v).
// Units 0 .. rot/16 - 1 of a q or k head hold the rotated pairs, the others the dims that pass
// through; V units are plain 16-dim groups.  TURNS false: no pair turns (INTERLEAVED is true then).
template <typename T, bool FP4, bool INTERLEAVED, bool TURNS>
__global__ void __launch_bounds__(kRopeThreads, !TURNS ? (FP4 ? 7 : 8) : FP4 ? 4 : 5) rope_rows_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kBatch = 4;   // heads loaded before the first is stored
  const int units = p.head_dim >> 4, rot_units = TURNS ? p.rot_dim >> 4 : 0;
  const int64_t total = p.n_rows * units;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRopeThreads;
  const bool narrow = total <= INT32_MAX;
  const int h0 = blockIdx.y * p.heads_per_share;
  const int h1 = min(h0 + p.heads_per_share, p.n_qheads + p.n_kvheads + p.n_vheads);
  const int q1 = min(h1, p.n_qheads);
  // whole warps stay in the loop (the 4-bit half layout exchanges maxima between lanes)
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRopeThreads + (threadIdx.x & ~31); t0 < total;
       t0 += stride) {
    const int64_t t = t0 + (threadIdx.x & 31);
    const bool here = t < total;
    const int64_t tc = here ? t : total - 1;
    const int64_t row = narrow ? static_cast<uint32_t>(tc) / static_cast<uint32_t>(units) : tc / units;
    const int u = static_cast<int>(tc - row * units);
    const int32_t pos = p.positions ? __ldg(p.positions + row) : 0;
    const bool live = here && pos >= 0;

    const bool turns = TURNS && u < rot_units;
    int da, db;
    if (turns) {
      da = p.rot_offset + (INTERLEAVED ? 16 * u : 8 * u);
      db = INTERLEAVED ? da + 8 : da + p.rot_dim / 2;
    } else {
      const int d = 16 * (u - rot_units);
      da = !TURNS || d < p.rot_offset ? d : d + p.rot_dim;
      db = da + 8;
    }
    const bool joined = INTERLEAVED || !turns;   // db = da + 8
    float cs[8], sn[8];
    if (turns && live && h0 < p.n_qheads + p.n_kvheads) {
#pragma unroll
      for (int k = 0; k < 8; ++k) angle_of(p, 8 * u + k, pos, cs[k], sn[k]);
    }
    auto rotate = [&](float* f) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int ia = INTERLEAVED ? 2 * k : k, ib = INTERLEAVED ? 2 * k + 1 : k + 8;
        const float a = f[ia], b = f[ib];
        f[ia] = a * cs[k] - b * sn[k];
        f[ib] = b * cs[k] + a * sn[k];
      }
    };
    if (live && (turns || p.q != p.q_out)) {     // (in place, passing dims stay where they are)
      for (int h = h0; h < q1; h += kBatch) {
        const int64_t at = row * p.q_stride + static_cast<int64_t>(h) * p.head_dim;
        const int64_t to = row * p.q_out_stride + static_cast<int64_t>(h) * p.head_dim;
        uint4 ra[kBatch], rb[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (h + k < q1) load_halves<T>(p.q, at + k * p.head_dim, da, db, joined && p.wide_q, ra[k], rb[k]);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          if (h + k < q1) {
            float f[16];
            unpack8<T>(ra[k], f);
            unpack8<T>(rb[k], f + 8);
            if (turns) rotate(f);
            store_halves<T>(p.q_out, to + k * p.head_dim, da, db, joined && p.wide_q, f);
          }
        }
      }
    }
    if (h1 <= p.n_qheads) continue;
    const int32_t slot = __ldg(p.slots + row);
    const bool stored = live && slot >= 0 && slot < p.n_slots;
    // K and V heads, two loaded before the first is worked on
    constexpr int kAhead = 2;
    uint4 raw[kAhead][2];
    for (int h = max(h0, p.n_qheads), n = 0; h < h1; ++h, n ^= 1) {
      if (n == 0 && stored) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (h + k >= h1) continue;
          const bool is_v = h + k >= p.n_qheads + p.n_kvheads;
          const int kvh = h + k - p.n_qheads - (is_v ? p.n_kvheads : 0);
          const int64_t at = row * (is_v ? p.v_stride : p.k_stride) + static_cast<int64_t>(kvh) * p.head_dim;
          load_halves<T>(is_v ? p.v : p.k, at, is_v ? 16 * u : da, is_v ? 16 * u + 8 : db, (joined || is_v) && p.wide_kv,
                         raw[k][0], raw[k][1]);
        }
      }
      const bool is_v = h >= p.n_qheads + p.n_kvheads;
      const int kvh = is_v ? h - p.n_qheads - p.n_kvheads : h - p.n_qheads;
      const int ea = is_v ? 16 * u : da, eb = is_v ? 16 * u + 8 : db;
      const int64_t cell = static_cast<int64_t>(slot) * p.n_kvheads + kvh;
      const bool whole = joined || is_v;
      float f[16];
      if (stored) {
        unpack8<T>(n == 0 ? raw[0][0] : raw[1][0], f);
        unpack8<T>(n == 0 ? raw[0][1] : raw[1][1], f + 8);
        if (turns && !is_v) rotate(f);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) f[k] = 0.0f;
      }
      if constexpr (FP4) {
        float inv = is_v ? p.v_inverse : p.k_inverse, unit = is_v ? p.v_global : p.k_global;
        if (inv == 0.0f) {       // not a power of two: quotients by the cache's scale, rounded to fp32
#pragma unroll
          for (int k = 0; k < 16; ++k) f[k] = __fdiv_rn(f[k], unit);
          inv = unit = 1.0f;
        }
        float ma = amax8(f), mb = amax8(f + 8);
        if constexpr (!INTERLEAVED) {
          // a rotated half shares its block with the neighbouring unit's
          const float na = __shfl_xor_sync(0xffffffffu, ma, 1), nb = __shfl_xor_sync(0xffffffffu, mb, 1);
          const bool split = turns && !is_v;
          const float both = fmaxf(ma, mb);
          ma = split ? fmaxf(ma, na) : both;
          mb = split ? fmaxf(mb, nb) : both;
        } else {
          ma = mb = fmaxf(ma, mb);
        }
        if (stored) write_fp4<T, INTERLEAVED>(p, is_v, row, kvh, cell, ea, eb, unit, inv, ma, mb, f);
      } else if (stored) {
        store_halves<T>(is_v ? p.v_cache : p.k_cache, cell * p.head_dim, ea, eb, whole && p.wide_kv, f);
      }
    }
  }
}

__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_float(float f, __nv_bfloat16& v) { v = __float2bfloat16_rn(f); }
__device__ __forceinline__ void from_float(float f, __half& v) { v = __float2half_rn(f); }

// Rows of any width, offset, stride and alignment: thread = (row, head, pair or passing dim), 2 bytes at a time, the
// angles anew for every head.  Far from memory's rate: 8192 rows of 28 heads of 96 dims, 24 of them turned, take 105 us
// (88 MB); with 32 at an offset of 16 the kernel above takes 20.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_any_kernel(const __grid_constant__ RopeParams p) {
  const int pairs = p.rot_dim >> 1, per_head = p.head_dim - pairs;
  const int heads = p.n_qheads + p.n_kvheads + p.n_vheads;
  const int64_t total = p.n_rows * heads * per_head;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRopeThreads;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x; t < total; t += stride) {
    const int e = static_cast<int>(t % per_head);
    const int64_t rh = t / per_head;
    const int h = static_cast<int>(rh % heads);
    const int64_t row = rh / heads;
    const int32_t pos = p.positions ? __ldg(p.positions + row) : 0;
    if (pos < 0) continue;
    const T* src;
    T* dst;
    const bool is_v = h >= p.n_qheads + p.n_kvheads;
    if (h < p.n_qheads) {
      src = static_cast<const T*>(p.q) + row * p.q_stride + static_cast<int64_t>(h) * p.head_dim;
      dst = static_cast<T*>(p.q_out) + row * p.q_out_stride + static_cast<int64_t>(h) * p.head_dim;
    } else {
      const int32_t slot = __ldg(p.slots + row);
      if (slot < 0 || slot >= p.n_slots) continue;
      const int kvh = is_v ? h - p.n_qheads - p.n_kvheads : h - p.n_qheads;
      src = static_cast<const T*>(is_v ? p.v : p.k) + row * (is_v ? p.v_stride : p.k_stride) +
            static_cast<int64_t>(kvh) * p.head_dim;
      dst = static_cast<T*>(is_v ? p.v_cache : p.k_cache) +
            (static_cast<int64_t>(slot) * p.n_kvheads + kvh) * p.head_dim;
    }
    if (e >= pairs || is_v) {
      // passing dims: everything but the rotated range, or for V all of it (the first `pairs`
      // threads of a V head take two dims)
      if (is_v) {
        dst[e] = src[e];
        if (e < pairs) dst[per_head + e] = src[per_head + e];
      } else {
        const int d = e - pairs, at = d < p.rot_offset ? d : d + p.rot_dim;
        if (src != dst) dst[at] = src[at];
      }
      continue;
    }
    const int ia = p.rot_offset + (p.interleaved ? 2 * e : e), ib = p.interleaved ? ia + 1 : ia + pairs;
    float c, s;
    angle_of(p, e, pos, c, s);
    const float a = to_float(src[ia]), b = to_float(src[ib]);
    from_float(a * c - b * s, dst[ia]);
    from_float(b * c + a * s, dst[ib]);
  }
}

template <typename T, bool FP4>
cudaError_t launch_rows(const RopeParams& p, dim3 grid, cudaStream_t stream) {
  if (p.rot_dim == 0) rope_rows_kernel<T, FP4, true, false><<<grid, kRopeThreads, 0, stream>>>(p);
  else if (p.interleaved) rope_rows_kernel<T, FP4, true, true><<<grid, kRopeThreads, 0, stream>>>(p);
  else rope_rows_kernel<T, FP4, false, true><<<grid, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

// Whether the 16-byte kernel serves the call: every unit starts on a 16-byte boundary.
bool rope_is_aligned(const RopeParams& p) {
  return p.head_dim % 16 == 0 && p.rot_dim % 16 == 0 && p.rot_offset % 16 == 0 && p.q_stride % 8 == 0 &&
         p.q_out_stride % 8 == 0 && p.k_stride % 8 == 0 && p.v_stride % 8 == 0 && aligned(p.q, 16) &&
         aligned(p.q_out, 16) && aligned(p.k, 16) && aligned(p.v, 16) && aligned(p.k_cache, 16) &&
         aligned(p.v_cache, 16) && aligned(p.k_seen, 16) && aligned(p.v_seen, 16);
}

cudaError_t launch_rope(RopeParams p, bool fp16, bool fp4, int num_sms, cudaStream_t stream) {
  const int heads = p.n_qheads + p.n_kvheads + p.n_vheads;
  if (!fp4 && !rope_is_aligned(p)) {
    const int64_t total = p.n_rows * heads * (p.head_dim - p.rot_dim / 2);
    const int64_t want = (total + kRopeThreads - 1) / kRopeThreads, cap = static_cast<int64_t>(num_sms) * 32;
    const unsigned grid = static_cast<unsigned>(want < cap ? want : cap);
    if (fp16) rope_any_kernel<__half><<<grid, kRopeThreads, 0, stream>>>(p);
    else rope_any_kernel<__nv_bfloat16><<<grid, kRopeThreads, 0, stream>>>(p);
    return cudaGetLastError();
  }
  // 32-byte accesses where every unit of a row starts on a 32-byte boundary
  auto wide = [](const void* a, const void* b, int64_t stride_a, int64_t stride_b) {
    return aligned(a, 32) && aligned(b, 32) && stride_a % 16 == 0 && stride_b % 16 == 0;
  };
  p.wide_q = wide(p.q, p.q_out, p.q_stride, p.q_out_stride);
  p.wide_kv = wide(p.k, p.v, p.k_stride, p.v_stride) && (fp4 || wide(p.k_cache, p.v_cache, 0, 0));
  p.wide_seen = wide(p.k_seen, p.v_seen, 0, 0);
  // 1 / g where g is a power of two and g and 1 / g times any block scale or its reciprocal (2^-9 .. 2^9) are normal
  // and finite; else 0, and the rows are divided by g
  auto inverse = [](float g) {
    int e = 0;
    return std::frexp(g, &e) == 0.5f && e > -100 && e < 100 ? 1.0f / g : 0.0f;
  };
  p.k_inverse = inverse(p.k_global);
  p.v_inverse = inverse(p.v_global);
  // Shares of the heads: as few as still give every SM about 1024 threads, since each share computes
  // a row's angles again.
  const int64_t threads = p.n_rows * (p.head_dim / 16);
  int64_t shares = (static_cast<int64_t>(num_sms) * 1024 + threads - 1) / threads;
  if (shares > heads) shares = heads;
  p.heads_per_share = static_cast<int32_t>((heads + shares - 1) / shares);
  shares = (heads + p.heads_per_share - 1) / p.heads_per_share;
  const int64_t blocks = (threads + kRopeThreads - 1) / kRopeThreads;
  const int64_t cap = static_cast<int64_t>(num_sms) * 64;
  const dim3 grid(static_cast<unsigned>(blocks < cap ? blocks : cap), static_cast<unsigned>(shares));
  if (fp4) return fp16 ? launch_rows<__half, true>(p, grid, stream) : launch_rows<__nv_bfloat16, true>(p, grid, stream);
  return fp16 ? launch_rows<__half, false>(p, grid, stream) : launch_rows<__nv_bfloat16, false>(p, grid, stream);
}

}  // namespace qsa
