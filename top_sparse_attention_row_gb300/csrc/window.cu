// Attention over paged caches: tensor maps, kernel choice and the join of units that several blocks share.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

#include "window.cuh"

namespace qsa {
namespace {

constexpr int kJoinThreads = 512;
constexpr int kJoinRows = 16;      // blocks that share a unit's rows
constexpr int kJoinWarpParts = 8;  // parts up to which a warp takes a row

// Joins the parts of a unit (equal shares): with L_s a part's log-sum-exp and O_s its normalised output,
// lse = ln sum exp(L_s) and O = sum exp(L_s - lse) O_s.  The blocks (c, y) take the rows of the unit that
// begins in block c of the attention grid and goes on in the following ones.  Two parts are the rule for
// units of many rows, and then a warp takes a row; a long unit of few rows has a part in every block, and
// then a block takes a row, D / 4 threads across it and the groups of threads each some of the parts.
// Parts are added in a fixed order, so the result does not depend on timing.  A part that is NaN makes the row NaN,
// its lse too (the maximum passes over NaN, the sum of the weights does not).
template <int D, typename T>
__global__ void __launch_bounds__(kJoinThreads) window_join_kernel(const __grid_constant__ WindowParams p) {
  constexpr int kCols = D / 4, kGroups = kJoinThreads / kCols;
  __shared__ float4 sums[kGroups][kCols];
  pdl_wait();   // first thing in every thread: the grid must not end before the attention kernel has
  const JoinRecord j = p.joins[blockIdx.x];
  if (j.first < 0) return;
  const int tid = threadIdx.x, lane = tid & 31, col = tid % kCols, group = tid / kCols;
  const int parts = j.more + 1;
  auto slot = [&](int s) { return s == 0 ? j.first : 2 * (static_cast<int>(blockIdx.x) + s); };
  if (parts <= kJoinWarpParts) {
    constexpr int kPer = D / 32;
    const int row = blockIdx.y * (kJoinThreads / 32) + (tid >> 5);   // 16 x 16 rows are more than a unit has
    if (row >= j.tokens * p.group) return;
    const float l = lane < parts ? p.part_lse[slot(lane) * kWinTile + row] : -INFINITY;
    float m = l;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float w = l == -INFINITY ? 0.0f : __expf(l - m);
    float total = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const float inv = m == -INFINITY ? 0.0f : 1.0f / total;
    // a part that saw nothing of this row wrote no output: whatever is there stays out
    const uint32_t saw = __ballot_sync(0xffffffffu, l != -INFINITY);
    float acc[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] = 0.0f;
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
      const float ws = __shfl_sync(0xffffffffu, w, s) * inv;
      const float* const src = p.part_o + static_cast<int64_t>(slot(s) * kWinTile + row) * D + lane * kPer;
#pragma unroll
      for (int k = 0; k < kPer; k += 2) {
        const float2 x = *reinterpret_cast<const float2*>(src + k);
        if (saw >> s & 1) {
          acc[k] += ws * x.x;
          acc[k + 1] += ws * x.y;
        }
      }
    }
    const int tok = row / p.group;
    const int64_t rh = (static_cast<int64_t>(j.row0) + tok) * p.n_qheads + j.kvh * p.group + (row - tok * p.group);
    uint32_t* const out = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + rh * D + lane * kPer);
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k) out[k] = window_detail::pack16(acc[2 * k], acc[2 * k + 1], T{});
    if (lane == 0 && p.lse) p.lse[rh] = total == 0.0f ? -INFINITY : m + logf(total);
    return;
  }
  for (int row = blockIdx.y; row < j.tokens * p.group; row += kJoinRows) {
    // the first parts' rows are on their way while every warp works out the parts' total weight
    constexpr int kFirst = 4, kLaneParts = 5;              // (a unit has at most 152 parts, 160 fit)
    float4 x[kFirst];
    float lx[kFirst], l[kLaneParts];
#pragma unroll
    for (int i = 0; i < kFirst; ++i) {
      const int s = group + i * kGroups;
      lx[i] = -INFINITY;
      if (s < parts) {
        const int64_t at = slot(s) * kWinTile + row;
        lx[i] = p.part_lse[at];
        x[i] = *reinterpret_cast<const float4*>(p.part_o + at * D + col * 4);
      }
    }
    float m = -INFINITY, total = 0.0f;
#pragma unroll
    for (int i = 0; i < kLaneParts; ++i) {
      const int s = lane + 32 * i;
      l[i] = s < parts ? p.part_lse[slot(s) * kWinTile + row] : -INFINITY;
      m = fmaxf(m, l[i]);
    }
    for (int s = lane + 32 * kLaneParts; s < parts; s += 32) m = fmaxf(m, p.part_lse[slot(s) * kWinTile + row]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
    for (int i = 0; i < kLaneParts; ++i) total += l[i] == -INFINITY ? 0.0f : __expf(l[i] - m);
    for (int s = lane + 32 * kLaneParts; s < parts; s += 32) {
      const float v = p.part_lse[slot(s) * kWinTile + row];
      total += v == -INFINITY ? 0.0f : __expf(v - m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const float inv = m == -INFINITY ? 0.0f : 1.0f / total;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](float v, const float4& o) {
      if (v == -INFINITY) return;      // (saw nothing, as above)
      const float w = __expf(v - m) * inv;
      acc.x += w * o.x;
      acc.y += w * o.y;
      acc.z += w * o.z;
      acc.w += w * o.w;
    };
#pragma unroll
    for (int i = 0; i < kFirst; ++i) add(lx[i], x[i]);
#pragma unroll 4
    for (int s = group + kFirst * kGroups; s < parts; s += kGroups) {
      const int64_t at = slot(s) * kWinTile + row;
      add(p.part_lse[at], *reinterpret_cast<const float4*>(p.part_o + at * D + col * 4));
    }
    sums[group][col] = acc;
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int g = 1; g < kGroups; ++g) {
        const float4 x = sums[g][col];
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
      }
      const int tok = row / p.group;
      const int64_t rh = (static_cast<int64_t>(j.row0) + tok) * p.n_qheads + j.kvh * p.group + (row - tok * p.group);
      *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + rh * D + col * 4) =
          make_uint2(window_detail::pack16(acc.x, acc.y, T{}), window_detail::pack16(acc.z, acc.w, T{}));
      if (col == 0 && p.lse) p.lse[rh] = total == 0.0f ? -INFINITY : m + logf(total);
    }
    __syncthreads();
  }
}

template <int D, typename T>
cudaError_t launch_join_dim(const WindowParams& p, cudaStream_t stream) {
  // launched while the attention kernel runs (programmatic dependent launch): it waits for that grid's end
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.shares), kJoinRows);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, window_join_kernel<D, T>, p);
}
template <typename T>
cudaError_t launch_join(const WindowParams& p, int head_dim, cudaStream_t stream) {
  return head_dim == 64    ? launch_join_dim<64, T>(p, stream)
         : head_dim == 128 ? launch_join_dim<128, T>(p, stream)
                           : launch_join_dim<256, T>(p, stream);
}

}  // namespace

CUresult encode_tensor_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base,
                           const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  if (!fn) return CUDA_ERROR_NOT_SUPPORTED;
  const cuuint32_t ones[3] = {1, 1, 1};
  return fn(m, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

namespace {
// Tensor maps of the query rows (one token's heads, a tile's) and of the caches.
CUresult encode_maps(const WindowParams& p, int head_dim, const void* k_cache, const void* v_cache, CUtensorMap* tk,
                     CUtensorMap* tv, CUtensorMap* tq1, CUtensorMap* tqt) {
  // (the element type only decides how many bits are moved: 16 either way)
  const CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t d = static_cast<cuuint64_t>(head_dim);
  const cuuint64_t q_dims[3] = {d, static_cast<cuuint64_t>(p.n_qheads), static_cast<cuuint64_t>(p.n_rows)};
  const cuuint64_t q_strides[2] = {d * 2, d * 2 * static_cast<cuuint64_t>(p.n_qheads)};
  const cuuint32_t q_box1[3] = {64, static_cast<cuuint32_t>(p.group), 1};
  const cuuint32_t q_boxt[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(p.tile_tokens)};
  CUresult r = encode_tensor_map(tq1, type, 3, p.q, q_dims, q_strides, q_box1);
  if (r == CUDA_SUCCESS) r = encode_tensor_map(tqt, type, 3, p.q, q_dims, q_strides, q_boxt);
  const cuuint64_t slots = static_cast<cuuint64_t>(p.n_slots), heads = static_cast<cuuint64_t>(p.n_kvheads);
  for (int i = 0; i < 2 && r == CUDA_SUCCESS; ++i) {
    CUtensorMap* const m = i == 0 ? tk : tv;
    const void* const cache = i == 0 ? k_cache : v_cache;
    if (p.box > 0) {      // boxes of `box` slots of one KV head
      const cuuint64_t dims[3] = {d, heads, slots};
      const cuuint64_t strides[2] = {d * 2, d * 2 * heads};
      const cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(p.box)};
      r = encode_tensor_map(m, type, 3, cache, dims, strides, box);
    } else {              // gathers of four rows (slot x heads + head)
      const cuuint64_t dims[2] = {d, slots * heads};
      const cuuint64_t strides[1] = {d * 2};
      const cuuint32_t box[2] = {64, 1};
      r = encode_tensor_map(m, type, 2, cache, dims, strides, box);
    }
  }
  return r;
}
}  // namespace

cudaError_t launch_window(const WindowParams& p, int head_dim, bool fp16, bool fp4, const void* k_cache,
                          const void* v_cache, cudaStream_t stream) {
  CUtensorMap tk{}, tv{}, tq1{}, tqt{};
  if (!fp4 && encode_maps(p, head_dim, k_cache, v_cache, &tk, &tv, &tq1, &tqt) != CUDA_SUCCESS) return cudaErrorInvalidValue;
  const int grid = p.shares > 0 ? p.shares : static_cast<int>(p.n_units);
  const cudaError_t e = head_dim == 64    ? launch_window_d64(p, fp16, fp4, tk, tv, tq1, tqt, grid, stream)
                        : head_dim == 128 ? launch_window_d128(p, fp16, fp4, tk, tv, tq1, tqt, grid, stream)
                                          : launch_window_d256(p, fp16, fp4, tk, tv, tq1, tqt, grid, stream);
  if (e != cudaSuccess || p.shares == 0) return e;
  return fp16 ? launch_join<__half>(p, head_dim, stream) : launch_join<__nv_bfloat16>(p, head_dim, stream);
}

cudaError_t launch_listed(const WindowParams& p, const ListParams& l, UnitSource source, int head_dim, bool fp16,
                          const void* k_cache, const void* v_cache, cudaStream_t stream) {
  CUtensorMap tk{}, tv{}, tq1{}, tqt{};
  if (encode_maps(p, head_dim, k_cache, v_cache, &tk, &tv, &tq1, &tqt) != CUDA_SUCCESS) return cudaErrorInvalidValue;
  const bool prefix = source == kSharedPrefix;
  cudaError_t e = prefix ? launch_list_prefix(l, stream) : launch_list_pages(l, stream);
  if (e != cudaSuccess) return e;
  const int grid = p.shares > 0 ? p.shares : p.n_tiles;
  e = head_dim == 64    ? launch_listed_d64(p, fp16, prefix, tk, tv, tq1, tqt, grid, stream)
      : head_dim == 128 ? launch_listed_d128(p, fp16, prefix, tk, tv, tq1, tqt, grid, stream)
                        : launch_listed_d256(p, fp16, prefix, tk, tv, tq1, tqt, grid, stream);
  if (e != cudaSuccess || p.shares == 0) return e;
  if (prefix) return launch_join_prefix(p, l, head_dim, fp16, stream);
  return fp16 ? launch_join<__half>(p, head_dim, stream) : launch_join<__nv_bfloat16>(p, head_dim, stream);
}

}  // namespace qsa
