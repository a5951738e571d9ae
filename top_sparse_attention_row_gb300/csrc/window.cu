// Window attention: tensor maps, kernel choice and the join of split key ranges.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

#include "window.cuh"

namespace qsa {
namespace {

constexpr int kJoinWarps = 4;

// Joins the splits of a row and head: with L_s the split's log-sum-exp and O_s its normalised output,
// lse = ln sum exp(L_s) and O = sum exp(L_s - lse) O_s.  A warp per row and head; the splits are added in
// order, so the result does not depend on which finished first.  Rows behind the last request stay as
// they were.
template <int D, typename T>
__global__ void __launch_bounds__(kJoinWarps * 32) window_join_kernel(const __grid_constant__ WindowParams p) {
  constexpr int kPer = D / 32;
  pdl_wait();   // first thing in every thread: the grid must not end before the attention kernel has
  const int lane = threadIdx.x & 31;
  const int64_t rh = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
  if (rh >= p.n_rows * p.n_qheads) return;
  const int64_t row = rh / p.n_qheads;
  if (row < __ldg(p.pa.cu_seqlens_q) || row >= __ldg(p.pa.cu_seqlens_q + p.pa.n_requests)) return;
  const float* const ls = p.part_lse + rh * p.splits;
  const float* const os = p.part_o + rh * p.splits * D + lane * kPer;
  // lane s holds the weight of split s (up to 128 splits: four per lane)
  float w[4], m = -INFINITY;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    w[g] = g * 32 + lane < p.splits ? ls[g * 32 + lane] : -INFINITY;
    m = fmaxf(m, w[g]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float acc[kPer], total = 0.0f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.0f;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    w[g] = w[g] == -INFINITY ? 0.0f : __expf(w[g] - m);
    total += w[g];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int n = min(p.splits - g * 32, 32);
#pragma unroll 8
    for (int s = 0; s < n; ++s) {
      const float ws = __shfl_sync(0xffffffffu, w[g], s);
      float x[kPer];
#pragma unroll
      for (int k = 0; k < kPer; k += 2) {
        const float2 t = *reinterpret_cast<const float2*>(os + static_cast<int64_t>(g * 32 + s) * D + k);
        x[k] = t.x;
        x[k + 1] = t.y;
      }
      // a split that saw nothing wrote no output: whatever is there stays out
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] += ws == 0.0f ? 0.0f : ws * x[k];
    }
  }
  const float inv = m == -INFINITY ? 0.0f : 1.0f / total;
  T* const out = static_cast<T*>(p.out) + rh * D + lane * kPer;
#pragma unroll
  for (int k = 0; k < kPer; k += 2)
    *reinterpret_cast<uint32_t*>(out + k) = window_detail::pack16(acc[k] * inv, acc[k + 1] * inv, T{});
  if (lane == 0 && p.lse) p.lse[rh] = m == -INFINITY ? -INFINITY : m + logf(total);
}

template <int D, typename T>
cudaError_t launch_join_dim(const WindowParams& p, cudaStream_t stream) {
  // launched while the attention kernel runs (programmatic dependent launch): it waits for that grid's end
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  const int64_t rows = p.n_rows * p.n_qheads;
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(kJoinWarps * 32);
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

cudaError_t launch_window(const WindowParams& p, int head_dim, bool fp16, bool fp4, const void* k_cache,
                          const void* v_cache, cudaStream_t stream) {
  // (the element type only decides how many bits are moved: 16 either way)
  const CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap tk{}, tv{}, tq1{}, tqt{};
  if (!fp4) {
    const cuuint64_t d = static_cast<cuuint64_t>(head_dim);
    const cuuint64_t q_dims[3] = {d, static_cast<cuuint64_t>(p.n_qheads), static_cast<cuuint64_t>(p.n_rows)};
    const cuuint64_t q_strides[2] = {d * 2, d * 2 * static_cast<cuuint64_t>(p.n_qheads)};
    const cuuint32_t q_box1[3] = {64, static_cast<cuuint32_t>(p.group), 1};
    const cuuint32_t q_boxt[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(p.tile_tokens)};
    CUresult r = encode_tensor_map(&tq1, type, 3, p.q, q_dims, q_strides, q_box1);
    if (r == CUDA_SUCCESS) r = encode_tensor_map(&tqt, type, 3, p.q, q_dims, q_strides, q_boxt);
    const cuuint64_t slots = static_cast<cuuint64_t>(p.n_slots), heads = static_cast<cuuint64_t>(p.n_kvheads);
    for (int i = 0; i < 2 && r == CUDA_SUCCESS; ++i) {
      CUtensorMap* const m = i == 0 ? &tk : &tv;
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
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  }
  const int grid = static_cast<int>(p.n_units);
  const cudaError_t e = head_dim == 64    ? launch_window_d64(p, fp16, fp4, tk, tv, tq1, tqt, grid, stream)
                        : head_dim == 128 ? launch_window_d128(p, fp16, fp4, tk, tv, tq1, tqt, grid, stream)
                                          : launch_window_d256(p, fp16, fp4, tk, tv, tq1, tqt, grid, stream);
  if (e != cudaSuccess || p.splits <= 1) return e;
  return fp16 ? launch_join<__half>(p, head_dim, stream) : launch_join<__nv_bfloat16>(p, head_dim, stream);
}

}  // namespace qsa
