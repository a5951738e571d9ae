// Attention of each row over the positions of its listed pages.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "paged.cuh"

namespace qsa {
namespace {

constexpr int kSelThreads = 256;

// A warp takes a row's head: one key after the other, the dims over the lanes, the running maximum and sum of the
// softmax in fp32.  A page that is listed twice counts once.
template <int D, typename T>
__global__ void __launch_bounds__(kSelThreads) selected_attention_kernel(const __grid_constant__ SelectedParams p) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t rh = static_cast<int64_t>(blockIdx.x) * (kSelThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = rh / p.n_qheads;
  if (row >= p.n_rows || row >= __ldg(p.pa.cu_seqlens_q + p.pa.n_requests)) return;
  const int32_t kvh = static_cast<int32_t>(rh - row * p.n_qheads) / p.group;
  const int32_t req = paged_request_of_row(p.pa, row, lane);
  const int64_t pos = static_cast<int64_t>(__ldg(p.pa.kv_lens + req)) - __ldg(p.pa.cu_seqlens_q + req + 1) + row;
  const int32_t* const list = p.pages + (row * p.n_kvheads + kvh) * p.n_select;
  float q[kPer], o[kPer], m = -INFINITY, l = 0.0f;
  for (int c = 0; c < kPer; ++c) {
    q[c] = static_cast<float>(static_cast<const T*>(p.q)[rh * D + lane * kPer + c]) * p.scale_log2;
    o[c] = 0.0f;
  }
  for (int32_t i = 0; i < p.n_select; ++i) {
    const int32_t e = __ldg(list + i);
    if (e < 0 || e >= p.pa.pages_per_req) continue;
    bool before = false;
    for (int32_t k = lane; k < i; k += 32) before |= __ldg(list + k) == e;
    if (__any_sync(0xffffffffu, before)) continue;
    const int32_t page = __ldg(p.pa.page_table + static_cast<int64_t>(req) * p.pa.pages_per_req + e);
    if (page < 0 || page >= p.pa.n_pages) continue;
    const int64_t start = static_cast<int64_t>(e) * p.pa.page_size;
    const int64_t seen = pos + 1 - start < p.pa.page_size ? pos + 1 - start : p.pa.page_size;
    for (int32_t j = 0; j < seen; ++j) {
      const int64_t at = ((static_cast<int64_t>(page) * p.pa.page_size + j) * p.n_kvheads + kvh) * D + lane * kPer;
      float s = 0.0f;
      for (int c = 0; c < kPer; ++c) s += q[c] * static_cast<float>(static_cast<const T*>(p.k_cache)[at + c]);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      if (s == -INFINITY) continue;
      const float nm = s > m ? s : m, f = exp2f(m - nm), w = exp2f(s - nm);
      m = nm;
      l = l * f + w;
      for (int c = 0; c < kPer; ++c) o[c] = o[c] * f + w * static_cast<float>(static_cast<const T*>(p.v_cache)[at + c]);
    }
  }
  const bool empty = l == 0.0f && m == -INFINITY;
  for (int c = 0; c < kPer; ++c) static_cast<T*>(p.out)[rh * D + lane * kPer + c] = static_cast<T>(empty ? 0.0f : o[c] / l);
  if (p.lse && lane == 0) p.lse[rh] = empty ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

}  // namespace

cudaError_t launch_selected(const SelectedParams& p, int head_dim, bool fp16, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((p.n_rows * p.n_qheads + kSelThreads / 32 - 1) / (kSelThreads / 32));
  auto go = [&](auto kern) {
    kern<<<grid, kSelThreads, 0, stream>>>(p);
    return cudaGetLastError();
  };
  if (fp16)
    return head_dim == 64    ? go(selected_attention_kernel<64, __half>)
           : head_dim == 128 ? go(selected_attention_kernel<128, __half>)
                             : go(selected_attention_kernel<256, __half>);
  return head_dim == 64    ? go(selected_attention_kernel<64, __nv_bfloat16>)
         : head_dim == 128 ? go(selected_attention_kernel<128, __nv_bfloat16>)
                           : go(selected_attention_kernel<256, __nv_bfloat16>);
}

}  // namespace qsa
