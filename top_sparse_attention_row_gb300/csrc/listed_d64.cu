// Attention kernels over listed units (chosen pages, shared prompts) of head dim 64 (window.cuh).
#include "window.cuh"

namespace qsa {

cudaError_t launch_listed_d64(const WindowParams& p, bool fp16, bool prefix, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tq1, const CUtensorMap& tqt, int grid, cudaStream_t stream) {
  return launch_listed_dim<64>(p, fp16, prefix, tk, tv, tq1, tqt, grid, stream);
}

}  // namespace qsa
