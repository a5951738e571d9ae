// Window attention kernels of head dim 256 (window.cuh).
#include "window.cuh"

namespace qsa {

cudaError_t launch_window_d256(const WindowParams& p, bool fp16, bool fp4, const CUtensorMap& tk,
                              const CUtensorMap& tv, const CUtensorMap& tq1, const CUtensorMap& tqt, int grid,
                              cudaStream_t stream) {
  return launch_window_dim<256>(p, fp16, fp4, tk, tv, tq1, tqt, grid, stream);
}

}  // namespace qsa
