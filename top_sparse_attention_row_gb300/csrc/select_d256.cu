// Page selection of head dim 256 (select.cuh).
#include "select.cuh"

namespace qsa {

cudaError_t launch_select_d256(const ChooseParams& p, bool fp16, int num_sms, cudaStream_t stream) {
  return launch_select_dim<256>(p, fp16, num_sms, stream);
}

}  // namespace qsa
