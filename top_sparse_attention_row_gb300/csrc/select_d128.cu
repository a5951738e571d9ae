// Page selection of head dim 128 (select.cuh).
#include "select.cuh"

namespace qsa {

cudaError_t launch_select_d128(const ChooseParams& p, bool fp16, int num_sms, cudaStream_t stream) {
  return launch_select_dim<128>(p, fp16, num_sms, stream);
}

}  // namespace qsa
