// Tensor-memory attention with a sliding window and first tokens that stay visible.
#include "pattn_tc_dev.cuh"

namespace sv {

cudaError_t launch_pattn_tc_window(const PAttn& a, int num_sms, cudaStream_t st) {
  return launch_ta_items<kPaWindow>(a, num_sms, st);
}

}  // namespace sv
