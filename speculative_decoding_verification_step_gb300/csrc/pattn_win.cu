// Register-tile attention with a sliding window and first tokens that stay visible.
#include "pattn_dev.cuh"

namespace sv {

cudaError_t launch_pa_window(const PAttn& a, int num_sms, cudaStream_t st) {
  return a.hd == 32   ? launch_pa_hd<32, kPaWindow>(a, num_sms, st)
         : a.hd == 64 ? launch_pa_hd<64, kPaWindow>(a, num_sms, st)
                      : launch_pa_hd<128, kPaWindow>(a, num_sms, st);
}

}  // namespace sv
