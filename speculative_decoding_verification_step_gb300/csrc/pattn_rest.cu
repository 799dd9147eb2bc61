// Register-tile attention of what sequences have behind a shared prefix, joined with the
// prefix's parts.
#include "pattn_dev.cuh"

namespace sv {

cudaError_t launch_pa_rest(const PAttn& a, int num_sms, cudaStream_t st) {
  return a.hd == 64 ? launch_pa_hd<64, kPaRest>(a, num_sms, st) : launch_pa_hd<128, kPaRest>(a, num_sms, st);
}

}  // namespace sv
