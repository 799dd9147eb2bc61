// Launches of the tensor-memory attention kernel (pattn_tc_dev.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdlib>

#include "common.cuh"
#include "kernels.h"
#include "pa_dev.cuh"
#include "paged.h"
#include "pattn_tc_dev.cuh"

namespace sv {

bool pattn_tc_supported(const PAttn& a) {
  const int G = a.hq / a.hkv;
  if ((a.hd != 64 && a.hd != 128) || G > kTaRows) return false;
  // tensor maps take positive strides only (a broadcast head has stride 0)
  auto pos = [](int64_t s, int64_t d) { return d == 1 || (s > 0 && s < (1LL << 38)); };
  if (!pos(a.q_ts, a.tokens) || !pos(a.q_hs, a.hq)) return false;
  if (std::abs(a.o_ts) >= 1 << 23 || std::abs(a.o_hs) >= 1 << 23) return false;   // 32-bit offsets within a tile
  if (!a.paged)
    return pos(a.k_ts, a.tokens) && pos(a.k_hs, a.hkv) && pos(a.v_ts, a.tokens) && pos(a.v_hs, a.hkv);
  return pos(a.page_stride, a.pages) && (int64_t)a.hkv << a.page_shift <= 0x7fffffffLL;
}

cudaError_t launch_pattn_tc(const PAttn& a, int num_sms, cudaStream_t st) {
  return launch_ta_items<kPaCausal>(a, num_sms, st);
}

}  // namespace sv
