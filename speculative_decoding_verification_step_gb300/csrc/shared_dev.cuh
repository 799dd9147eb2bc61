// Shared prefixes: what a group of sequences shares, as the kernels work it out.
#pragma once
#include "common.cuh"
#include "paged.h"

namespace sv {

namespace {

// The rows of sequences first .. last - 1, none unless they lie in the call's.
struct ShRows {
  int row0, toks;
};
SV_DEV ShRows sh_rows(const PAttn& a, int first, int last) {
  if (first < 0 || last > a.seqs || first >= last) return ShRows{0, 0};
  const int r0 = __ldg(a.cu + first), r1 = __ldg(a.cu + last);
  if (r0 < 0 || r1 <= r0 || r1 > a.tokens) return ShRows{0, 0};
  return ShRows{r0, r1 - r0};
}
// What the sequences first .. last - 1 share: as many positions as the call says, cut to what all
// of their rows see (sequences without rows do not count).  Whole warps.  all, count, reader: the
// positions of those sequences, their number, and the first of them, by whose row of the table the
// prefix is read (the entries of a sequence without rows may be gone).
SV_DEV int sh_eff(const PAttn& a, int group, int first, int last, float* all, int* count, int* reader) {
  const int lane = threadIdx.x & 31, said = __ldg(a.shared + group);
  const int cap = (int)min((int64_t)0x7fffffff, (int64_t)a.max_pages << a.page_shift);
  int least = 0x7fffffff, seqs = 0, own = 0x7fffffff;
  float keys_all = 0.f;
  for (int s = max(first, 0) + lane; s < min(last, a.seqs); s += 32) {
    const int r = __ldg(a.cu + s), n = __ldg(a.cu + s + 1) - r, keys = min(max(__ldg(a.lens + s), 0), cap);
    if (r >= 0 && n > 0 && n <= a.tokens - r) {
      least = min(least, max(0, keys - n));
      keys_all += (float)keys;
      own = min(own, s);
      ++seqs;
    }
  }
  *all = warp_sum(keys_all);
  *count = __reduce_add_sync(0xffffffffu, seqs);
  *reader = __reduce_min_sync(0xffffffffu, own);
  least = __reduce_min_sync(0xffffffffu, least);
  return least == 0x7fffffff ? 0 : max(0, min(said, least));
}
}  // namespace

}  // namespace sv
