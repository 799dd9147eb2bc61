// Attention of sequences that share a long prefix, which is read once for all of them.
//
//   out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i
// over the parts i of a row's keys, each with its own exponent reference m, sum l and
// unscaled output O, all fp32.  Three launches:
//   plan    one block works out what each group of sequences really shares (the call's
//           number, cut to what every row of the group sees) and cuts the work: units of
//           128 keys of one (group, KV head, pair of 128-row tiles) in one row;
//   prefix  the tensor-memory kernel (pattn_tc_dev.cuh): every SM takes an equal run of
//           units, whatever the groups' sizes, and leaves a part for each tile that its
//           run touches.  All rows of a group see the whole prefix, so there is no mask;
//   rest    the register-tile kernel (pattn_dev.cuh) over each sequence's own keys; it
//           adds the parts to its rows before it scales them.  It starts while the last
//           prefix blocks still run and waits for them before the join.
// A prefix key is worth its bytes once for all rows and 4 flops per element and row: at
// B sequences of R rows per KV head the bytes fall from B (S + r) to S + B r keys.
#include <cuda_runtime.h>

#include <algorithm>

#include "pattn_tc_dev.cuh"

namespace sv {

namespace {

constexpr int kShThreads = 256;

// One block: groups in turn, their sequences over the threads.
__global__ void __launch_bounds__(kShThreads) shared_plan_kernel(const __grid_constant__ PAttn a, int tpt, int most_runs) {
  __shared__ int s_least;
  pdl_trigger();
  ShPlan* plan = reinterpret_cast<ShPlan*>(a.ws);
  ShGroup* groups = reinterpret_cast<ShGroup*>(plan + 1);
  int unit = 0, tile = 0, seq_end = 0, row_end = 0;
  for (int g = 0; g < a.n_groups; ++g) {
    const int first = a.groups ? __ldg(a.groups + g) : 0, last = a.groups ? __ldg(a.groups + g + 1) : a.seqs;
    if (threadIdx.x == 0) s_least = 0x7fffffff;
    __syncthreads();
    const int least = sh_least(a, first, last);
    if (least < 0x7fffffff) atomicMin(&s_least, least);
    __syncthreads();
    ShRows r = sh_rows(a, first, last);
    // (groups or rows out of order hold nothing: the tiles stay within what the workspace has room for)
    if (first < seq_end || r.row0 < row_end) r = ShRows{0, 0};
    if (r.toks > 0) {
      seq_end = last;
      row_end = r.row0 + r.toks;
    }
    ShGroup o{};
    o.eff = r.toks > 0 ? sh_eff(a, g, s_least) : 0;
    o.row0 = r.row0;
    o.toks = r.toks;
    o.seq0 = first;
    o.pairs = o.eff > 0 ? (r.toks + 2 * tpt - 1) / (2 * tpt) : 0;
    o.steps = (o.eff + kTaKeys - 1) / kTaKeys;
    o.unit0 = unit;
    o.tile0 = tile;
    unit += a.hkv * o.pairs * o.steps;
    tile += a.hkv * o.pairs;
    if (threadIdx.x == 0) groups[g] = o;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    plan->units = unit;
    plan->runs = min(unit, most_runs);
  }
}

// Tiles (KV head, pair) that the groups can hold.
int64_t most_tiles(const PAttn& a) {
  const int tpt = kTaRows / (a.hq / a.hkv);
  return (int64_t)a.hkv * (a.tokens / (2 * tpt) + std::min<int64_t>(a.n_groups, a.tokens));
}

}  // namespace

size_t pattn_shared_workspace(const PAttn& a, int num_sms) {
  if (!a.paged || !pattn_tc_supported(a)) return 0;
  const int64_t keys = (int64_t)a.max_pages << a.page_shift, tiles = most_tiles(a);
  if (tiles * ((keys + kTaKeys - 1) / kTaKeys) > 0x3fffffffLL) return 0;
  return sh_slots_at(a.n_groups) + (size_t)(num_sms + tiles) * 256 * (a.hd + 2) * sizeof(float);
}

cudaError_t launch_pattn_shared(const PAttn& a, int num_sms, cudaStream_t st) {
  TaArgs ta{};
  if (!ta_args(ta, a)) return cudaErrorInvalidValue;
  ta.items = num_sms;
  ta.split = 1;
  cudaError_t e = launch_rows(shared_plan_kernel, dim3(1), dim3(kShThreads), 0, 1, st, a, ta.tpt, num_sms);
  if (e == cudaSuccess) e = launch_ta_mode<kPaPrefix>(ta, st);
  return e == cudaSuccess ? launch_pa_rest(a, num_sms, st) : e;
}

}  // namespace sv
