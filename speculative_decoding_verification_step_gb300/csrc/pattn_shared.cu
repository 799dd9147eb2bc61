// Attention of sequences that share a long prefix, which is read once for all of them.
//
//   out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i
// over the parts i of a row's keys, each with its own exponent reference m, sum l and
// unscaled output O, all fp32.  Four launches, each begun before the one in front ends:
//   plan    one block works out what each group of sequences really shares (the call's
//           number, cut to what every row of the group sees), the work's order (units of
//           128 keys of one (group, KV head, pair of 128-row tiles) in one row) and how
//           many SMs take part in the prefix;
//   prefix  the tensor-memory kernel (pattn_tc_dev.cuh): each of those SMs takes an equal
//           run of units, whatever the groups' sizes, and leaves a part for each tile that
//           its run touches.  All rows of a group see the whole prefix: there is no mask;
//   rest    the register-tile kernel (pattn_dev.cuh) over each sequence's own keys, on the
//           other SMs beside it: neither fills HBM alone, and a prefix block leaves no
//           room for another on its SM;
//   join    a row to a half or whole warp: its parts' references and sums one a lane,
//           then their O.
// A prefix key is worth its bytes once for all rows and 4 flops per element and row: at
// B sequences of R rows per KV head the bytes fall from B (S + r) to S + B r keys.
// Measured (8 KV heads of 128, one group): 64 x 1 tokens behind 16384, up to 512 of their own
// 47 us (one by one 339), behind 65536 85 us (62% of the bytes' floor); 64 x 6 behind 16384
// 108 us (51%); 64 x 6 behind four prompts of up to 8192, e4m3, 82 us (one by one 172).  What is fixed is
// some 25 us: the plan 3, the first part's page ids, Q and keys 6, a part's rows out 2, the
// join 6 and the handovers between.  Beyond that 16-bit prefixes go by HBM (from 32768 to
// 65536 keys 6.2 TB/s), 8-bit ones by the conversion of K and V (2 us a unit of 256
// rows, a unit's products 1.3).  L2 prefetches ahead of the ring delayed the first keys and
// gained nothing; sums written by eight dims of a row for coalescing made the join slower.
#include <cuda_runtime.h>

#include <algorithm>

#include "pattn_tc_dev.cuh"
#include "shared_dev.cuh"

namespace sv {

namespace {

constexpr int kShThreads = 256;

// Weights by which the SMs are divided between prefix and rest, about ns on one SM: a unit of the
// prefix; a key of the rest for one KV head of one sequence, and a block's start in keys.  They are
// estimates, not measurements (the results are right whatever they are).  Measured on all SMs, from
// 16384 to 65536 prefix positions, a unit is 1.7 us for bf16 and 2.0 for e4m3 at head dim 128, 1.2
// and 1.9 to 2.0 at 64; a key of the register tiles alone, from 256 to 768 positions, is 10.5 to
// 11.6 ns and 6.6 to 9.8 at 128, 5.4 to 6.5 and 3.9 to 6.0 at 64 (1 to 6 tokens of 4 rows).
struct ShCost {
  float unit, key, block;
};
ShCost sh_cost(const PAttn& a) {
  const int64_t rows = (int64_t)std::min(a.max_q, a.tokens) * (a.hq / a.hkv), tiles = (rows + 31) / 32;
  ShCost c;
  c.unit = (a.f8 ? 2600.f : 1450.f) * (a.hd == 64 ? 0.75f : 1.f);
  c.key = (rows <= 8 ? 2.f : rows <= 16 ? 3.f : 5.f) * (float)tiles * (a.hd == 64 && !a.f8 ? 0.6f : 1.f);
  c.block = 600.f;
  return c;
}

// One block: what every group shares, a warp a group, and the order of the work.
__global__ void __launch_bounds__(kShThreads) shared_plan_kernel(const __grid_constant__ PAttn a, ShCost cost) {
  constexpr int kWarps = kShThreads / 32;
  __shared__ ShGroup s_group[kWarps];
  __shared__ int s_first[kWarps];
  __shared__ float s_rest[kWarps];             // keys behind the prefixes, and as many as a block's start costs
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tpt = kTaRows / (a.hq / a.hkv);
  ShPlan* plan = reinterpret_cast<ShPlan*>(a.ws);
  ShGroup* groups = sh_groups(a.ws);
  int unit = 0, tile = 0, seq_end = 0, row_end = 0;
  float rest = 0.f;
  // the thread's first sequence, on its way
  int r0 = (int)threadIdx.x < a.seqs ? __ldg(a.cu + threadIdx.x) : 0, r1 = (int)threadIdx.x < a.seqs ? __ldg(a.cu + threadIdx.x + 1) : 0;
  for (int g0 = 0; g0 < a.n_groups; g0 += kWarps) {
    const int g = g0 + warp;
    if (g < a.n_groups) {
      const int first = a.groups ? __ldg(a.groups + g) : 0, last = a.groups ? __ldg(a.groups + g + 1) : a.seqs;
      const ShRows r = sh_rows(a, first, last);
      ShGroup o{};
      float keys;
      int seqs;
      o.eff = sh_eff(a, g, first, last, &keys, &seqs, &o.seq0);
      if (r.toks == 0) o.eff = 0;
      o.row0 = r.row0;
      o.toks = r.toks;
      o.pairs = (r.toks + 2 * tpt - 1) / (2 * tpt);
      o.steps = (o.eff + kTaKeys - 1) / kTaKeys;
      if (lane == 0) {
        s_group[warp] = o;
        s_first[warp] = first;
        s_rest[warp] = keys + (float)seqs * (cost.block - (float)o.eff);
      }
    }
    __syncthreads();
    if (threadIdx.x == 0)
      for (int w = 0; w < kWarps && g0 + w < a.n_groups; ++w) {
        ShGroup o = s_group[w];
        // (groups or rows out of order hold nothing: the tiles stay within what the workspace has room for)
        if (s_first[w] < seq_end || o.row0 < row_end) o.eff = o.toks = 0;
        if (o.eff == 0) o.pairs = o.steps = 0;
        if (o.toks > 0) {
          seq_end = a.groups ? __ldg(a.groups + g0 + w + 1) : a.seqs;
          row_end = o.row0 + o.toks;
        }
        o.unit0 = unit;
        o.tile0 = tile;
        unit += a.hkv * o.pairs * o.steps;
        tile += a.hkv * o.pairs;
        rest += s_rest[w];
        groups[g0 + w] = s_group[w] = o;
      }
    __syncthreads();
  }
  // every sequence's group: the last that begins at or before it, if it has not ended there
  for (int s = threadIdx.x; s < a.seqs; s += kShThreads) {
    int g = 0, end = a.groups ? a.n_groups : 1;
    while (end - g > 1) {
      const int mid = (g + end) >> 1;
      if (__ldg(a.groups + mid) <= s) g = mid;
      else end = mid;
    }
    ShSeq o{};
    const ShGroup gr = a.n_groups <= kWarps ? s_group[g] : groups[g];
    if (s >= kShThreads) {
      r0 = __ldg(a.cu + s);
      r1 = __ldg(a.cu + s + 1);
    }
    if ((!a.groups || (__ldg(a.groups + g) <= s && s < __ldg(a.groups + g + 1))) && r0 >= gr.row0 && r1 <= gr.row0 + gr.toks)
      o = ShSeq{gr.eff, gr.row0, gr.unit0, gr.tile0, gr.pairs, gr.steps, {0, 0}};   // (else there is no order in cu)
    sh_seqs(a.ws, a.n_groups)[s] = o;
  }
  if (threadIdx.x == 0) {
    // SMs for the prefix by its share of the time; the rest's blocks take the others
    const float p = (float)unit * cost.unit, q = rest * (float)a.hkv * cost.key;
    plan->units = unit;
    plan->runs = min(unit, max(1, min(a.runs, (int)((float)a.runs * p / (p + q) + 0.5f))));
  }
}

// Adds the prefix's parts to row `tok`, head `h` of KV head kvh, dims col .. col + 3, whose HD / 4
// adjacent lanes work together: first the parts' references and sums, one a lane, then their O.
template <int HD>
SV_DEV void sh_join(const PAttn& a, const ShSeq& p, int units, int runs, int kvh, int tok, int h, int col, float4& x, float& mm,
                    float& ll) {
  if (p.eff == 0) return;
  constexpr int kLanes = HD / 4;
  const int G = a.hq / a.hkv, tpt = 128 / G, t = tok - p.row0, pair = t / (2 * tpt), in = t - pair * 2 * tpt;
  const int half = in / tpt, r = (in - half * tpt) * G + h, tile = kvh * p.pairs + pair, u0 = p.unit0 + tile * p.steps;
  const int r0 = sh_run(u0, units, runs), n = sh_run(u0 + p.steps - 1, units, runs) - r0 + 1;
  const int lane = col / 4;
  const unsigned mask = kLanes == 32 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16);
  const float* first = sh_slot(a.ws, a.n_groups, a.seqs, HD, r0 + p.tile0 + tile);
  const size_t next = (size_t)256 * (HD + 2);
  const float* at = first + (half * 128 + r) * HD + col;
  for (int i0 = 0; i0 < n; i0 += kLanes) {
    const int np = min(kLanes, n - i0);
    float2 ml = make_float2(kTaNone, 0.f);
    if (lane < np) ml = __ldcg(reinterpret_cast<const float2*>(first + (i0 + lane) * next + 256 * HD) + half * 128 + r);
    float to = ml.x;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) to = fmaxf(to, __shfl_xor_sync(mask, to, o, kLanes));
    to = fmaxf(to, mm);
    const float f = ta_exp2(ml.x - to), keep = ta_exp2(mm - to);
    float l = ml.y * f;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) l += __shfl_xor_sync(mask, l, o, kLanes);
    ll = ll * keep + l;
    mm = to;
    x.x *= keep; x.y *= keep; x.z *= keep; x.w *= keep;
#pragma unroll 16
    for (int i = 0; i < np; ++i) {
      const float fi = __shfl_sync(mask, f, i, kLanes);
      const float4 y = __ldcg(reinterpret_cast<const float4*>(at + (i0 + i) * next));
      x.x = fmaf(y.x, fi, x.x); x.y = fmaf(y.y, fi, x.y); x.z = fmaf(y.z, fi, x.z); x.w = fmaf(y.w, fi, x.w);
    }
  }
}

// Rows of a sequence in blocks of kShThreads / (HD / 4): what lies behind the prefix, then the
// prefix's parts.
template <int HD>
__global__ void __launch_bounds__(kShThreads) shared_join_kernel(const __grid_constant__ PAttn a, int per) {
  constexpr int kLanes = HD / 4, kRows = kShThreads / kLanes;
  const int b = blockIdx.x / per, R = (blockIdx.x - b * per) * kRows + (int)threadIdx.x / kLanes;
  const int r_first = __ldg(a.cu + b), n = __ldg(a.cu + b + 1) - r_first;
  // (The plan has been done since before the rest began.)
  const int4* own = reinterpret_cast<const int4*>(sh_seqs(a.ws, a.n_groups) + b);
  const int4 p0 = __ldcg(own), p1 = __ldcg(own + 1), plan = __ldcg(reinterpret_cast<const int4*>(a.ws));
  const ShSeq p{p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, {0, 0}};
  const int t = R / a.hq, h = R - t * a.hq, G = a.hq / a.hkv, col = (int)(threadIdx.x % kLanes) * 4;
  const size_t at = (size_t)(r_first + t) * a.hq + h;
  const bool live = r_first >= 0 && n > 0 && n <= a.tokens - r_first && t < min(n, a.max_q);
  pdl_wait();                                  // the prefix and the rest
  if (!live) return;
  float4 x = __ldcg(reinterpret_cast<const float4*>(a.rest + at * HD + col));
  const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.rest + (size_t)a.tokens * a.hq * HD) + at);
  float mm = ml.x, ll = ml.y;
  sh_join<HD>(a, p, plan.x, plan.y, h / G, r_first + t, h % G, col, x, mm, ll);
  const float f = ll > 0.f || !(ll == ll) ? 1.f / ll : 0.f;
  bf16* d = (bf16*)a.out + (int64_t)(r_first + t) * a.o_ts + (int64_t)h * a.o_hs + col;
  *reinterpret_cast<uint2*>(d) = make_uint2(ta_pack(x.x * f, x.y * f), ta_pack(x.z * f, x.w * f));
  if (a.lse && col == 0) a.lse[at] = ll == 0.f ? neg_inf() : (mm + log2f(ll)) * 0.6931471805599453f;
}

// Tiles (KV head, pair) that the groups can hold.
int64_t most_tiles(const PAttn& a) {
  const int tpt = kTaRows / (a.hq / a.hkv);
  return (int64_t)a.hkv * (a.tokens / (2 * tpt) + std::min<int64_t>(a.n_groups, a.tokens));
}

// The parts of 8-bit prefixes leave in 32-byte stores and slots lie at multiples of 32 bytes from the
// workspace's start, which callers align to 16: the start moves up to 32, in room asked for that.
constexpr size_t kShAlign = 32;

}  // namespace

size_t pattn_shared_workspace(const PAttn& a, int num_sms) {
  if (!a.paged || a.seqs > 1 << 24 || !pattn_tc_supported(a)) return 0;
  const int64_t keys = (int64_t)a.max_pages << a.page_shift, tiles = most_tiles(a);
  const int64_t rows = (int64_t)std::min(a.max_q, a.tokens) * a.hq;
  if (tiles * ((keys + kTaKeys - 1) / kTaKeys) > 0x3fffffffLL || (rows + 7) / 8 * a.seqs > 0x7fffffffLL) return 0;
  return kShAlign - 16 + sh_slots_at(a.n_groups, a.seqs) + ((size_t)(num_sms + tiles) * 256 + (size_t)a.tokens * a.hq) * (a.hd + 2) * sizeof(float);
}

cudaError_t launch_pattn_shared(const PAttn& call, int num_sms, cudaStream_t st) {
  PAttn a = call;
  a.runs = num_sms;
  a.ws = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(a.ws) + kShAlign - 1) & ~(uintptr_t)(kShAlign - 1));
  a.rest = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(a.ws) + sh_slots_at(a.n_groups, a.seqs)) +
           (size_t)(num_sms + most_tiles(a)) * 256 * (a.hd + 2);
  TaArgs ta{};
  if (!ta_args<kPaPrefix>(ta, a)) return cudaErrorInvalidValue;
  ta.items = num_sms;
  ta.split = 1;
  cudaError_t e = launch_rows(shared_plan_kernel, dim3(1), dim3(kShThreads), 0, 1, st, a, sh_cost(a));
  if (e == cudaSuccess) e = launch_ta_mode<kPaPrefix>(ta, st);
  if (e == cudaSuccess) e = launch_pa_rest(a, num_sms, st);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)std::min(a.max_q, a.tokens) * a.hq;
  auto join = [&](auto kernel, int per_block) {
    const int per = (int)((rows + per_block - 1) / per_block);
    return launch_rows_early(true, kernel, dim3((unsigned)(per * a.seqs)), dim3(kShThreads), 0, 1, st, a, per);
  };
  return a.hd == 64 ? join(shared_join_kernel<64>, kShThreads / 16) : join(shared_join_kernel<128>, kShThreads / 32);
}

}  // namespace sv
