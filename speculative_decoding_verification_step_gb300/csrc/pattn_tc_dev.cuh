// Attention of many rows per KV head (a chunk of prompt tokens, a whole
// prompt) on the fifth-generation tensor cores.
//
// Past ~64 rows a key is worth more arithmetic than its bytes: 4 flops per
// element and row, so the products bound the time, and next to them the
// exponentials (one per 4 head_dim flops: at head_dim 128 the two are close).
// The kernel keeps the tensor pipe fed while the softmax of one tile runs
// behind the products of the other.
//
// A block walks work items: two tiles of 128 rows (tokens x the G query heads
// of one KV head) against the keys in steps of 128, over a ring of
// shared-memory tiles filled by tensor copies, one box per page (128-byte
// swizzle, 64-dim halves).
//   warps 0-3, 4-7  softmax of tile 0, 1: a thread owns a row.  It reads its
//                   128 scores from tensor memory, takes the maximum without
//                   any exchange, writes p as bf16 over the scores and keeps
//                   the row sum in fp32.  The exponent reference is lazy: it
//                   moves only when a score exceeds it by 2^8, and only then
//                   O is rescaled in tensor memory.  Rows leave through 4 KB
//                   of shared memory a warp, as whole lines (a thread storing
//                   its own row took 6000 clocks a tile);
//   warp 8          producer: page ids and tensor copies (K_0 V_0 K_1 V_1 ..);
//   warp 9          issues the products, per step and tile O += P V (P from
//                   tensor memory, V as it lies, keys along K; the first 64
//                   keys while the other exponentials are taken), then
//                   S = Q K^T of the next step over the same columns that P
//                   occupied: the tensor pipe runs in issue order.  The warp
//                   stays converged and one elected lane issues: from a single
//                   thread's control flow an MMA took 100 clocks to issue;
//   warp 10         scheduler: hands the work items to the others through a
//                   queue in shared memory, two ahead;
//   warp 11         allocates and frees tensor memory;
//   warps 12-15     8-bit keys only: a thread turns one row of codes into bf16
//                   (code * 2^e is exact there), from the copies' ring into
//                   the products'.  Rows past the length become zero.
// Tensor memory, 512 columns: S/P 2 x 128, O 2 x head_dim.
// A block goes on to further items by taking over blocks of the grid that
// have not started (cluster launch control), and the ring runs on across
// items: the next item's Q, K and first scores are ready while the rows of
// this one leave (a block per item spent 13 thousand clocks on start and
// end, and a fixed share of the items per block left some 9% longer at
// work).  Items come heads side by side within a chunk of heads, so that they
// share keys in L2, and rows from each sequence's last to its first, so that
// the causal triangle's long rows start first.
// With few items (chunks of a few sequences) a cluster of two blocks shares an
// item's keys; block t finishes tile t with the other's sums, read from its
// shared memory.
// Bound by the tensor pipe where walks are long, and by a fixed 4 to 5 us an item
// (the softmax warps also drain, scale and store O before their next item): at 64
// steps an item takes 1.4 us a step, at 4.5 steps 10 us.  8-bit keys add the
// conversion of both tiles by four warps.  Measured at head dim 128, 32 heads on 8:
// six packed prompts of up to 4096 276 us (1.31 PFLOP/s, 69% of the library
// product's rate), one of 16384 1260 to 1300 us (90%), 16 of 1024 139 us (52%);
// four chunks of up to 512 tokens over up to 16384 keys 164 us (1.1 PFLOP/s), four
// of 512 over 16384 364 us (78%), with 8-bit keys 514 us (56%); head dim 64, four
// prompts of 4096 349 us (42%).
// Windows (Mode, paged.h).  An item walks the first tokens and, close behind them, the keys
// from the first that its first token's window reaches, so that four first tokens are 16 keys
// of a step and not a step of their own (six prompts in a window of 1024 173 -> 158 us); boxes
// are then 16 rows where a step holds both, else pages or 128 rows of a prompt.  A row's
// mask is 128 bits, from three bounds that go down by a step's keys.  Of nine steps an item
// takes in that window 8.25 would do, and the fixed time of an item is a third of its time:
// 158 us is 1.05 PFLOP/s of what the rows see (55%).  Four chunks of up to 512 in a window
// of 2048 36 us: 136 items of 18 steps, fewer than SMs, 1.4 us a step and 10 around them.
// Prefixes (pattn_shared.cu): no mask; a block's items are the parts of its run, and their sums
// leave as they are.  8-bit ones keep four tiles of codes in flight, where the other modes keep
// rows on their way out, and have eight warps to convert them: either alone gained 2%,
// both 6% of 96 us (64 x 6 tokens behind four prompts).
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "pa_dev.cuh"
#include "paged.h"

namespace sv {

namespace {

constexpr int kTaRows = 128;        // rows of a tile (MMA M)
constexpr int kTaKeys = 128;        // keys of a step
constexpr float kTaLazy = 8.f;
constexpr float kTaNone = -1e30f;

struct TaArgs {
  TensorMap128 qm, km, vm;
  PAttn a;
  int tpt;          // tokens of a tile: 128 / G
  uint32_t g_mul;   // ceil(2^16 / G): r * g_mul >> 16 = r / G for r < 128
  int pairs;        // row pairs of the longest sequence
  int chunk;        // (sequence, KV head) pairs in flight at a time
  int items;        // (sequence, KV head, row pair): seqs * hkv * pairs
  int split;        // 2: clusters of two blocks share an item's keys
  int by_length;    // sequences in order of their lengths (paged, at most 32)
  int box_rows;     // key rows of a K / V box
};

struct TaWindowArgs : TaArgs {
  TensorMap128 ks, vs;   // K and V in boxes of 16 rows
  int take;              // blocks take over further items
};
template <int Mode>
using TaArgsOf = std::conditional_t<Mode == kPaWindow, TaWindowArgs, TaArgs>;

template <int HD, bool F8, int Mode>
struct TaLayout {
  // 8-bit prefixes: sums leave by the thread that holds the row, in whole sectors, the room where
  // other rows wait on their way out holds more codes in flight, and eight warps convert them.
  static constexpr bool deep = F8 && Mode == kPaPrefix;
  static constexpr int convert = deep ? 8 : 4;             // warps that convert codes
  static constexpr int threads = F8 ? 384 + 32 * convert : 384;
  static constexpr int stages = F8 ? 3 : 4;                // bf16 K / V tiles
  static constexpr int raws = !F8 ? 0 : !deep ? 2 : HD == 128 ? 4 : 6;   // tiles of codes
  static constexpr uint32_t tile = kTaKeys * HD * 2;
  static constexpr uint32_t raw = kTaKeys * HD;
  static constexpr uint32_t q = 0, kv = 2 * tile, raw_at = kv + stages * tile, stage_at = raw_at + raws * raw;
  static constexpr uint32_t stage = 32 * 128;              // a warp's rows on their way out, 64 dims at a time
  static constexpr int smem = (int)(stage_at + (deep ? 0 : 8 * stage)) + 1024;
  static_assert(smem <= 227 * 1024 - 1536, "with the barriers and queues, one block's shared memory");
  // registers (multiples of 8): softmax, others, 8-bit conversion; 2 x 216 + 56 <= 3 x 168, 2 x 184 + 56 + 88 <= 4 x 128,
  // 2 x 176 + 48 + 2 x 40 <= 5 x 96
  static constexpr int soft_regs = deep ? 176 : F8 ? 184 : 216, other_regs = deep ? 48 : 56, convert_regs = deep ? 40 : 88;
};

SV_DEV uint32_t ta_cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
SV_DEV uint32_t ta_map_peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
SV_DEV void ta_arrive_peer(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
SV_DEV float4 ta_ld_peer(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
// The response of a take-over: the index of the block taken, or -1.
SV_DEV int ta_taken(const uint4* at) {
  uint32_t x = 0, got;
  asm volatile(
      "{\n .reg .b128 r;\n .reg .pred p;\n ld.shared.b128 r, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n selp.u32 %1, 1, 0, p;\n"
      " mov.u32 %0, 0;\n @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n}"
      : "=r"(x), "=r"(got) : "r"(smem_u32(at)) : "memory");
  return got ? (int)x : -1;
}
SV_DEV void ta_take(uint4* at, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
               ::"r"(smem_u32(at)), "r"(smem_u32(bar)) : "memory");
}

// A work item as every warp sees it.
struct TaItemBase {
  int valid;          // 0: no more items
  int kvh, b, r_first, toks, keys, first_pos, tok0, ntile;
  int beg, nst;       // this block's key steps beg .. beg + nst - 1
  int steps[2];       // of those, each tile's (from beg)
};
template <int Mode>
struct TaItemOf : TaItemBase {};
template <>
struct TaItemOf<kPaWindow> : TaItemBase {
  int lo, lead, gap;  // keys below lo (but the sinks) are seen by no row; place p of the walk is key p, from `lead` on p + gap
};
template <>
struct TaItemOf<kPaPrefix> : TaItemBase {
  int slot, unit;     // where the part goes, the unit behind it
};

// Hook: the form of SPEC_FAULT_ATTN_TIMEOUT, whose a.give_up-th step waits for what never comes.
template <int HD, bool F8, bool Hook, int Mode>
__global__ void __launch_bounds__(TaLayout<HD, F8, Mode>::threads, 1) pattn_tc_kernel(const __grid_constant__ TaArgsOf<Mode> ta) {
  using L = TaLayout<HD, F8, Mode>;
  using TaItem = TaItemOf<Mode>;
  constexpr int kHalf = HD / 64;                       // 64-dim halves of a row
  constexpr uint32_t kTile = L::tile;
  constexpr int kS = L::stages, kR = F8 ? L::raws : 1;
  extern __shared__ __align__(1024) unsigned char tsm[];
  __shared__ uint64_t q_full, q_free, kv_full[kS], kv_empty[kS], s_full[2], p_half[2], p_full[2], pv_done[2];
  __shared__ uint64_t raw_full[kR], raw_empty[kR], drained, part_full, item_full[2], item_empty[2], taken;
  __shared__ __align__(16) uint4 s_taken;
  __shared__ TaItem s_item[2];
  __shared__ __align__(16) unsigned char s_scale[kR][kTaKeys];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ int s_filled, s_qloads;
  const PAttn& a = ta.a;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int G = a.hq / a.hkv, tpt = ta.tpt;
  const int rank = ta.split > 1 ? (int)ta_cluster_rank() : 0;
  const int sinks = Mode == kPaWindow ? a.sinks : 0;
  // Key at place p of the item's walk.  Windows walk the first tokens, in runs of 16,
  // and the window close behind them, so that both may lie in one step.  What is left
  // out between them is whole boxes of a paged cache: a box lies within one page.
  auto key_at = [&](const TaItem& it, int p) {
    if constexpr (Mode == kPaWindow) return p + (p < it.lead ? 0 : it.gap);
    else return p;
  };
  // Some row of the item may see one of the n keys from `key` on.
  [[maybe_unused]] auto reached = [&](const TaItem& it, int64_t key, int n) {
    if constexpr (Mode == kPaWindow) return key + n > it.lo || key < sinks;
    else return true;
  };
  // Prefixes: the part of this block's run that starts at unit u; false at its end.
  [[maybe_unused]] auto part_at = [&](int u, TaItem& it) {
    if constexpr (Mode == kPaPrefix) {
      // the plan and the first groups' records, one a lane, in one round of loads
      const int4* at = reinterpret_cast<const int4*>(sh_groups(a.ws));
      const int4 plan = __ldcg(reinterpret_cast<const int4*>(a.ws));      // units, runs
      int4 x = __ldcg(at + 2 * min(lane, a.n_groups - 1)), y = __ldcg(at + 2 * min(lane, a.n_groups - 1) + 1);   // a ShGroup
      const int units = plan.x, runs = plan.y, run = (int)blockIdx.x;
      if (run >= runs) return false;
      const int end = sh_begin(run + 1, units, runs);
      if (u < 0) u = sh_begin(run, units, runs);
      if (u >= end) return false;
      int g = 0;                                 // the last group that begins at or before u: one that holds units
      for (int g0 = 0; g0 < a.n_groups; g0 += 32) {
        const int first = g0 == 0 ? x.y : __ldcg(&sh_groups(a.ws)[min(g0 + lane, a.n_groups - 1)].unit0);
        const unsigned in = __ballot_sync(0xffffffffu, g0 + lane < a.n_groups && first <= u);
        if (in) g = g0 + 31 - __clz(in);
      }
      if (g >= 32) {
        x = __ldcg(at + 2 * g);
        y = __ldcg(at + 2 * g + 1);
      }
      auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, g & 31); };
      const int in = u - of(x.y), steps = of(y.w), pairs = of(y.z), tile = in / steps, off = in - tile * steps;
      it.kvh = tile / pairs;
      it.b = of(y.y);
      it.r_first = of(x.w);
      it.toks = of(y.x);
      it.keys = it.first_pos = of(x.x);
      it.tok0 = (tile - it.kvh * pairs) * 2 * tpt;
      it.ntile = it.tok0 + tpt < it.toks ? 2 : 1;
      it.beg = off;
      it.nst = min(steps - off, end - u);
      it.steps[0] = it.nst;
      it.steps[1] = it.ntile == 2 ? it.nst : 0;
      it.slot = run + of(x.z) + tile;
      it.unit = u + it.nst;
      return true;
    } else {
      return false;
    }
  };
  // Item `idx` (its rows and lengths read from the index arrays); false when
  // it holds no rows.  Called by whole warps.
  auto item_at = [&](int idx, TaItem& it) {
    if constexpr (Mode == kPaPrefix) return part_at(idx, it);
    if (ta.by_length) {                        // the warp's lanes rank the sequences, longest first
      const int per_seq = a.hkv * ta.pairs, k = idx / per_seq, in = idx - k * per_seq, up = in / a.hkv;
      const int len = lane < a.seqs ? __ldg(a.lens + lane) : -0x7fffffff - 1;
      int before = 0;
      for (int j = 0; j < a.seqs; ++j) {
        const int other = __shfl_sync(0xffffffffu, len, j);
        before += other > len || (other == len && j < lane);
      }
      it.b = __ffs(__ballot_sync(0xffffffffu, lane < a.seqs && before == k)) - 1;
      it.kvh = in - up * a.hkv;
      it.tok0 = (ta.pairs - 1 - up) * 2 * tpt;
    } else {
      const int per_chunk = ta.chunk * ta.pairs, ch = idx / per_chunk, in = idx - ch * per_chunk;
      const int width = min(ta.chunk, a.hkv * a.seqs - ch * ta.chunk);
      const int up = in / width, head = ch * ta.chunk + in - up * width;
      it.b = head / a.hkv;
      it.kvh = head - it.b * a.hkv;
      it.tok0 = (ta.pairs - 1 - up) * 2 * tpt;
    }
    it.r_first = __ldg(a.cu + it.b);
    const int n = __ldg(a.cu + it.b + 1) - it.r_first;
    int keys = a.paged ? __ldg(a.lens + it.b) : n;
    if (it.r_first < 0 || n <= 0 || n > a.tokens - it.r_first) return false;
    it.toks = min(n, a.max_q);                // tokens that are computed
    if (it.tok0 >= it.toks) return false;
    if (a.paged) keys = keys < 0 ? 0 : (int)min((int64_t)keys, (int64_t)a.max_pages << a.page_shift);
    it.keys = keys;
    it.first_pos = keys - n;
    it.ntile = it.tok0 + tpt < it.toks ? 2 : 1;
    if constexpr (Mode == kPaWindow) {
      it.lo = max(0, max(0, it.first_pos + it.tok0) - a.window + 1);
      it.lead = (min(sinks, keys) + 15) & ~15;
      it.gap = max(0, it.lo - it.lead);
      if (a.paged) it.gap -= it.gap & (ta.box_rows - 1);
    }
    int all[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {             // key steps of each tile: what its last token sees
      const int last = min(it.toks, it.tok0 + (t + 1) * tpt) - 1;
      int see = min(keys, max(0, it.first_pos + last + 1));
      if constexpr (Mode == kPaWindow) see = max(0, see - it.gap);
      all[t] = t < it.ntile ? (see + kTaKeys - 1) / kTaKeys : 0;
    }
    const int total = max(all[0], all[1]);
    it.beg = total * rank / ta.split;
    it.nst = total * (rank + 1) / ta.split - it.beg;
#pragma unroll
    for (int t = 0; t < 2; ++t) it.steps[t] = max(0, min(all[t] - it.beg, it.nst));
    return true;
  };
  TaItem mine;
  mine.valid = Mode != kPaPrefix && item_at((int)blockIdx.x / ta.split, mine);
  if (Mode != kPaPrefix && !mine.valid) return;                    // (all blocks of a cluster)

  const uint32_t base = (smem_u32(tsm) + 1023u) & ~1023u;
  const uint32_t q_at = base + L::q, kv_at = base + L::kv, raw_at = base + L::raw_at;
  if (warp == 8 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&ta.qm)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&ta.km)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&ta.vm)) : "memory");
    mbar_init(&q_full, 1);
    mbar_init(&q_free, 1);
    mbar_init(&drained, 1);
    mbar_init(&part_full, 4 * max(1, ta.split - 1));   // four warps of every other block
    mbar_init(&taken, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&item_full[s], 1);
      mbar_init(&item_empty[s], F8 ? 10 + L::convert : 10);   // one arrival per warp that works on items
    }
    for (int s = 0; s < kS; ++s) {
      mbar_init(&kv_full[s], F8 ? L::convert : 1);   // converted by so many warps, or copied
      mbar_init(&kv_empty[s], 1);
    }
    for (int s = 0; s < kR; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], L::convert);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_half[t], 4);        // one arrival per softmax warp
      mbar_init(&p_full[t], 4);
      mbar_init(&pv_done[t], 1);
    }
    s_abort = 0;
    s_filled = s_qloads = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 11) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  ta_fence_before();
  __syncthreads();
  // a peer's barrier exists before anything arrives there
  if (ta.split > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
  ta_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  constexpr uint32_t o_at = 256;
  if constexpr (Mode == kPaPrefix) {           // begun early: what the launch in front left is read from here on
    pdl_wait();
    pdl_trigger();
    mine.valid = part_at(-1, mine);
  }

  // Next item of the queue (the k-th of this block); false at the end or, but for
  // `last`, when a wait gave up.  The softmax warps take all that is handed out:
  // no other block will write those rows.
  auto get_item = [&](int k, TaItem& it, bool last = false) {
    const bool got = __all_sync(0xffffffffu, last ? ta_land(&item_full[k & 1], (unsigned)((k >> 1) & 1))
                                                  : ta_wait(&item_full[k & 1], (unsigned)((k >> 1) & 1), &s_abort));
    if (Mode != kPaPrefix || s_item[k & 1].valid) it = s_item[k & 1];   // (the end leaves the last part where it is)
    else it.valid = 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[k & 1]);
    return got && it.valid;
  };

  if (warp >= 12) {
    if constexpr (F8) {
      // ---- 8-bit rows to bf16: thread = key row, or half of one ----
      constexpr int kChunks = HD / 16 * 4 / L::convert;
      ta_regs_less<L::convert_regs>();
      const int r = (threadIdx.x - 384) & 127, c0 = (threadIdx.x - 384) / 128 * kChunks;
      int i = 0;                               // tile: K and V of the steps of all items in turn
      bool ok = true;
      TaItem it;
      for (int k = 0; ok && get_item(k, it); ++k) {
        for (int j = 0; ok && j < 2 * it.nst; ++j, ++i) {
          const int rs = i % kR, s = i % kS;
          ok = ta_wait(&raw_full[rs], (unsigned)((i / kR) & 1), &s_abort);
          if (ok && i >= kS) ok = ta_wait(&kv_empty[s], (unsigned)((i / kS - 1) & 1), &s_abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t code = s_scale[rs][r];
          const int key = key_at(it, (it.beg + j / 2) * kTaKeys + r);
          const bool live = key < it.keys && reached(it, key, 1);
          // a row past the length, or that no row sees, is zero whatever it holds
          const float f = !live ? 0.f : row_power(code);
          const uint64_t scale = ta_pair(f, f);
          const uint32_t src = raw_at + rs * L::raw + r * HD, dst = kv_at + s * kTile + r * 128;
#pragma unroll
          for (int ci = 0; ci < kChunks; ++ci) {
            uint32_t w[4], o[8];
            const int c = c0 + ci;
            const int sw = HD == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(src + (sw << 4)) : "memory");
#pragma unroll
            for (int k = 0; k < 4; ++k) ta_codes(live ? w[k] : 0u, scale, o[2 * k], o[2 * k + 1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int cc = 2 * c + h, col = cc & 7;
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                           ::"r"(dst + (cc >> 3) * (kTile / kHalf) + ((col ^ (r & 7)) << 4)), "r"(o[4 * h]), "r"(o[4 * h + 1]),
                             "r"(o[4 * h + 2]), "r"(o[4 * h + 3]) : "memory");
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&raw_empty[rs]);
            mbar_arrive(&kv_full[s]);
          }
        }
      }
    }
  } else if (warp >= 8) {
    ta_regs_less<L::other_regs>();
    if (warp == 8) {
      // ---- producer ----
      const int per_step = a.paged ? kTaKeys / ta.box_rows : 1;   // boxes of a step
      constexpr int kRing = F8 ? L::raws : kS;
      uint64_t* const full = F8 ? raw_full : kv_full;
      uint64_t* const empty = F8 ? raw_empty : kv_empty;
      int i = 0, loads = 0;                                    // ring fills, Q loads
      bool live = true;
      TaItem it;
      for (int k = 0; live && get_item(k, it); ++k) {
        if (it.nst == 0) continue;
        if (loads > 0) live = __all_sync(0xffffffffu, ta_wait(&q_free, (unsigned)((loads - 1) & 1), &s_abort));
        if (!live) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full, (unsigned)(it.ntile * kHalf * 128 * G * tpt));
          s_qloads = loads + 1;
          for (int t = 0; t < it.ntile; ++t)
            for (int h = 0; h < kHalf; ++h)
              ta_tma_3d(q_at + t * kTile + h * (kTile / kHalf), &ta.qm, h * 64, it.kvh * G, it.r_first + it.tok0 + t * tpt,
                        &q_full);
        }
        ++loads;
        const int32_t* table = a.paged ? a.table + it.b * a.table_stride : nullptr;
        const int npages = a.paged ? (int)(((int64_t)it.keys + (1 << a.page_shift) - 1) >> a.page_shift) : 0;
        // small boxes where a step holds first tokens and window
        auto is_small = [&](int j) {
          if constexpr (Mode == kPaWindow) {
            const int at = (it.beg + j) * kTaKeys;
            return it.gap > 0 && at < it.lead && at + kTaKeys > it.lead;
          } else {
            return false;
          }
        };
        auto box_key = [&](int j) {   // first key of box `lane`
          if constexpr (Mode == kPaWindow) return (int64_t)key_at(it, (it.beg + j) * kTaKeys + lane * (is_small(j) ? 16 : ta.box_rows));
          else return (int64_t)(it.beg + j) * kTaKeys + (a.paged ? lane * ta.box_rows : 0);
        };
        // lane b: page of box b of step j; -1 (zero rows) past the length, outside the pool or where no row sees it
        auto page_of = [&](int j) {
          const int64_t key = box_key(j);
          const int pg = (int)(key >> a.page_shift);
          const bool small = is_small(j);
          const int page = lane < (small ? kTaKeys / 16 : per_step) && j < it.nst && pg < npages &&
                                   reached(it, key, small ? 16 : ta.box_rows)
                               ? __ldg(table + pg)
                               : -1;
          return page >= a.pages ? -1 : page;
        };
        int next = a.paged ? page_of(0) : 0;
        for (int j = 0; j < it.nst && live; ++j) {
          const int page = next;
          if (a.paged) next = page_of(j + 1);
          const int64_t key = box_key(j);
          const int row = a.paged ? (it.kvh << a.page_shift) + (int)(key & ((1 << a.page_shift) - 1)) : it.kvh;
          const bool small = is_small(j);
          const int box = small ? 16 : ta.box_rows, per = small ? kTaKeys / 16 : per_step;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++i) {
            const int s = i % kRing;
            if (i >= kRing) live = live && ta_wait(&empty[s], (unsigned)((i / kRing - 1) & 1), &s_abort);
            live = __all_sync(0xffffffffu, live);
            if (!live) break;
            const void* map = kv ? &ta.vm : &ta.km;
            if constexpr (Mode == kPaWindow)
              if (small) map = kv ? &ta.vs : &ta.ks;
            if constexpr (F8) {
              const bool in = lane < per && page >= 0;
              const unsigned some = __ballot_sync(0xffffffffu, in);
              if (lane < per && !in)
                for (int e = 0; e < box; e += 4) *reinterpret_cast<uint32_t*>(&s_scale[s][lane * box + e]) = 0x7f7f7f7fu;
              __syncwarp();
              if (lane == 0) {
                mbar_arrive_expect_tx(&full[s], L::raw + __popc(some) * box);
                s_filled = i + 1;
              }
              __syncwarp();
              if (lane < per) {
                ta_tma_3d(raw_at + s * L::raw + lane * box * HD, map, 0, row, page, &full[s]);
                if (in) bulk_g2s(&s_scale[s][lane * box], (kv ? a.vs : a.ks) + (int64_t)page * a.scale_stride + row,
                                 box, &full[s]);
              }
            } else {
              if (lane == 0) {
                mbar_arrive_expect_tx(&full[s], kTile);
                s_filled = i + 1;
              }
              __syncwarp();
              if (lane < per) {
                for (int h = 0; h < kHalf; ++h)
                  ta_tma_3d(kv_at + s * kTile + h * (kTile / kHalf) + lane * box * 128, map, h * 64, row,
                            a.paged ? page : it.r_first + (int)key, &full[s]);
              }
            }
          }
        }
      }
      // the last fills are used, and the products' signals have landed, before the block ends
      for (int k = max(0, i - kRing); live && k < i; ++k)
        live = __all_sync(0xffffffffu, ta_wait(&empty[k % kRing], (unsigned)((k / kRing) & 1), &s_abort));
      if (live && loads > 0) ta_wait(&q_free, (unsigned)((loads - 1) & 1), &s_abort);
      if constexpr (F8) {
        for (int k = max(0, i - kS); live && k < i; ++k)
          live = __all_sync(0xffffffffu, ta_wait(&kv_empty[k % kS], (unsigned)((k / kS) & 1), &s_abort));
      }
    } else if (warp == 9) {
      // ---- products ----
      // The whole warp runs the control flow, so that descriptors and addresses
      // stay in uniform registers; one elected lane issues.
      constexpr uint32_t id_s = ta_idesc(kTaKeys, 0), id_o = ta_idesc(HD, 1);
      auto wait = [&](uint64_t* bar, unsigned parity) {
        const bool got = __all_sync(0xffffffffu, ta_wait(bar, parity, &s_abort));
        ta_fence_after();
        return got;
      };
      // S_t = Q_t K^T from ring fill i
      auto score = [&](int t, int i) {
        const uint64_t qd = ta_desc(q_at + t * kTile, 1), kd = ta_desc(kv_at + (uint32_t)(i % kS) * kTile, 1);
        if (ta_elect()) {
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks) {
            constexpr uint32_t half = kTile / kHalf / 16;
            const uint32_t off = (ks / 4) * half + (ks % 4) * 2;   // 16-byte units
            ta_mma_ss(tmem + t * 128, qd + off, kd + off, id_s, ks > 0);
          }
          ta_commit(&s_full[t]);
        }
        __syncwarp();
      };
      // O_t += P_t V over half of a step's keys, V from ring fill i
      auto gather = [&](int t, int i, int half, bool fresh) {
        const uint64_t vd = ta_desc(kv_at + (uint32_t)(i % kS) * kTile, (kTile / kHalf) >> 4);
        if (ta_elect()) {
#pragma unroll
          for (int k4 = 0; k4 < kTaKeys / 32; ++k4) {
            const int ks = half * (kTaKeys / 32) + k4;
            ta_mma_ts(tmem + o_at + t * HD, tmem + t * 128 + ks * 8, vd + ks * 128, id_o, !fresh || ks > 0);
          }
          if (half) ta_commit(&pv_done[t]);
        }
        __syncwarp();
      };
      // signals bar once the products issued so far are done
      auto signal = [&](uint64_t* bar) {
        if (ta_elect()) ta_commit(bar);
        __syncwarp();
      };
      int i0 = 0, loads = 0;                  // ring fill of the item's first K, Q loads
      unsigned np[2] = {0, 0};                // steps of each tile over all items
      [[maybe_unused]] int hook = a.give_up;
      bool ok = true;
      TaItem it;
      for (int k = 0; ok && get_item(k, it); ++k) {
        // (the same in every lane; said so for uniform registers)
        it.beg = __shfl_sync(0xffffffffu, it.beg, 0);
        it.nst = __shfl_sync(0xffffffffu, it.nst, 0);
        it.keys = __shfl_sync(0xffffffffu, it.keys, 0);
        if constexpr (Mode == kPaWindow) {
          it.lo = __shfl_sync(0xffffffffu, it.lo, 0);
          it.lead = __shfl_sync(0xffffffffu, it.lead, 0);
          it.gap = __shfl_sync(0xffffffffu, it.gap, 0);
        }
        it.steps[0] = __shfl_sync(0xffffffffu, it.steps[0], 0);
        it.steps[1] = __shfl_sync(0xffffffffu, it.steps[1], 0);
        if (it.nst == 0) continue;
        ok = wait(&q_full, (unsigned)(loads & 1)) && wait(&kv_full[i0 % kS], (unsigned)((i0 / kS) & 1));
        if (!ok) break;
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (it.steps[t] > 0) score(t, i0);
        signal(&kv_empty[i0 % kS]);
        if (it.nst == 1) signal(&q_free);
        for (int j = 0; ok && j < it.nst; ++j) {
          const int iv = i0 + 2 * j + 1, ik = iv + 1;
          ok = wait(&kv_full[iv % kS], (unsigned)((iv / kS) & 1));
          if constexpr (Hook) ok = ok && (--hook != 0 || __all_sync(0xffffffffu, ta_wait(&drained, 0, &s_abort, 0)));
          if constexpr (!F8) {
            // V's rows past the length: p is zero there, but the slots may hold anything
            const int at = (it.beg + j) * kTaKeys;
            int rows = it.keys - at;
            if constexpr (Mode == kPaWindow) rows -= it.gap;
            auto clear = [&](int from, int to) {
              for (int h = 0; h < kHalf; ++h)
                for (int e = from * 8 + lane; e < to * 8; e += 32)
                  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};"
                               ::"r"(kv_at + (iv % kS) * kTile + h * (kTile / kHalf) + e * 16), "r"(0) : "memory");
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
            };
            if (ok && rows < kTaKeys) clear(rows, kTaKeys);
            if constexpr (Mode == kPaWindow) {  // and those between the sinks and the windows
              const int from = min(max(sinks - at, 0), kTaKeys), to = min(max(it.lo - it.gap - at, 0), kTaKeys);
              if (ok && from < to) clear(from, to);
            }
          }
          bool have_k = false;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            // the first 64 keys' products run while the other exponentials are taken
            if (ok && j < it.steps[t]) {
              ok = wait(&p_half[t], np[t] & 1);
              if (ok) {
                gather(t, iv, 0, j == 0);
                ok = wait(&p_full[t], np[t] & 1);
                if (ok) gather(t, iv, 1, j == 0);
              }
              ++np[t];
            }
            if (ok && j + 1 < it.steps[t]) {
              if (!have_k) ok = wait(&kv_full[ik % kS], (unsigned)((ik / kS) & 1));
              have_k = true;
              if (ok) score(t, ik);
            }
          }
          if (!ok) break;
          signal(&kv_empty[iv % kS]);
          if (j + 1 < it.nst) signal(&kv_empty[ik % kS]);
          if (j + 2 == it.nst) signal(&q_free);   // the last scores are issued
        }
        i0 += 2 * it.nst;
        ++loads;
      }
    } else if (warp == 10) {
      // ---- scheduler ----
      // (An item is handed out after all have begun the one before, so the queue's
      // other place is free: the end of the queue is handed out without a wait.)
      TaItem it = mine;
      unsigned takes = 0;
      for (int k = 0;; ++k) {
        if (lane == 0) {
          s_item[k & 1] = it;
          mbar_arrive(&item_full[k & 1]);
        }
        __syncwarp();
        if (!it.valid) break;
        // one item ahead: the next is taken when all have begun this one
        const bool ok = __all_sync(0xffffffffu, ta_wait(&item_empty[k & 1], (unsigned)((k >> 1) & 1), &s_abort));
        it.valid = 0;
        // a block of the grid that has not started and holds rows; none once a wait gave up
        if constexpr (Mode == kPaPrefix) {
          const bool go = ok && !__any_sync(0xffffffffu, s_abort);
          it.valid = go && part_at(it.unit, it);
        }
        bool take = Mode == kPaCausal && ta.split == 1;
        if constexpr (Mode == kPaWindow) take = ta.take;
        while (take && ok && !__any_sync(0xffffffffu, s_abort)) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&taken, 16);
            ta_take(&s_taken, &taken);
          }
          // the response is waited for whatever else gave up: a block that was taken
          // over never starts, so its item is handed out (and becomes NaN)
          const bool got = __all_sync(0xffffffffu, ta_land(&taken, takes & 1));
          ++takes;
          if (!got) break;
          const int idx = ta_taken(&s_taken);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // read before the next response lands there
          __syncwarp();
          if (idx < 0) break;
          it.valid = item_at(idx, it);
          if (it.valid) break;
        }
      }
      // had that wait run out: the response lands (bounded) before the space goes
      long long spins = 0;
      while (takes > 0 && !mbar_test(&taken, (takes - 1) & 1) && ++spins < (1LL << 20)) {
      }
    }
  } else {
    ta_regs_more<L::soft_regs>();
    // ---- softmax of tile t: one row per thread ----
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;
    const int ti = (int)((uint32_t)r * ta.g_mul >> 16);      // r / G
    const uint32_t row = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + row + t * 128, out_at = tmem + row + o_at + t * HD;
    const uint32_t stage = base + L::stage_at + warp * L::stage;
    const float scale = a.scale_log2;
    unsigned np = 0;                           // steps of this tile over all items
    bool ok = true;
    TaItem it;
    if constexpr (Mode == kPaPrefix) it.unit = -1;
    for (int k = 0; get_item(k, it, true); ++k) {   // (after a wait gave up: what was handed out still gets its NaN)
      const int t_at = it.tok0 + t * tpt, tok = t_at + ti;
      const bool row_ok = t < it.ntile && ti < tpt && tok < it.toks;
      const int seen = row_ok ? min(it.keys, max(0, it.first_pos + tok + 1)) : 0;
      const int tile_all = min(it.keys, max(0, it.first_pos + t_at + 1));   // keys that every row sees
      // windows: places from here that the row sees, [low, high) and those below `first`
      // (rows that are none of the item's see all: they are not written)
      [[maybe_unused]] int high = 1 << 30, low = 0, first = 0;
      if constexpr (Mode == kPaWindow) {
        if (row_ok) {
          high = seen - it.gap - it.beg * kTaKeys;
          low = (int)max((int64_t)0, (int64_t)high - a.window);   // (below 0 is as good as 0)
          first = max(min(sinks, seen) - it.beg * kTaKeys, 0);
        }
      }
      float m = kTaNone, l = 0.f;
      const int my = it.steps[t];
      for (int j = 0; ok && j < my; ++j, ++np) {
        ok = ta_wait(&s_full[t], np & 1, &s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ta_fence_after();
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) ta_ld32(s_at + 32 * c, s + 32 * c);
        ta_wait_ld();
        if constexpr (Mode == kPaWindow) {
          if (__any_sync(0xffffffffu, high < kTaKeys || low > 0)) {
            auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t see = (below(high - 32 * w) & ~below(low - 32 * w)) | below(first - 32 * w);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(see >> c & 1u)) s[32 * w + c] = neg_inf();
            }
          }
          high -= kTaKeys;
          low = max(low - kTaKeys, 0);
          first = max(first - kTaKeys, 0);
        } else {
          const int key0 = (it.beg + j) * kTaKeys;
          if (key0 + kTaKeys > tile_all) {
            const int lim = seen - key0;
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c >= lim) s[c] = neg_inf();
          }
        }
        float t0 = s[0], t1 = s[1], t2 = s[2], t3 = s[3];
#pragma unroll
        for (int c = 4; c < 124; c += 8) {
          t0 = ta_max3(t0, s[c], s[c + 1]);
          t1 = ta_max3(t1, s[c + 2], s[c + 3]);
          t2 = ta_max3(t2, s[c + 4], s[c + 5]);
          t3 = ta_max3(t3, s[c + 6], s[c + 7]);
        }
        t0 = ta_max3(t0, s[124], s[125]);
        t1 = ta_max3(t1, s[126], s[127]);
        const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * scale;
        const bool move = top > m + kTaLazy;
        if (__any_sync(0xffffffffu, move)) {
          const float to = move ? top : m, f = ta_exp2(m - to);
          m = to;
          l *= f;
          if (j > 0) {
            ok = ta_wait(&pv_done[t], (np - 1) & 1, &s_abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ta_fence_after();
#pragma unroll 1
            for (int c = 0; c < HD; c += 32) {
              float o[32];
              ta_ld32(out_at + c, o);
              ta_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= f;
              ta_st32(out_at + c, reinterpret_cast<uint32_t*>(o));
            }
          }
        }
        const uint64_t neg2 = ta_pair(-m, -m), scale2 = ta_pair(scale, scale);
        uint64_t sum0 = ta_pair(0.f, 0.f), sum1 = sum0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {          // 32 keys at a time: scores out, probabilities in
          uint32_t p[16];
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const int i = 32 * q + c;
            float x0, x1, x2, x3;
            ta_split(ta_fma2(ta_pair(s[i], s[i + 1]), scale2, neg2), x0, x1);
            ta_split(ta_fma2(ta_pair(s[i + 2], s[i + 3]), scale2, neg2), x2, x3);
            x0 = ta_exp2(x0); x1 = ta_exp2(x1); x2 = ta_exp2(x2); x3 = ta_exp2(x3);
            sum0 = ta_add2(sum0, ta_pair(x0, x1));
            sum1 = ta_add2(sum1, ta_pair(x2, x3));
            p[c / 2] = ta_pack(x0, x1);
            p[c / 2 + 1] = ta_pack(x2, x3);
          }
          ta_st16(s_at + 16 * q, p);
          if (q & 1) {
            ta_wait_st();
            ta_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(q == 1 ? &p_half[t] : &p_full[t]);
          }
        }
        float a0, a1;
        ta_split(ta_add2(sum0, sum1), a0, a1);
        l += a0 + a1;
      }
      if (ok && my > 0) {
        ok = ta_wait(&pv_done[t], (np - 1) & 1, &s_abort);
        ok = __all_sync(0xffffffffu, ok);
        ta_fence_after();
      }
      if (t >= it.ntile) continue;
      float o[HD];
      if (ok && my > 0) {
#pragma unroll
        for (int c = 0; c < HD; c += 32) ta_ld32(out_at + c, o + c);
        ta_wait_ld();
        ta_fence_before();
      } else {
#pragma unroll
        for (int c = 0; c < HD; ++c) o[c] = 0.f;
      }
      if constexpr (Mode == kPaPrefix) {        // sums as they are, for the join
        if (!ok) l = __uint_as_float(0x7fffffffu);
        float* const slot = sh_slot(a.ws, a.n_groups, a.seqs, HD, it.slot);
        if constexpr (L::deep) {
          float* const at = slot + (size_t)(t * kTaRows + r) * HD;
          if (row_ok)
#pragma unroll
            for (int c = 0; c < HD; c += 8)
              asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                           ::"l"(at + c), "f"(o[c]), "f"(o[c + 1]), "f"(o[c + 2]), "f"(o[c + 3]), "f"(o[c + 4]), "f"(o[c + 5]),
                             "f"(o[c + 6]), "f"(o[c + 7]) : "memory");
        } else {
          const int c16 = lane & 7, first = t * kTaRows + (warp & 3) * 32, rows = min(tpt, it.toks - t_at) * G;
#pragma unroll
          for (int h = 0; h < HD / 32; ++h) {     // 32 dims of the warp's rows at a time, out as whole lines
#pragma unroll
            for (int c = 0; c < 8; ++c)
              asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};"
                           ::"r"(stage + (uint32_t)(lane * 128 + ((c ^ (lane & 7)) << 4))), "f"(o[32 * h + 4 * c]),
                             "f"(o[32 * h + 4 * c + 1]), "f"(o[32 * h + 4 * c + 2]), "f"(o[32 * h + 4 * c + 3]) : "memory");
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const int r2 = i + (lane >> 3);
              float4 x;
              asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                           : "r"(stage + (uint32_t)(r2 * 128 + ((c16 ^ (r2 & 7)) << 4))) : "memory");
              if ((warp & 3) * 32 + r2 < rows)
                __stcg(reinterpret_cast<float4*>(slot + (size_t)(first + r2) * HD + 32 * h) + c16, x);
            }
            __syncwarp();
          }
        }
        if (row_ok) __stcg(reinterpret_cast<float2*>(slot + 256 * HD) + t * kTaRows + r, make_float2(m, l));
        continue;
      }
      if (ta.split > 1) {
        // One item a block: the ring is free once both tiles' products are done.
        // (Each tile's warps have waited for their own, step by step; a wait for the
        // other tile's last one by its parity could pass two steps early.)
        if (it.ntile == 2) named_sync(1, 256);
        const uint32_t part = kv_at + t * 2 * kTile;       // [dims / 4][row] of four sums
        if (t != rank) {                       // for the tile's finisher
          if (!ok) l = __uint_as_float(0x7fffffffu);
#pragma unroll
          for (int c = 0; c < HD / 4; ++c)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};"
                         ::"r"(part + (uint32_t)(c * kTaRows + r) * 16), "f"(o[4 * c]), "f"(o[4 * c + 1]), "f"(o[4 * c + 2]),
                           "f"(o[4 * c + 3]) : "memory");
          // and its reference and sum, in the warp's room for rows
          asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(stage + lane * 8), "f"(m), "f"(l) : "memory");
          __syncwarp();
          if (lane == 0) ta_arrive_peer(ta_map_peer(smem_u32(&part_full), (uint32_t)t));
          continue;
        }
        bool got = ta_wait(&part_full, 0, &s_abort);
        got = __all_sync(0xffffffffu, got);
        ok = ok && got;
        if (ok) {
          asm volatile("fence.acq_rel.cluster;" ::: "memory");
          for (int peer = 0; peer < ta.split; ++peer) {
            if (peer == rank) continue;
            float m2, l2;
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                         : "=f"(m2), "=f"(l2) : "r"(ta_map_peer(stage + lane * 8, (uint32_t)peer)) : "memory");
            const float to = fmaxf(m, m2), f1 = ta_exp2(m - to), f2 = ta_exp2(m2 - to);
            const uint32_t po = ta_map_peer(part + (uint32_t)r * 16, (uint32_t)peer);
#pragma unroll
            for (int c = 0; c < HD / 4; ++c) {
              const float4 y = ta_ld_peer(po + (uint32_t)(c * kTaRows) * 16);
              o[4 * c] = o[4 * c] * f1 + y.x * f2;
              o[4 * c + 1] = o[4 * c + 1] * f1 + y.y * f2;
              o[4 * c + 2] = o[4 * c + 2] * f1 + y.z * f2;
              o[4 * c + 3] = o[4 * c + 3] * f1 + y.w * f2;
            }
            m = to;
            l = l * f1 + l2 * f2;
          }
        }
      }
      // rows out; a wait that gave up leaves NaN, not a wrong number
      const float inv = !ok ? __uint_as_float(0x7fffffffu) : l == 0.f ? 0.f : 1.f / l;
      const int cc = lane & 7, r_at = (warp & 3) * 32 + (lane >> 3);
      const int o_ts = (int)a.o_ts, o_hs = (int)a.o_hs;    // 128 tokens' rows lie within 2^31 elements
      const uint64_t inv2 = ta_pair(inv, inv);
      bf16* const out0 = (bf16*)a.out + (int64_t)(it.r_first + t_at) * a.o_ts + (int64_t)(it.kvh * G) * a.o_hs + cc * 8;
#pragma unroll
      for (int h = 0; h < kHalf; ++h) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x, y;
            ta_split(ta_mul2(ta_pair(o[64 * h + 8 * c + 2 * i], o[64 * h + 8 * c + 2 * i + 1]), inv2), x, y);
            w[i] = ta_pack(x, y);
          }
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                       ::"r"(stage + (uint32_t)(lane * 128 + ((c ^ (lane & 7)) << 4))), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                       : "memory");
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {      // four rows a store
          const int r2 = r_at + i, t2 = (int)((uint32_t)r2 * ta.g_mul >> 16);   // r2 / G
          uint32_t w[4];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(stage + (uint32_t)((r2 & 31) * 128 + ((cc ^ (r2 & 7)) << 4))) : "memory");
          if (t2 < tpt && t_at + t2 < it.toks)
            *reinterpret_cast<uint4*>(out0 + 64 * h + (t2 * o_ts + (r2 - t2 * G) * o_hs)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
      }
      if (row_ok && a.lse)
        a.lse[(int64_t)(it.r_first + tok) * a.hq + it.kvh * G + r - ti * G] =
            !ok ? __uint_as_float(0x7fffffffu) : l == 0.f ? neg_inf() : (m + log2f(l)) * 0.6931471805599453f;
    }
    if constexpr (Mode == kPaPrefix) {         // a wait gave up: the parts of the run that were not handed out are NaN
      if (__any_sync(0xffffffffu, s_abort))
        while (part_at(it.unit, it)) {
          float* const slot = sh_slot(a.ws, a.n_groups, a.seqs, HD, it.slot);
          __stcg(reinterpret_cast<float2*>(slot + 256 * HD) + t * kTaRows + r, make_float2(0.f, __uint_as_float(0x7fffffffu)));
        }
    }
  }
  __syncthreads();
  // a wait gave up, in whichever warp: products and copies in flight end (bounded) before the space goes
  if (s_abort && warp == 9) ta_drain(&drained);
  if (s_abort && threadIdx.x == 0) {
    constexpr int kRing = F8 ? L::raws : kS;
    for (int i = max(0, s_filled - kRing); i < s_filled; ++i) {
      long long spins = 0;
      while (!mbar_test(F8 ? &raw_full[i % kR] : &kv_full[i % kS], (unsigned)((i / kRing) & 1)) && ++spins < (1LL << 20)) {
      }
    }
    long long spins = 0;
    while (s_qloads > 0 && !mbar_test(&q_full, (unsigned)((s_qloads - 1) & 1)) && ++spins < (1LL << 20)) {
    }
  }
  __syncthreads();
  if (warp == 11) {
    ta_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
  // a block's sums stay until its peer has read them
  if (ta.split > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int HD, bool F8, bool Hook, int Mode>
cudaError_t launch_ta_hook(const TaArgsOf<Mode>& ta, cudaStream_t st) {
  using L = TaLayout<HD, F8, Mode>;
  auto kern = pattn_tc_kernel<HD, F8, Hook, Mode>;
  return launch_rows_smem<Mode == kPaPrefix>(std::integral_constant<int, Mode * 1000 + HD * 4 + F8 * 2 + Hook>(), kern,
                                             dim3((unsigned)(ta.split * ta.items)), dim3(L::threads), L::smem, ta.split, st, ta);
}

template <int HD, bool F8, int Mode>
cudaError_t launch_ta(const TaArgsOf<Mode>& ta, cudaStream_t st) {
  return ta.a.give_up > 0 ? launch_ta_hook<HD, F8, true, Mode>(ta, st) : launch_ta_hook<HD, F8, false, Mode>(ta, st);
}
template <int Mode>
cudaError_t launch_ta_mode(const TaArgsOf<Mode>& ta, cudaStream_t st) {
  if (ta.a.f8) return ta.a.hd == 64 ? launch_ta<64, true, Mode>(ta, st) : launch_ta<128, true, Mode>(ta, st);
  return ta.a.hd == 64 ? launch_ta<64, false, Mode>(ta, st) : launch_ta<128, false, Mode>(ta, st);
}
// The arguments of a call, but for how its items are cut; false where no tensor map can be made.
template <int Mode>
bool ta_args(TaArgsOf<Mode>& ta, const PAttn& a) {
  ta.a = a;
  const int G = a.hq / a.hkv, ps = a.paged ? 1 << a.page_shift : kTaKeys;
  ta.tpt = kTaRows / G;
  ta.g_mul = (65536u + G - 1) / G;
  ta.box_rows = std::min(ps, Mode == kPaWindow && a.paged ? 64 : kTaKeys);   // (a window's first box may be mostly in front of it)
  auto maps = [&](TensorMap128& k, TensorMap128& v, int rows) {
    if (a.paged)
      return ta_map(k, a.k, a.hd, (int64_t)a.hkv * ps, a.pages, a.hd, a.page_stride, rows, 1, a.f8) &&
             ta_map(v, a.v, a.hd, (int64_t)a.hkv * ps, a.pages, a.hd, a.page_stride, rows, 1, a.f8);
    return ta_map(k, a.k, a.hd, a.hkv, a.tokens, a.k_hs, a.k_ts, 1, rows) &&
           ta_map(v, a.v, a.hd, a.hkv, a.tokens, a.v_hs, a.v_ts, 1, rows);
  };
  if constexpr (Mode == kPaWindow)
    if (!maps(ta.ks, ta.vs, 16)) return false;
  return ta_map(ta.qm, a.q, a.hd, a.hq, a.tokens, a.q_hs, a.q_ts, G, ta.tpt) && maps(ta.km, ta.vm, ta.box_rows);
}
// Items of a causal or windowed call.
template <int Mode>
cudaError_t launch_ta_items(const PAttn& a, int num_sms, cudaStream_t st) {
  TaArgsOf<Mode> ta{};
  if (!ta_args<Mode>(ta, a)) return cudaErrorInvalidValue;
  ta.pairs = (std::min(a.max_q, a.tokens) + 2 * ta.tpt - 1) / (2 * ta.tpt);
  // A block reads all the keys that its rows see, so blocks of one KV head
  // run together and share them in L2: as many heads at a time as give the
  // SMs four rounds of items.
  ta.chunk = std::max(1, std::min(a.hkv * a.seqs, (4 * num_sms + ta.pairs - 1) / ta.pairs));
  const int64_t items = (int64_t)a.hkv * a.seqs * ta.pairs;
  if (items > 0x1fffffffLL) return cudaErrorInvalidConfiguration;
  ta.items = (int)items;
  // items that can hold rows: no more than the tokens fill, and one ragged pair a sequence
  const int64_t most = a.hkv * std::min<int64_t>((int64_t)a.seqs * ta.pairs, a.tokens / (2 * ta.tpt) + a.seqs);
  // Two blocks an item where items leave half of the SMs idle, or where they
  // fill them less than once with walks of very different lengths (64 items of
  // 128 steps: 178 -> 99 us; 128 equal items of 32 steps: 53 us, and 67 split).
  int64_t max_keys = a.paged ? (int64_t)a.max_pages << a.page_shift : std::min(a.max_q, a.tokens);
  if (Mode == kPaWindow) max_keys = std::min(max_keys, (int64_t)a.window + a.sinks + 2 * ta.tpt + 2 * kTaKeys);
  const bool uneven = Mode == kPaCausal && (int64_t)a.seqs * a.max_q * 2 > 3LL * a.tokens;
  ta.split = most * (uneven ? 1 : 2) <= num_sms && max_keys >= 16 * kTaKeys ? 2 : 1;
  // new tokens few beside their contexts: a walk's length is its sequence's
  ta.by_length = Mode == kPaCausal && a.paged && a.seqs <= 32 && max_keys >= 2LL * a.max_q ? 1 : 0;
  // (Windows:) where blocks cover the items, each keeps to its own: one that starts early would take
  // items whose blocks find free SMs (136 items of 18 steps in a grid of 256: 65 -> 36 us).
  if constexpr (Mode == kPaWindow) ta.take = ta.split == 1 && most > num_sms;
  return launch_ta_mode<Mode>(ta, st);
}

}  // namespace

}  // namespace sv
