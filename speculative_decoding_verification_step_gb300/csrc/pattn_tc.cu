// Attention of many rows per KV head (a chunk of prompt tokens, a whole
// prompt) on the fifth-generation tensor cores.
//
// Past ~64 rows a key is worth more arithmetic than its bytes: 4 flops per
// element and row, so the products bound the time, and next to them the
// exponentials (one per 4 head_dim flops: at head_dim 128 the two are close).
// The kernel keeps the tensor pipe fed while the softmax of one tile runs
// behind the products of the other.
//
// Block = two tiles of 128 rows (tokens x the G query heads of one KV head)
// against the keys in steps of 128, over a ring of shared-memory tiles filled
// by tensor copies, one box per page (128-byte swizzle, two 64-dim halves).
//   warps 0-3, 4-7  softmax of tile 0, 1: a thread owns a row.  It reads its
//                   128 scores from tensor memory, takes the maximum without
//                   any exchange, writes p as bf16 over the scores and keeps
//                   the row sum in fp32.  The exponent reference is lazy: it
//                   moves only when a score exceeds it by 2^8, and only then
//                   O is rescaled in tensor memory;
//   warp 8          producer: page ids and tensor copies (K_0 V_0 K_1 V_1 ..);
//                   it zeroes V's rows past the length in the last step;
//   warp 9          issues the products, per step and tile
//                   O += P V (P from tensor memory, V as it lies, keys along
//                   K), then S = Q K^T of the next step over the same columns
//                   that P occupied: the tensor pipe runs in issue order;
//   warp 11         allocates and frees tensor memory.
// Tensor memory, 512 columns: S/P 2 x 128, O 2 x head_dim.
// Rows leave through the shared memory of their Q tile: a thread's row is
// staged there and the warp writes whole rows (a thread writing its own row,
// 16 bytes in each of 32 lines at a time, took 6000 clocks a tile, a fifth of
// a block's time at 4096 tokens).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "paged.h"

namespace sv {

namespace {

constexpr int kTaRows = 128;        // rows of a tile (MMA M)
constexpr int kTaKeys = 128;        // keys of a step
constexpr int kTaThreads = 384;
constexpr int kTaStages = 4;
constexpr long long kTaWaitLimit = 1LL << 24;
constexpr float kTaLazy = 8.f;
constexpr float kTaNone = -1e30f;

struct TaArgs {
  TensorMap128 qm, km, vm;
  PAttn a;
  int tpt;          // tokens of a tile: 128 / G
  uint32_t g_mul;   // ceil(2^16 / G): r * g_mul >> 16 = r / G for r < 128
  int pairs;        // row pairs of the longest sequence
  int chunk;        // (sequence, KV head) pairs in flight at a time
  int box_rows;     // key rows of a K / V box
};

template <int HD>
constexpr int ta_smem() { return 2 * kTaRows * HD * 2 + kTaStages * kTaKeys * HD * 2 + 1024; }

SV_DEV uint64_t ta_desc(uint32_t addr, uint32_t lbo) {   // 128-byte swizzle, 8-row groups 1024 bytes apart
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)lbo << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// kind::f16, fp32 accumulator, bf16 operands, M = 128; tb: B lies with its N
// dimension contiguous.
SV_DEV constexpr uint32_t ta_idesc(int n, int tb) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)tb << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kTaRows >> 4) << 24);
}
SV_DEV void ta_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
               " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
SV_DEV void ta_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
               " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
               ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
SV_DEV void ta_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               ::"r"(smem_u32(bar)) : "memory");
}
SV_DEV bool ta_elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(p));
  return p != 0;
}
SV_DEV void ta_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
SV_DEV void ta_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
SV_DEV void ta_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
SV_DEV void ta_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 32 consecutive columns of this thread's lane (not waited for).
SV_DEV void ta_ld32(uint32_t t, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
}
SV_DEV void ta_st16(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
SV_DEV void ta_st32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
SV_DEV float ta_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 values in one 64-bit register pair: one instruction for both.
SV_DEV uint64_t ta_pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
SV_DEV void ta_split(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
SV_DEV uint64_t ta_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
SV_DEV uint64_t ta_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
SV_DEV float ta_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Keeps what uses v[0 .. N-1] from being scheduled above this point.
template <int N>
SV_DEV void ta_pin(float* v) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
SV_DEV uint32_t ta_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
SV_DEV void ta_tma_3d(uint32_t dst, const void* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)) : "memory");
}
// Bounded wait; false (after raising the abort flag) when it gives up.
SV_DEV bool ta_wait(uint64_t* bar, unsigned parity, volatile int* abort) {
  long long spins = 0;
  while (!mbar_test(bar, parity)) {
    if (*abort || ++spins > kTaWaitLimit) {
      *abort = 1;
      return false;
    }
  }
  return true;
}

// Block i: chunks of `chunk` (sequence, KV head) pairs one after the other; in
// a chunk the row pairs from each sequence's last to its first, all its heads
// side by side.
template <int HD>
__global__ void __launch_bounds__(kTaThreads, 1) pattn_tc_kernel(const __grid_constant__ TaArgs ta) {
  constexpr int kHalf = HD / 64;                       // 64-dim halves of a row
  constexpr uint32_t kTile = kTaKeys * HD * 2;         // bytes of a Q, K or V tile
  extern __shared__ __align__(1024) unsigned char tsm[];
  __shared__ uint64_t q_full, kv_full[kTaStages], kv_empty[kTaStages], s_full[2], p_half[2], p_full[2], pv_done[2], v_fixed, drained;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ int s_filled;
  const PAttn& a = ta.a;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int per_chunk = ta.chunk * ta.pairs, chunk = (int)blockIdx.x / per_chunk, in_chunk = (int)blockIdx.x % per_chunk;
  const int width = min(ta.chunk, a.hkv * a.seqs - chunk * ta.chunk);
  const int item = chunk * ta.chunk + in_chunk % width, pair = ta.pairs - 1 - in_chunk / width;
  const int kvh = item % a.hkv, b = item / a.hkv;
  const int G = a.hq / a.hkv, tpt = ta.tpt;

  const int r_first = __ldg(a.cu + b);
  const int n = __ldg(a.cu + b + 1) - r_first;
  if (r_first < 0 || n <= 0 || n > a.tokens - r_first || (int64_t)n * G <= a.max_rows) return;
  const int toks = min(n, a.max_q);           // tokens that are computed
  const int tok0 = pair * 2 * tpt;
  if (tok0 >= toks) return;
  int keys = n;
  if (a.paged) {
    keys = __ldg(a.lens + b);
    const int64_t cap = (int64_t)a.max_pages << a.page_shift;
    keys = keys < 0 ? 0 : (int)min((int64_t)keys, cap);
  }
  const int first_pos = keys - n;
  const int ntile = tok0 + tpt < toks ? 2 : 1;
  // key steps of each tile: what its last token sees
  int steps[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = min(toks, tok0 + (t + 1) * tpt) - 1;
    const int see = min(keys, max(0, first_pos + last + 1));
    steps[t] = t < ntile ? (see + kTaKeys - 1) / kTaKeys : 0;
  }
  const int nst = max(steps[0], steps[1]);
  const int last_rows = keys - (nst - 1) * kTaKeys;    // valid keys of the last step (>= 128: all)

  const uint32_t base = (smem_u32(tsm) + 1023u) & ~1023u;
  const uint32_t q_at = base, kv_at = base + 2 * kTile;
  if (warp == 8 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&ta.qm)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&ta.km)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&ta.vm)) : "memory");
    mbar_init(&q_full, 1);
    mbar_init(&v_fixed, 1);
    mbar_init(&drained, 1);
    for (int s = 0; s < kTaStages; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_half[t], 4);        // one arrival per softmax warp
      mbar_init(&p_full[t], 4);
      mbar_init(&pv_done[t], 1);
    }
    s_abort = 0;
    s_filled = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (nst > 0) {   // Q is on its way while tensor memory is allocated
      mbar_arrive_expect_tx(&q_full, (unsigned)(ntile * kHalf * 128 * G * tpt));
      for (int t = 0; t < ntile; ++t)
        for (int h = 0; h < kHalf; ++h)
          ta_tma_3d(q_at + t * kTile + h * (kTile / kHalf), &ta.qm, h * 64, kvh * G, r_first + tok0 + t * tpt, &q_full);
    }
  }
  if (warp == 11) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  ta_fence_before();
  __syncthreads();
  ta_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  constexpr uint32_t o_at = 256;

  // registers: the softmax warps hold a row's 128 scores (2 x 216 + 56 <= 3 x 168)
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  if (warp == 8) {
    // ---- producer ----
    const int per = a.paged ? kTaKeys / ta.box_rows : 1;     // boxes of a step
    const int32_t* table = a.paged ? a.table + b * a.table_stride : nullptr;
    const int npages = a.paged ? (int)(((int64_t)keys + (1 << a.page_shift) - 1) >> a.page_shift) : 0;
    auto page_of = [&](int j) {   // lane i: page of box i of step j; -1 (zero rows) past the length
      const int64_t key = (int64_t)j * kTaKeys + lane * ta.box_rows;
      const int pg = (int)(key >> a.page_shift);
      return lane < per && j < nst && pg < npages ? __ldg(table + pg) : -1;
    };
    int next = a.paged ? page_of(0) : 0;
    bool live = true;
    for (int j = 0; j < nst && live; ++j) {
      const int page = next;
      if (a.paged) next = page_of(j + 1);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int i = 2 * j + kv, s = i % kTaStages;
        if (i >= kTaStages) live = live && ta_wait(&kv_empty[s], (unsigned)((i / kTaStages - 1) & 1), &s_abort);
        live = __all_sync(0xffffffffu, live);
        if (!live) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&kv_full[s], kTile);
          s_filled = i + 1;
        }
        __syncwarp();
        const void* map = kv ? &ta.vm : &ta.km;
        const uint32_t dst = kv_at + s * kTile;
        if (lane < per) {
          for (int h = 0; h < kHalf; ++h) {
            const uint32_t d = dst + h * (kTile / kHalf) + lane * ta.box_rows * 128;
            if (a.paged)
              ta_tma_3d(d, map, h * 64,
                        (kvh << a.page_shift) + (int)(((int64_t)j * kTaKeys + lane * ta.box_rows) & ((1 << a.page_shift) - 1)),
                        page, &kv_full[s]);
            else
              ta_tma_3d(d, map, h * 64, kvh, r_first + j * kTaKeys, &kv_full[s]);
          }
        }
      }
    }
    if (live && nst > 0 && last_rows < kTaKeys) {
      // V's rows past the length: p is zero there, but the slots may hold
      // anything.  (This warp has seen the entry's earlier fills consumed, so
      // its parity is the last fill's.)
      const int iv = 2 * nst - 1, s = iv % kTaStages;
      if (__all_sync(0xffffffffu, ta_wait(&kv_full[s], (unsigned)((iv / kTaStages) & 1), &s_abort))) {
        for (int h = 0; h < kHalf; ++h)
          for (int e = last_rows * 8 + lane; e < kTaKeys * 8; e += 32)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};"
                         ::"r"(kv_at + s * kTile + h * (kTile / kHalf) + e * 16), "r"(0) : "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_fixed);
      }
    }
  } else if (warp == 9) {
    // ---- products ----
    // The whole warp runs the control flow, so that descriptors and addresses
    // stay in uniform registers; one elected lane issues.
    if (nst > 0) {
      constexpr uint32_t id_s = ta_idesc(kTaKeys, 0), id_o = ta_idesc(HD, 1);
      auto wait = [&](uint64_t* bar, unsigned parity) {
        const bool got = __all_sync(0xffffffffu, ta_wait(bar, parity, &s_abort));
        ta_fence_after();
        return got;
      };
      // S_t = Q_t K^T of step j from ring entry 2 j
      auto score = [&](int t, int j) {
        const uint64_t qd = ta_desc(q_at + t * kTile, 1), kd = ta_desc(kv_at + (uint32_t)((2 * j) % kTaStages) * kTile, 1);
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
      // O_t += P_t V over half of step j's keys
      auto gather = [&](int t, int j, int half) {
        const uint64_t vd = ta_desc(kv_at + (uint32_t)((2 * j + 1) % kTaStages) * kTile, (kTile / kHalf) >> 4);
        if (ta_elect()) {
#pragma unroll
          for (int k4 = 0; k4 < kTaKeys / 32; ++k4) {
            const int ks = half * (kTaKeys / 32) + k4;
            ta_mma_ts(tmem + o_at + t * HD, tmem + t * 128 + ks * 8, vd + ks * 128, id_o, j > 0 || ks > 0);
          }
          if (half) ta_commit(&pv_done[t]);
        }
        __syncwarp();
      };
      // frees ring entry i once the products issued so far are done, where a later fill waits for it
      auto release = [&](int i) {
        if (i + kTaStages < 2 * nst && ta_elect()) ta_commit(&kv_empty[i % kTaStages]);
        __syncwarp();
      };
      bool ok = wait(&q_full, 0) && wait(&kv_full[0], 0);
      if (ok) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (steps[t] > 0) score(t, 0);
        release(0);
      }
      for (int j = 0; ok && j < nst; ++j) {
        const int iv = 2 * j + 1, ik = 2 * j + 2;
        ok = wait(&kv_full[iv % kTaStages], (unsigned)((iv / kTaStages) & 1));
        if (ok && j == nst - 1 && last_rows < kTaKeys) ok = wait(&v_fixed, 0);
        bool have_k = false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          // the first 64 keys' products run while the other exponentials are taken
          if (ok && j < steps[t]) {
            ok = wait(&p_half[t], (unsigned)(j & 1));
            if (ok) {
              gather(t, j, 0);
              ok = wait(&p_full[t], (unsigned)(j & 1));
              if (ok) gather(t, j, 1);
            }
          }
          if (ok && j + 1 < steps[t]) {
            if (!have_k) ok = wait(&kv_full[ik % kTaStages], (unsigned)((ik / kTaStages) & 1));
            have_k = true;
            if (ok) score(t, j + 1);
          }
        }
        if (!ok) break;
        release(iv);
        release(ik);
      }
      if (!ok) {   // the products issued so far end before the space goes
        if (ta_elect()) ta_commit(&drained);
        __syncwarp();
        long long spins = 0;
        while (!mbar_test(&drained, 0) && ++spins < (1LL << 20)) {
        }
      }
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ---- softmax of tile t: one row per thread ----
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;
    const int ti = r / G, tok = tok0 + t * tpt + ti;
    const bool row_ok = t < ntile && ti < tpt && tok < toks;
    const int seen = row_ok ? min(keys, max(0, first_pos + tok + 1)) : 0;
    const int tile_all = min(keys, max(0, first_pos + tok0 + t * tpt + 1));   // keys that every row sees
    const uint32_t row = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + row + t * 128, out_at = tmem + row + o_at + t * HD;
    const float scale = a.scale_log2;
    float m = kTaNone, l = 0.f;
    bool ok = true;
    const int my = t < ntile ? steps[t] : 0;
    for (int j = 0; j < my; ++j) {
      ok = ta_wait(&s_full[t], (unsigned)(j & 1), &s_abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ta_fence_after();
      float s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) ta_ld32(s_at + 32 * c, s + 32 * c);
      ta_wait_ld();
      const int key0 = j * kTaKeys;
      if (key0 + kTaKeys > tile_all) {
        const int lim = seen - key0;
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= lim) s[c] = neg_inf();
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
      ta_pin<128>(s);                        // the maximum first, then the exponentials
      const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * scale;
      const bool move = top > m + kTaLazy;
      if (__any_sync(0xffffffffu, move)) {
        const float to = move ? top : m, f = ta_exp2(m - to);
        m = to;
        l *= f;
        if (j > 0) {
          ok = ta_wait(&pv_done[t], (unsigned)((j - 1) & 1), &s_abort);
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
          // the second half's exponentials stay behind the first's arrival
          // (moved up among them they hold it back: 2440 clocks a step for 1770)
          if (q == 1) ta_pin<64>(s + 64);
        }
      }
      float a0, a1;
      ta_split(ta_add2(sum0, sum1), a0, a1);
      l += a0 + a1;
    }
    if (ok && my > 0) {
      ok = ta_wait(&pv_done[t], (unsigned)((my - 1) & 1), &s_abort);
      ok = __all_sync(0xffffffffu, ok);
      ta_fence_after();
    }
    // rows out; a wait that gave up leaves NaN, not a wrong number
    const float inv = !ok ? __uint_as_float(0x7fffffffu) : l == 0.f ? 0.f : 1.f / l;
    const int64_t at = r_first + tok;
    const int h = kvh * G + r - ti * G;
    constexpr int kChunks = HD / 8;                      // 16-byte chunks of a row
    const uint32_t stage = q_at + t * kTile + (uint32_t)((warp & 3) * 32 * HD * 2);
    if (t < ntile) {
      float o[HD];
      if (ok && my > 0) {
#pragma unroll
        for (int c = 0; c < HD; c += 32) ta_ld32(out_at + c, o + c);
        ta_wait_ld();
      } else {
#pragma unroll
        for (int c = 0; c < HD; ++c) o[c] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = ta_pack(o[8 * c + 2 * i] * inv, o[8 * c + 2 * i + 1] * inv);
        }
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                     ::"r"(stage + (uint32_t)(lane * HD * 2 + ((c ^ (lane & 7)) << 4))), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                     : "memory");
      }
      __syncwarp();
      constexpr int kStep = 32 / kChunks;                // rows of one store
      const int cc = lane % kChunks, r_at = (warp & 3) * 32 + lane / kChunks, t_at = tok0 + t * tpt;
      bf16* const out0 = (bf16*)a.out + (int64_t)(r_first + t_at) * a.o_ts + (int64_t)(kvh * G) * a.o_hs + cc * 8;
#pragma unroll 4
      for (int i = 0; i < 32; i += kStep) {
        const int r2 = r_at + i, t2 = (int)((uint32_t)r2 * ta.g_mul >> 16);   // r2 / G
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(stage + (uint32_t)((r2 & 31) * HD * 2 + ((cc ^ (r2 & 7)) << 4))) : "memory");
        if (t2 < tpt && t_at + t2 < toks)
          *reinterpret_cast<uint4*>(out0 + t2 * a.o_ts + (r2 - t2 * G) * a.o_hs) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if (row_ok && a.lse)
      a.lse[at * a.hq + h] = !ok ? __uint_as_float(0x7fffffffu) : l == 0.f ? neg_inf() : (m + log2f(l)) * 0.6931471805599453f;
  }
  __syncthreads();
  if (s_abort && threadIdx.x == 0) {
    // a wait gave up: copies in flight land (bounded) before the space goes
    for (int i = max(0, s_filled - kTaStages); i < s_filled; ++i) {
      long long spins = 0;
      while (!mbar_test(&kv_full[i % kTaStages], (unsigned)((i / kTaStages) & 1)) && ++spins < (1LL << 20)) {
      }
    }
    long long spins = 0;
    while (nst > 0 && !mbar_test(&q_full, 0) && ++spins < (1LL << 20)) {
    }
  }
  __syncthreads();
  if (warp == 11) {
    ta_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

PFN_cuTensorMapEncodeTiled_v12000 ta_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}
// [d2][d1][hd] bf16 with strides s1, s2 (elements), boxes of 64 x b1 x b2.
bool ta_map(TensorMap128& m, const void* base, int hd, int64_t d1, int64_t d2, int64_t s1, int64_t s2, int b1, int b2) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = ta_encoder();
  if (!enc) return false;
  // the stride of a dimension of one element is never used, but has to be valid
  if (d1 == 1) s1 = hd;
  if (d2 == 1) s2 = hd;
  cuuint64_t dims[3] = {(cuuint64_t)hd, (cuuint64_t)d1, (cuuint64_t)d2};
  cuuint64_t strides[2] = {(cuuint64_t)s1 * 2, (cuuint64_t)s2 * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)b1, (cuuint32_t)b2};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(reinterpret_cast<CUtensorMap*>(&m), CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
             strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD>
cudaError_t launch_ta(const TaArgs& ta, cudaStream_t st) {
  auto kern = pattn_tc_kernel<HD>;
  const int64_t blocks = (int64_t)ta.a.hkv * ta.a.seqs * ta.pairs;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_rows_smem(std::integral_constant<int, HD>(), kern, dim3((unsigned)blocks), dim3(kTaThreads), ta_smem<HD>(), 1,
                          st, ta);
}

}  // namespace

bool pattn_tc_supported(const PAttn& a) {
  const int G = a.hq / a.hkv;
  if ((a.hd != 64 && a.hd != 128) || a.f8 || G > kTaRows) return false;
  // tensor maps take positive strides only (a broadcast head has stride 0)
  auto pos = [](int64_t s, int64_t d) { return d == 1 || (s > 0 && s < (1LL << 38)); };
  if (!pos(a.q_ts, a.tokens) || !pos(a.q_hs, a.hq)) return false;
  if (!a.paged)
    return pos(a.k_ts, a.tokens) && pos(a.k_hs, a.hkv) && pos(a.v_ts, a.tokens) && pos(a.v_hs, a.hkv);
  return pos(a.page_stride, a.pages) && (int64_t)a.hkv << a.page_shift <= 0x7fffffffLL;
}

cudaError_t launch_pattn_tc(const PAttn& a, int num_sms, cudaStream_t st) {
  TaArgs ta{};
  ta.a = a;
  const int G = a.hq / a.hkv;
  ta.tpt = kTaRows / G;
  ta.g_mul = (65536u + G - 1) / G;
  ta.pairs = (std::min(a.max_q, a.tokens) + 2 * ta.tpt - 1) / (2 * ta.tpt);
  // A block reads all the keys that its rows see, so blocks of one KV head
  // run together and share them in L2: as many heads at a time as give the
  // SMs four rounds of blocks (enough for their unequal lengths to even out).
  ta.chunk = std::max(1, std::min(a.hkv * a.seqs, (4 * num_sms + ta.pairs - 1) / ta.pairs));
  const int ps = a.paged ? 1 << a.page_shift : kTaKeys;
  ta.box_rows = std::min(ps, kTaKeys);
  bool ok = ta_map(ta.qm, a.q, a.hd, a.hq, a.tokens, a.q_hs, a.q_ts, G, ta.tpt);
  if (a.paged) {
    ok = ok && ta_map(ta.km, a.k, a.hd, (int64_t)a.hkv * ps, a.pages, a.hd, a.page_stride, ta.box_rows, 1) &&
         ta_map(ta.vm, a.v, a.hd, (int64_t)a.hkv * ps, a.pages, a.hd, a.page_stride, ta.box_rows, 1);
  } else {
    ok = ok && ta_map(ta.km, a.k, a.hd, a.hkv, a.tokens, a.k_hs, a.k_ts, 1, kTaKeys) &&
         ta_map(ta.vm, a.v, a.hd, a.hkv, a.tokens, a.v_hs, a.v_ts, 1, kTaKeys);
  }
  if (!ok) return cudaErrorInvalidValue;
  return a.hd == 64 ? launch_ta<64>(ta, st) : launch_ta<128>(ta, st);
}

}  // namespace sv
