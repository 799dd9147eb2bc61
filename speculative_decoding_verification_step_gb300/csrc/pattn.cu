// Attention of a sequence's newest tokens over its keys, for few rows per KV
// head: a verify step's (K + 1) x G, one decoded token's G, a short prompt.
//
// With R rows per tile a key costs 4 R head_dim flops against its
// 2 head_dim elements of K and V: below ~64 rows the cache's bytes bound the
// time, so a key is read once per tile, straight from its page into shared
// memory, and everything else is arranged around keeping those reads going.
//
// Block = (row tile of 8 NT rows, KV head, share of the keys), four warps.
// The keys are walked in 16-key steps, step s on warp s mod 4.  Every warp
// keeps its own ring of steps filled by 16-byte asynchronous copies (no block
// barrier in the walk), swizzled by row so that ldmatrix finds its eight rows
// in distinct banks; rows past the length are filled with zeros, so whatever
// those slots hold cannot reach a product.
//   S^T = K Q^T and O^T += V^T P^T: the keys (dims) are the 16-row side of the
//   MMAs and the query rows the 8-column side, so that 4 or 24 rows waste
//   little (24 rows: 3 column tiles, where rows on the 16-row side took 4),
//   and the accumulators of 24 rows leave room for three blocks on an SM.
//   P^T turns from an accumulator into an operand by transposing 8 x 8 blocks
//   within the warp (movmatrix).  Q waits in shared memory in operand order.
//   Online softmax with a lazy reference: a row's exponent reference only
//   moves when a score exceeds it by more than 2^8, so the usual step has no
//   shuffles and no rescaling of O; p <= 256 and the sums stay in fp32.
//   Probabilities are rounded to bf16 for P V (half a step, 2^-9 of each on
//   average, of random sign: the size of the output's own rounding); the row
//   sum keeps them in fp32.
// 8-bit keys become f16, which holds every code exactly, two codes an
// instruction (the bit moves that make a bf16 of a code cost two and a half
// times as much, measured, and an e4m3 mma.sync is itself emulated here: 37
// clocks of an SM partition against 8).  Q rows are f16 too, scaled by a power
// of two to just below 2^15: exact down to 2^-29 of the row's largest.  The
// rows' powers of two meet the scores in fp32.  Values go on from f16 to bf16,
// also exact, and their powers of two meet the probabilities before the rounding
// to bf16: its range holds p * 2^e of every row at once, whatever other rows and
// queries of the tile need.  (Products in f16 against a shared reference exponent
// lost small rows beside large ones; they took 4% less time at 4 rows, 6% at 12
// and 2% at 24.  Leaving them for bf16 only once rows lie far apart cost as much in
// choices as the conversions do.)
// The share of the keys: a cluster of up to 8 blocks splits one tile's keys
// and merges through distributed shared memory in a fixed order (no scratch
// memory, no second launch, no atomics): blocks merge their four warps, then
// block j of the cluster finishes the rows j, j + C, ...
// Bound: by the copies for a few rows (64 sequences x 4096 keys of 8 heads of
// 128, 16-bit, one token each: 129 us, 91% of a copy's rate; 16 x 16384 of 64
// dims 66 us, 89%; 64 x 4096 8-bit of 128 dims 86 us, 71%), by the latencies of a
// step's instructions (three warps a partition) for more: 24 rows of 64 x 4096
// 164 us (75%), 8-bit 153 us (40%), which is why long 8-bit contexts go to tensor
// memory.  8-bit rows of 64 dims hold half the bytes for the same conversions a
// step: 64 x 4096 65 us of one token (49%), 108 us of 24 rows (29%).  One sequence of 512 keys and 24 rows takes 9 us, most of it the
// start, one walk of a few steps and two merges.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "common.cuh"
#include "paged.h"

namespace sv {

std::atomic<int> g_attn_give_up{0};

namespace {

constexpr int kPaThreads = 128;
constexpr int kPaWarps = 4;
constexpr int kPaStep = 16;          // keys of a step
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPaLazy = 8.f;       // exponent reference moves past 2^8
constexpr float kPaNone = -1e30f;    // reference of a row that has seen nothing

template <int HD, bool F8, int NT>
struct PaLayout {
  static constexpr int row = HD * (F8 ? 1 : 2);      // bytes of a key row
  static constexpr int chunks = row / 16;
  static constexpr int tile = kPaStep * row;         // K or V of a step
  static constexpr int stage = 2 * tile + (F8 ? 32 : 0);
  static constexpr int q_bytes = NT * 8 * HD * 2;    // Q in operand order: 16 bytes a lane hold two k slices
  // Blocks on an SM: as many as the accumulators allow (NT = 4: 128 of them),
  // more where steps are small and rows few, so that their copies leave room
  // (64 x 4096 keys of one token, 8-bit head dim 128: 3 blocks 100 us, 4 87, 5 86;
  // 16-bit head dim 64: 75, 70, 68; 8-bit head dim 64, whose ring is full with 4:
  // 65, 65, 67).
  static constexpr int blocks = NT == 4 && HD >= 128 ? 2 : NT > 2 || stage >= 5000 ? 3 : NT == 1 && stage > 3000 ? 5 : 4;
  static constexpr int room = (blocks == 2 ? 112 : blocks == 3 ? 74 : blocks == 4 ? 55 : 44) * 1024 - q_bytes;
  static constexpr int fit = room / (kPaWarps * stage);
  static constexpr int depth = fit > 6 ? 6 : fit;
  static_assert(depth >= 2, "the ring holds the step in use and the next");
  static constexpr int ring = kPaWarps * depth * stage;
  static constexpr int ld = HD + 4;                  // merge rows: odd multiples of 4 banks apart
  static constexpr int merge = kPaWarps * NT * 8 * ld * 4;
  static constexpr int smem = q_bytes + (ring > merge ? ring : merge);
  // Byte offset of 16-byte chunk c of row r: rows of less than 128 bytes
  // share a 128-byte line, so the row bits that vary over eight consecutive
  // lines are the ones to mix in.
  static SV_DEV int at(int r, int c) {
    constexpr int m = chunks >= 8 ? 7 : chunks - 1;
    const int x = chunks >= 8 ? r : r / (8 / chunks);
    return r * row + ((c ^ (x & m)) << 4);
  }
};

SV_DEV void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
SV_DEV void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// 8 x 8 block of 16-bit elements, two per lane, transposed within the warp.
SV_DEV uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool F16>
SV_DEV void pa_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    mma_bf16_16816_acc(d, a[0], a[1], a[2], a[3], b0, b1);
}
// Four codes: the two of the lower half, and of the upper, as f16 pairs.
SV_DEV void f8_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}
SV_DEV float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
SV_DEV uint32_t pa_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// An f16 pair as a bf16 pair (exact for what codes become).
SV_DEV uint32_t f16_to_bf16(uint32_t h) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pa_pack(v.x, v.y);
}

SV_DEV void cluster_arrive_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
SV_DEV uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
SV_DEV float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
SV_DEV float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// Block x: tile (x / C) % tpq of sequence (x / C) / tpq, share x % C of its
// keys; y: KV head.
template <int HD, bool F8, int NT>
__global__ void __launch_bounds__(kPaThreads, PaLayout<HD, F8, NT>::blocks)
    pattn_kernel(const __grid_constant__ PAttn a, int tpq, int C) {
  using L = PaLayout<HD, F8, NT>;
  constexpr int kRows = NT * 8, kMt = HD / 16, D = L::depth;
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ float s_m[kPaWarps][kRows], s_l[kPaWarps][kRows];
  __shared__ float s_cm[kRows], s_cl[kRows], s_qf[kRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
  const int share = blockIdx.x % C, item = blockIdx.x / C;
  const int b = item / tpq, tile = item - b * tpq, kvh = blockIdx.y;
  const int G = a.hq / a.hkv;

  // the sequence's rows and keys (every block of a cluster sees the same)
  const int r_first = __ldg(a.cu + b);
  const int n = __ldg(a.cu + b + 1) - r_first;
  int keys = a.paged ? __ldg(a.lens + b) : n;
  if (r_first < 0 || n <= 0 || n > a.tokens - r_first) return;
  if (a.paged) keys = keys < 0 ? 0 : (int)min((int64_t)keys, (int64_t)a.max_pages << a.page_shift);
  const int rows = min(n, a.max_q) * G;       // rows that are computed
  const int row0 = tile * kRows;
  if (row0 >= rows) return;
  const int first_pos = keys - n;             // position of the sequence's row 0
  const int last_row = min(rows, row0 + kRows) - 1;
  const int see_max = min(keys, max(0, first_pos + last_row / G + 1));   // keys that any row of the tile sees
  const int see_all = first_pos + row0 / G + 1;                          // keys that every row sees

  // this block's steps, and the warp's: s0 + 4 j
  const int steps = (see_max + kPaStep - 1) / kPaStep;
  const int s_beg = (int)((int64_t)steps * share / C), s_end = (int)((int64_t)steps * (share + 1) / C);
  const int s0 = s_beg + warp;
  const int nj = s_end > s0 ? (s_end - s0 + kPaWarps - 1) / kPaWarps : 0;
  unsigned char* ring = sm + L::q_bytes + (size_t)warp * D * L::stage;
  const uint32_t ring_u = smem_u32(ring);
  const int32_t* table = a.paged ? a.table + b * a.table_stride : nullptr;
  const int ps_mask = (1 << a.page_shift) - 1;
  int pid = 0;   // lane i: page of the warp's step (j & ~31) + i (V's copies follow K's of the same step)

  // Copies of K (v = 0) or V (v = 1) of the warp's step j into its ring slot;
  // one group each, so that the scores do not wait for V and K's slot is
  // filled again as soon as they are done.
  const uint32_t lane_at = (uint32_t)L::at(lane / L::chunks, lane % L::chunks);
  auto issue = [&](int j, int v) {
    if (a.paged && !v && (j & 31) == 0) {
      const int64_t key = (int64_t)(s0 + kPaWarps * (j + lane)) * kPaStep;
      pid = j + lane < nj ? __ldg(table + (key >> a.page_shift)) : -1;
    }
    if (j < nj) {
      const int key0 = (s0 + kPaWarps * j) * kPaStep;
      int valid = min(kPaStep, keys - key0);
      const unsigned char* p;
      const uint8_t* sp = nullptr;
      if (a.paged) {
        const int page = __shfl_sync(0xffffffffu, pid, j & 31);
        const bool in = page >= 0 && page < a.pages;
        if (!in) valid = 0;
        const int64_t row = ((int64_t)kvh << a.page_shift) + (key0 & ps_mask);
        const int64_t pg = in ? page : 0;
        p = (const unsigned char*)(v ? a.v : a.k) + (pg * a.page_stride + row * HD) * (F8 ? 1 : 2);
        if constexpr (F8) sp = (v ? a.vs : a.ks) + pg * a.scale_stride + row;
      } else {
        p = (const unsigned char*)((const bf16*)(v ? a.v : a.k) + (int64_t)(r_first + key0) * (v ? a.v_ts : a.k_ts) +
                                   (int64_t)kvh * (v ? a.v_hs : a.k_hs));
      }
      const uint32_t slot = (uint32_t)((j % D) * L::stage + v * L::tile);
      if (a.paged && valid == kPaStep) {      // sixteen rows of a page lie one after the other
        p += lane * 16;
#pragma unroll
        for (int i = 0; i < kPaStep * L::chunks / 32; ++i) {
          // row i * per + lane / chunks: its swizzle bits are the lane's,
          // changed by those of i * per (shorter rows: eight rows or more
          // later the pattern repeats)
          constexpr int per = 32 / L::chunks;
          const uint32_t d = lane_at ^ (uint32_t)(per >= 8 ? 0 : ((i * per) & 7) << 4);
          cp_async16(ring + slot + d + i * 512, p + i * 512, true);
        }
      } else {
        const int64_t rs = a.paged ? L::row : (v ? a.v_ts : a.k_ts) * 2;
#pragma unroll
        for (int i = 0; i < kPaStep * L::chunks / 32; ++i) {
          const int e = i * 32 + lane, r = e / L::chunks, c = e % L::chunks;
          const bool in = r < valid;
          // rows past the length are not read: the source stays on row 0
          cp_async16(ring + slot + L::at(r, c), p + (in ? r : 0) * rs + c * 16, in);
        }
      }
      if constexpr (F8) {
        if (lane == 0) cp_async16(ring + (j % D) * L::stage + 2 * L::tile + 16 * v, sp, valid > 0);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int j = 0; j < D; ++j) {
    issue(j, 0);
    issue(j, 1);
  }

  // Q into shared memory as B operands, [slice pair][column tile][lane] of 16
  // bytes (two 16-element k slices of two words).  A lane's words hold
  // elements 2 q, 2 q + 1 and 8 more; with 8-bit keys, whose four neighbours
  // come in one word, elements 4 q .. 4 q + 3.
  for (int r = warp; r < kRows; r += kPaWarps) {
    const int R = row0 + r, t = R / G;
    const bool ok = R < rows;
    constexpr int kPer = HD / 32;             // elements of a lane: kPer lane .. + kPer - 1
    const int k = kPer * lane;
    const bf16* qr = (const bf16*)a.q + (int64_t)(r_first + (ok ? t : 0)) * a.q_ts +
                     (int64_t)(kvh * G + (ok ? R - t * G : 0)) * a.q_hs + k;
    float x[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = ok ? __bfloat162float(qr[i]) : 0.f;
    if constexpr (F8) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      // 2^e: the row's largest lands in [2^14, 2^15); a row that is not finite scores NaN
      const bool bad = m >= 0x7f800000u;
      const int e = m == 0 || bad ? 0 : max((int)(m >> 23) - 127 - 14, -100);
      const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int i = 0; i < kPer; ++i) x[i] = bad ? 0.f : x[i] * f;
      if (lane == 0)
        s_qf[r] = bad ? __uint_as_float(0x7fffffffu) : fmaxf(__uint_as_float((uint32_t)(127 + e) << 23) * a.scale_log2, 1.2e-38f);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int kk = k + i, sl = kk >> 4, in = kk & 15;
      const int quad = F8 ? in >> 2 : (in & 7) >> 1, word = F8 ? (in >> 1) & 1 : in >> 3;
      unsigned char* d = sm + (((sl >> 1) * NT + (r >> 3)) * 32 + (r & 7) * 4 + quad) * 16 + (sl & 1) * 8 + word * 4 + (in & 1) * 2;
      if constexpr (F8) *reinterpret_cast<__half*>(d) = __float2half_rn(x[i]);
      else *reinterpret_cast<bf16*>(d) = __float2bfloat16_rn(x[i]);
    }
  }
  __syncthreads();
  int seen[NT][2];                            // the lane's rows: 8 nt + 2 q4, + 1
  float qf[NT][2];                            // scores to units of log2
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = nt * 8 + 2 * q4 + e, R = row0 + r;
      seen[nt][e] = R < rows ? min(keys, first_pos + R / G + 1) : 0;
      qf[nt][e] = F8 ? s_qf[r] : a.scale_log2;
    }

  float o[kMt][NT][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < kMt; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][nt][e] = 0.f;
    m[nt][0] = m[nt][1] = kPaNone;
    l[nt][0] = l[nt][1] = 0.f;
  }

  const int lr = lane & 7, l8 = (lane >> 3) & 1, l16 = lane >> 4;
  const uint4* qs = reinterpret_cast<const uint4*>(sm) + lane;
  for (int j = 0; j < nj; ++j) {
    cp_async_wait<2 * D - 1>();
    __syncwarp();
    const int key0 = (s0 + kPaWarps * j) * kPaStep;
    const uint32_t kt = ring_u + (uint32_t)((j % D) * L::stage), vt = kt + L::tile;
    // scores: element e of column tile nt is key key0 + g + 8 (e / 2), row 8 nt + 2 q4 + (e & 1)
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
    for (int sl = 0; sl < kMt; sl += 2) {
      uint32_t ka[2][4];                      // keys 0-7, 8-15 of a slice's first 8 elements, then of its last
      if constexpr (F8) {
        uint32_t w[4];                        // keys 0-7, 8-15 of chunk sl, then of sl + 1
        ldsm4(w, kt + L::at(lr + 8 * l8, sl + l16));
#pragma unroll
        for (int x = 0; x < 4; ++x) f8_to_f16(w[x], ka[x >> 1][x & 1], ka[x >> 1][2 + (x & 1)]);
      } else {
        ldsm4(ka[0], kt + L::at(lr + 8 * l8, 2 * sl + l16));
        ldsm4(ka[1], kt + L::at(lr + 8 * l8, 2 * sl + 2 + l16));
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 w = qs[((sl / 2) * NT + nt) * 32];
        pa_mma<F8>(s[nt], ka[0], w.x, w.y);
        pa_mma<F8>(s[nt], ka[1], w.z, w.w);
      }
    }
    bool move = false;
    if constexpr (F8) {
      const unsigned char* sc = ring + (j % D) * L::stage + 2 * L::tile;
      const float k0 = row_power(sc[g]), k1 = row_power(sc[g + 8]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] *= e < 2 ? k0 : k1;
    }
    __syncwarp();
    issue(j + D, 0);
    const bool edge = key0 + kPaStep > see_all;   // some row does not see all of the step
    if (edge) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key0 + g + 8 * (e >> 1) >= seen[nt][e & 1]) s[nt][e] = neg_inf();
    }
    // exponents against the references
    float x[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[nt][e] = fmaf(s[nt][e], qf[nt][e & 1], -m[nt][e & 1]);
      move |= fmaxf(fmaxf(x[nt][0], x[nt][1]), fmaxf(x[nt][2], x[nt][3])) > kPaLazy;
    }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = fmaxf(s[nt][e], s[nt][e + 2]) * qf[nt][e];
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
          t = fmaxf(t, m[nt][e]);
          const float f = exp2_fast(m[nt][e] - t);
          m[nt][e] = t;
          l[nt][e] *= f;
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt) {
            o[mt][nt][e] *= f;
            o[mt][nt][e + 2] *= f;
          }
          x[nt][e] = fmaf(s[nt][e], qf[nt][e], -t);
          x[nt][e + 2] = fmaf(s[nt][e + 2], qf[nt][e], -t);
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[nt][e] = exp2_fast(x[nt][e]);
      l[nt][0] += x[nt][0] + x[nt][2];
      l[nt][1] += x[nt][1] + x[nt][3];
    }
    cp_async_wait<2 * D - 1>();
    __syncwarp();
    uint32_t pb[NT][2];
    if constexpr (F8) {
      const unsigned char* sc = ring + (j % D) * L::stage + 2 * L::tile + 16;
      const float vs[2] = {row_power(sc[g]), row_power(sc[g + 8])};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = x[nt][e] * vs[e >> 1];
        if (edge) {                           // a row that does not see a NaN key or its huge scale takes nothing of it
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (x[nt][e] == 0.f) p[e] = 0.f;
        }
        pb[nt][0] = transpose8(pa_pack(p[0], p[1]));
        pb[nt][1] = transpose8(pa_pack(p[2], p[3]));
      }
#pragma unroll
      for (int c = 0; c < kMt; c += 2) {      // chunks of 16 dims: row g is dim 2 g, row g + 8 dim 2 g + 1
        uint32_t w[4];                        // keys 0-7, 8-15 of chunk c, then of c + 1
        ldsm4t(w, vt + L::at(lr + 8 * l8, c + l16));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t va[4];                     // two dims of two keys a word: dims apart, keys together
          f8_to_f16(__byte_perm(w[2 * h], 0, 0x3120), va[0], va[1]);
          f8_to_f16(__byte_perm(w[2 * h + 1], 0, 0x3120), va[2], va[3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) va[i] = f16_to_bf16(va[i]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) pa_mma<false>(o[c + h][nt], va, pb[nt][0], pb[nt][1]);
        }
      }
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        pb[nt][0] = transpose8(pa_pack(x[nt][0], x[nt][1]));
        pb[nt][1] = transpose8(pa_pack(x[nt][2], x[nt][3]));
      }
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) {
        uint32_t w[4];                        // keys 0-7 of dims 0-7, 8-15; keys 8-15 of the same
        ldsm4t(w, vt + L::at(lr + 8 * l16, 2 * mt + l8));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) pa_mma<false>(o[mt][nt], w, pb[nt][0], pb[nt][1]);
      }
    }
    __syncwarp();
    issue(j + D, 1);
  }
  cp_async_wait<0>();
  __syncthreads();   // the rings become the merge area

  // ---- merge of the four warps: [warp][row][ld] ----
  float* part = reinterpret_cast<float*>(sm + L::q_bytes);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float t = l[nt][e];
      t += __shfl_xor_sync(0xffffffffu, t, 4);
      t += __shfl_xor_sync(0xffffffffu, t, 8);
      t += __shfl_xor_sync(0xffffffffu, t, 16);
      const int r = nt * 8 + 2 * q4 + e;
      if (g == 0) {
        s_m[warp][r] = m[nt][e];
        s_l[warp][r] = t;
      }
      float* d = part + ((size_t)warp * kRows + r) * L::ld;
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) {
        if constexpr (F8) {
          *reinterpret_cast<float2*>(d + mt * 16 + 2 * g) = make_float2(o[mt][nt][e], o[mt][nt][e + 2]);
        } else {
          d[mt * 16 + g] = o[mt][nt][e];
          d[mt * 16 + g + 8] = o[mt][nt][e + 2];
        }
      }
    }
  __syncthreads();
  constexpr int kLpr = HD / 4;                 // lanes of a row, four dims each
  const int col = (tid % kLpr) * 4;
  auto write_row = [&](int r, float4 x, float mm, float ll) {
    const int R = row0 + r, t = R / G, h = kvh * G + R - t * G;
    const float f = ll > 0.f || !(ll == ll) ? 1.f / ll : 0.f;
    bf16* d = (bf16*)a.out + (int64_t)(r_first + t) * a.o_ts + (int64_t)h * a.o_hs + col;
    *reinterpret_cast<uint2*>(d) = make_uint2(pa_pack(x.x * f, x.y * f), pa_pack(x.z * f, x.w * f));
    if (a.lse && col == 0)
      a.lse[(int64_t)(r_first + t) * a.hq + h] = ll == 0.f ? neg_inf() : (mm + log2f(ll)) * 0.6931471805599453f;
  };
  const int live = min(kRows, rows - row0);
  for (int r = tid / kLpr; r < live; r += kPaThreads / kLpr) {
    float mm = kPaNone, ll = 0.f;
#pragma unroll
    for (int w = 0; w < kPaWarps; ++w) mm = fmaxf(mm, s_m[w][r]);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kPaWarps; ++w) {
      const float f = exp2_fast(s_m[w][r] - mm);
      const float4 y = *reinterpret_cast<const float4*>(part + ((size_t)w * kRows + r) * L::ld + col);
      ll += s_l[w][r] * f;
      x.x += y.x * f; x.y += y.y * f; x.z += y.z * f; x.w += y.w * f;
    }
    if (C == 1) {
      write_row(r, x, mm, ll);
    } else {
      *reinterpret_cast<float4*>(part + (size_t)r * L::ld + col) = x;   // warp 0's slot of this element, read above
      if (col == 0) {
        s_cm[r] = mm;
        s_cl[r] = ll;
      }
    }
  }
  if (C == 1) return;
  // ---- merge of the cluster's blocks, in block order ----
  cluster_arrive_wait();
  const uint32_t pu = smem_u32(part), mu = smem_u32(s_cm), lu = smem_u32(s_cl);
  for (int r = share + C * (tid / kLpr); r < live; r += C * (kPaThreads / kLpr)) {
    float mm = kPaNone, ll = 0.f;
    for (int c = 0; c < C; ++c) mm = fmaxf(mm, ld_cluster_f32(cluster_map(mu + 4 * r, c)));
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = 0; c < C; ++c) {
      const float f = exp2_fast(ld_cluster_f32(cluster_map(mu + 4 * r, c)) - mm);
      const float4 y = ld_cluster_f32x4(cluster_map(pu + (uint32_t)(r * L::ld + col) * 4, c));
      ll += ld_cluster_f32(cluster_map(lu + 4 * r, c)) * f;
      x.x += y.x * f; x.y += y.y * f; x.z += y.z * f; x.w += y.w * f;
    }
    write_row(r, x, mm, ll);
  }
  cluster_arrive_wait();   // a block's memory stays until its peers have read it
}

template <int HD, bool F8, int NT>
cudaError_t launch_pa(const PAttn& a, int64_t rows, int tpq, int num_sms, cudaStream_t st) {
  using L = PaLayout<HD, F8, NT>;
  auto kern = pattn_kernel<HD, F8, NT>;
  const int64_t items = (int64_t)a.seqs * tpq;
  // Blocks of a cluster: what the GPU holds at once, one wave of equal blocks, with
  // at least 64 keys (four steps a block, one per warp) of the longest context
  // each: 1, 2, 3, 4 or 8 (clusters of 7 found room badly: 8 x 8192 keys 49 us
  // for 40; 3 for 2, 16 x 4096 keys of 24 rows and 64 dims, 27 for 30; a second,
  // part-filled wave there 36).
  const int64_t max_keys = a.paged ? (int64_t)a.max_pages << a.page_shift : rows / (a.hq / a.hkv);
  const int64_t room = (int64_t)L::blocks * num_sms / (items * a.hkv);
  int C = 1;
  while (C < 8 && C * 2 <= room && max_keys >= 128 * C) C *= 2;
  if (C == 2 && room >= 3 && max_keys >= 192) C = 3;
  if (items * C > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_rows_smem(std::integral_constant<int, NT * 1000 + HD * 2 + F8>(), kern, dim3((unsigned)(items * C), a.hkv),
                          dim3(kPaThreads), L::smem, C, st, a, tpq, C);
}
template <int HD, bool F8>
cudaError_t launch_pa_nt(const PAttn& a, int num_sms, cudaStream_t st) {
  // tiles of at most 32 rows, as even as column tiles of 8 allow
  const int64_t rows = (int64_t)std::min(a.max_q, a.tokens) * (a.hq / a.hkv);
  const int64_t least = (rows + 31) / 32;
  const int nt = (int)std::min<int64_t>(4, ((rows + least - 1) / least + 7) / 8);
  const int tpq = (int)((rows + nt * 8 - 1) / (nt * 8));
  switch (nt) {
    case 1: return launch_pa<HD, F8, 1>(a, rows, tpq, num_sms, st);
    case 2: return launch_pa<HD, F8, 2>(a, rows, tpq, num_sms, st);
    case 3: return launch_pa<HD, F8, 3>(a, rows, tpq, num_sms, st);
    default: return launch_pa<HD, F8, 4>(a, rows, tpq, num_sms, st);
  }
}
template <int HD>
cudaError_t launch_pa_hd(const PAttn& a, int num_sms, cudaStream_t st) {
  return a.f8 ? launch_pa_nt<HD, true>(a, num_sms, st) : launch_pa_nt<HD, false>(a, num_sms, st);
}

int fail(int code, const std::string& msg) {
  set_thread_error(msg);
  return code;
}
bool row_aligned(const void* p, int64_t ts, int64_t hs) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ts % 8 == 0 && hs % 8 == 0;
}

// Workspace of launch_pattn_td where it is taken, else 0.  It costs 5 us a tile
// and 10 us for its start and join, and saves up to a third of a long context's
// time.  It is taken at head dim 128 for more than 16 rows, tables of 2048
// positions or more and ten units of 128 keys an SM (20 below 4096 positions),
// for 9 to 16 with pages of 64, whose copies are fewer, and 50 units; and for any
// rows and dims where (sequence, KV head, tile) items are so few that the register
// tiles' clusters of eight blocks do not cover the SMs.  The lengths being on the
// device, a table's width stands for them.  Register tiles / this, us, 8 KV heads.
// 24 rows, head dim 128: 64 sequences x 4096 keys 153 / 116, x 2048 92 / 79,
// x 1024 56 / 63; 16 x 4096 49 / 43, x 2048 32 / 34; 4 x 8192
// 33 / 30, x 4096 23 / 26; 1 x 8192 28 / 26, x 4096 18 / 24, x 65536 147 / 52.  16
// rows, 64 x 4096: 111 / 112, with pages of 64 114 / 91, 16 x 4096 39 / 39; 2 x
// 16384 43 / 30.  4 rows: 64 x 4096 86 / 114, 1 x 16384 29 / 25, 2 x 16384 33 / 30.
// 24 rows, head dim 64: 64 x 4096 108 / 104, 4 x 8192 25 / 27, 1 x 16384 33 / 28.
size_t td_bytes(const PAttn& a, int64_t rows, int sms) {
  if (!a.paged || rows < 1 || rows > kPaMaxRows || !pattn_td_supported(a)) return 0;
  const int64_t keys = (int64_t)a.max_pages << a.page_shift, items = (int64_t)a.seqs * a.hkv * ((rows + 31) / 32);
  const int64_t units = items * ((keys + 127) / 128);
  if (units > 0x7fffffffLL) return 0;
  const bool wide = rows > 16;
  const int64_t least = !wide ? 50 : keys >= 4096 ? 10 : 20;
  const bool many = a.hd == 128 && (wide || (rows > 8 && a.page_shift >= 6)) && keys >= 2048 && units >= least * sms;
  const bool few = items * (rows > 8 ? 8 : 16) <= sms && keys >= (wide && a.hd == 128 ? 8192 : 16384);
  return many || few ? pattn_td_workspace(rows, a.hd, sms) : 0;
}

// Up to 32 rows per KV head the register-tile kernel, beyond kPaMaxRows the
// tensor-memory one where it applies.  Between them the first walks the keys
// once per 32 rows but cuts them between up to eight blocks, the second walks
// them once for all rows: it is taken where (sequence, KV head) pairs keep its
// blocks busy, at head dim 64 only from 49 rows and 16-bit keys on.  Measured,
// tensor memory against register tiles, 4096 keys, 8 KV heads, head dim 128:
// 64 rows of 16 sequences 61 / 75 us (8-bit keys 76 / 93), of 8 sequences
// 39 / 47 (45 / 56), of 4 37 / 31; 36 rows of 16 sequences 60 / 78 (76 / 94),
// of 12 60 / 52.  Head dim 64: 64 rows of 16 sequences 44 / 57 (67 / 72), of
// 12 44 / 39; 36 rows of 64 sequences 122 / 114 (191 / 160).  (The few-rows kernel
// takes 72 us for those 64 rows of 16 sequences of 8-bit keys, 62 for the 36, and
// 205 / 217 for 36 rows of 64 sequences: it is not asked here.)  A batch with
// both kinds goes whole: a short sequence costs the tensor-memory kernel one
// tile's walk over the keys beside the long ones, less than a second launch
// behind them.
struct Way {
  bool tc;        // pattn_tc.cu
  size_t td_ws;   // else pattn_td.cu with a workspace of so many bytes, if not 0; else the register tiles
};
Way choose_way(const PAttn& a, int sms) {
  const int64_t rows = (int64_t)std::min(a.max_q, a.tokens) * (a.hq / a.hkv), pairs = (int64_t)a.seqs * a.hkv;
  const bool many = rows > 48, busy = a.hd == 128 ? pairs * (many ? 8 : 4) >= 3 * sms : many && !a.f8 && pairs * 4 >= 3 * sms;
  if ((rows > kPaMaxRows || (rows > 32 && busy)) && pattn_tc_supported(a)) return {true, 0};
  return {false, td_bytes(a, rows, sms)};
}

// Both attention calls, after their own checks.
int run_attention(PAttn& a, size_t ws_bytes, const char* who, cudaStream_t st) {
  const std::string w = std::string(who) + ": ";
  if (a.hq < 1 || a.hkv < 1 || a.hq % a.hkv || a.hq > 65535 || a.hkv > 1024)
    return fail(SPEC_E_SHAPE, w + "n_heads must be a multiple of n_kv_heads (at most 1024)");
  if (a.hd != 32 && a.hd != 64 && a.hd != 128) return fail(SPEC_E_SHAPE, w + "head_dim must be 32, 64 or 128");
  if (a.tokens < 0 || a.max_q < 0 || a.seqs < 1) return fail(SPEC_E_ARG, w + "bad tokens, bound or seqs");
  if (!std::isfinite(a.scale_log2 * kLog2e) || a.scale_log2 < 0.f)
    return fail(SPEC_E_ARG, w + "scale must be finite, also times log2(e), and not negative");
  if ((int64_t)a.tokens * (a.hq / a.hkv) > 0x7fffffffLL) return fail(SPEC_E_ARG, w + "too many rows");
  if (a.tokens == 0 || a.max_q == 0) return SPEC_OK;
  if (!a.q || !a.out || !a.cu) return fail(SPEC_E_ARG, w + "null pointer");
  if (!row_aligned(a.q, a.q_ts, a.q_hs) || !row_aligned(a.out, a.o_ts, a.o_hs))
    return fail(SPEC_E_ARG, w + "q and out must be 16-byte aligned with strides multiples of 8");
  if (a.scale_log2 == 0.f) a.scale_log2 = 1.f / std::sqrt((float)a.hd);
  a.scale_log2 *= kLog2e;
  a.give_up = g_attn_give_up.load(std::memory_order_relaxed);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, w + cudaGetErrorString(e));
  const Way way = choose_way(a, sms);
  if (way.tc) e = launch_pattn_tc(a, sms, st);
  else if (way.td_ws && a.ws && ws_bytes >= way.td_ws) e = launch_pattn_td(a, sms, st);
  else e = a.hd == 32 ? launch_pa_hd<32>(a, sms, st) : a.hd == 64 ? launch_pa_hd<64>(a, sms, st) : launch_pa_hd<128>(a, sms, st);
  return e == cudaSuccess ? SPEC_OK : fail(SPEC_E_CUDA, w + cudaGetErrorString(e));
}

void cache_fields(PAttn& a, const spec_kv_cache* cache) {
  a.seqs = cache->seqs; a.hkv = cache->n_kv_heads; a.hd = cache->head_dim;
  a.paged = 1; a.f8 = cache->dtype == SPEC_DTYPE_E4M3;
  a.k = cache->k; a.v = cache->v; a.ks = cache->k_scale; a.vs = cache->v_scale;
  const int64_t row = (int64_t)cache->n_kv_heads * cache->page_size;
  a.page_stride = cache->page_stride ? cache->page_stride : row * cache->head_dim;
  a.scale_stride = cache->scale_page_stride ? cache->scale_page_stride : row;
  a.table = cache->table;
  a.table_stride = cache->table_stride ? cache->table_stride : cache->max_pages;
  a.pages = cache->pages; a.max_pages = cache->max_pages;
  while ((1 << a.page_shift) < cache->page_size) ++a.page_shift;
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" {

int spec_attn_paged(const spec_kv_cache* cache, const void* q, int64_t q_tok_stride, int64_t q_head_stride,
                    const int32_t* cu_q, const int32_t* kv_lens, int tokens, int max_q, int n_heads, float scale,
                    void* out, int64_t out_tok_stride, int64_t out_head_stride, float* lse, void* workspace,
                    int64_t workspace_bytes, void* stream) {
  const char* who = "spec_attn_paged";
  const int rc = check_cache(cache, who);
  if (rc) return rc;
  if (tokens > 0 && !kv_lens) return fail(SPEC_E_ARG, std::string(who) + ": null kv_lens");
  if (workspace_bytes < 0 || (reinterpret_cast<uintptr_t>(workspace) & 15u))
    return fail(SPEC_E_ARG, std::string(who) + ": workspace must be 16-byte aligned");
  PAttn a{};
  cache_fields(a, cache);
  a.q = q; a.q_ts = q_tok_stride; a.q_hs = q_head_stride;
  a.cu = cu_q; a.lens = kv_lens; a.tokens = tokens; a.max_q = max_q;
  a.hq = n_heads; a.scale_log2 = scale;
  a.out = out; a.o_ts = out_tok_stride; a.o_hs = out_head_stride; a.lse = lse;
  a.ws = (float*)workspace;
  return run_attention(a, workspace ? (size_t)workspace_bytes : 0, who, (cudaStream_t)stream);
}

int64_t spec_attn_paged_workspace(const spec_kv_cache* cache, int tokens, int max_q, int n_heads) {
  if (check_cache(cache, "spec_attn_paged_workspace") || tokens < 1 || max_q < 1 || n_heads < 1 ||
      n_heads % cache->n_kv_heads)
    return 0;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  PAttn a{};
  cache_fields(a, cache);
  // (queries and outputs with strides that the kernels take: others go to the register tiles)
  a.hq = n_heads; a.tokens = tokens; a.max_q = max_q;
  a.q_hs = a.o_hs = a.hd; a.q_ts = a.o_ts = (int64_t)n_heads * a.hd;
  return (int64_t)choose_way(a, sms).td_ws;
}

int spec_attn_prompt(const void* q, int64_t q_tok_stride, int64_t q_head_stride, const void* k, int64_t k_tok_stride,
                     int64_t k_head_stride, const void* v, int64_t v_tok_stride, int64_t v_head_stride,
                     const int32_t* cu, int seqs, int tokens, int max_len, int n_heads, int n_kv_heads, int head_dim,
                     float scale, void* out, int64_t out_tok_stride, int64_t out_head_stride, float* lse,
                     void* stream) {
  const char* who = "spec_attn_prompt";
  if (tokens > 0 && max_len > 0) {
    if (!k || !v) return fail(SPEC_E_ARG, std::string(who) + ": null pointer");
    if (!row_aligned(k, k_tok_stride, k_head_stride) || !row_aligned(v, v_tok_stride, v_head_stride))
      return fail(SPEC_E_ARG, std::string(who) + ": k and v must be 16-byte aligned with strides multiples of 8");
  }
  PAttn a{};
  a.q = q; a.q_ts = q_tok_stride; a.q_hs = q_head_stride;
  a.cu = cu; a.seqs = seqs; a.tokens = tokens; a.max_q = max_len;
  a.hq = n_heads; a.hkv = n_kv_heads; a.hd = head_dim; a.scale_log2 = scale;
  a.out = out; a.o_ts = out_tok_stride; a.o_hs = out_head_stride; a.lse = lse;
  a.k = k; a.v = v; a.k_ts = k_tok_stride; a.k_hs = k_head_stride; a.v_ts = v_tok_stride; a.v_hs = v_head_stride;
  return run_attention(a, 0, who, (cudaStream_t)stream);
}

}  // extern "C"
