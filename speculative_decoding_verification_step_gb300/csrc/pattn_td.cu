// Attention of few rows per KV head over long paged contexts with 8-bit keys: a
// verify step's (K + 1) x G rows.
//
// The cache's bytes bound the time (4 R flops against 2 bytes per key and dim):
// 128 keys of head dim 128 are 1450 clocks of an SM's share of HBM.  On
// mma.sync, with the codes expanded in registers, they cost twice that.  Here
// the keys are the 128-row side of tensor-memory products and the query rows
// the column side:
//   S^T [128 keys][R] = K Q^T, O^T [head_dim][R] += V^T P^T, R = 16 or 32,
// so a softmax thread owns a key and its R scores lie in its own lane: no
// exchange but the vote whether an exponent reference moves.
//   warps 0-3   softmax: thread = key, later thread = dim of O^T.  Row sums
//               stay in the thread until the tile ends;
//   warps 4, 7  copy K and V: page ids, one tensor copy per page, scales;
//   warp 5      issues S^T, up to four units ahead; warp 6 O^T.  (One warp for
//               both took 2100 clocks a unit, most of them its own waits);
//   warps 8-15  V's codes to bf16 (code * 2^e, exact), two groups of four warps
//               that take units in turn, and the next tile's Q.
// K is multiplied as it lies (kind::f8f6f4).  Each Q row, scaled by a power of
// two so that its largest element lies in (224, 448], is the sum of two e4m3
// terms, the upper four bits and the rest of a bf16's eight: exact for elements
// down to 2^-10 of the row's largest, off by at most 2^-17 of the largest below
// (half a step of e4m3's subnormals, 2^-10, of 224).  Both terms add up in the
// same fp32 sums; the two rows' powers of two multiply them exactly.
// The work is cut into units of 128 keys of one (sequence, KV head, row tile),
// all units in one row, and every SM takes one equal run of them, so that
// sequences of any lengths end together.  A run ends inside a tile at most at
// its two ends; those parts go to the workspace and a second launch joins
// them in order.  Copies run ahead across tiles.
// Every wait is for the phase after the last one that the same warp has seen (a
// wait by parity passes early when a barrier is two phases behind), so the V
// ring has an even number of stages: each belongs to one of the two groups.
// Bound by the softmax warps' latencies (1500 clocks a unit of 16 rows, 1800 of
// 24, 2000 of 32; the next unit's scores loaded early cost registers and were 4%
// slower, two units a pass 40%, a second softmax group with half of the rows 7%),
// by the copies of small pages next to them (16 rows over pages of 16 112 us, of
// 64 91) and by 5 us at the ends of a tile.  Measured (8 KV
// heads, head dim 128, 24 rows) against the register-tile kernel: 64 x 4096 keys
// 116 / 153 us (3.5 TB/s), 16 x 16384 115 / 140, 16 x 4096 43 / 49, 1 x 16384
// 29 / 45, 1 x 65536 52 / 147.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "pa_dev.cuh"
#include "paged.h"

namespace sv {

namespace {

constexpr int kTdKeys = 128, kTdThreads = 512;
constexpr int kTdBar = 1;            // named barrier of the softmax warps
constexpr float kTdLazy = 8.f, kTdNone = -1e30f;

struct TdArgs {
  TensorMap128 km, vm;
  PAttn a;
  int rows;         // rows of a tile, at most the product's columns (16 or 32)
  int runs;
};

// R rows of a tile are worked on (16, 24 or 32), cols columns of the products
// are theirs: what lies in the rest is never read.
template <int HD, int R>
struct TdLayout {
  static constexpr int cols = (R + 15) / 16 * 16;
  static constexpr int ks = 3, vs = 4, vb = 2;             // K and V tiles as copied, V tiles converted
  static constexpr uint32_t tile = kTdKeys * HD, vtile = kTdKeys * HD * 2;
  static constexpr uint32_t q = cols * HD * 2, p = kTdKeys * cols * 2;   // (two terms of HD bytes)
  static constexpr uint32_t k_at = 0, v_at = ks * tile, vb_at = v_at + vs * tile, q_at = vb_at + vb * vtile,
                            p_at = q_at + 2 * q;
  static constexpr int smem = (int)(p_at + 2 * p) + 1024;
  static_assert(smem <= 227 * 1024 - 2 * 1024, "with the scales and barriers, one block's shared memory");
};

// Units: 128 keys of one (sequence, KV head, row tile), in that order.
SV_DEV int td_seq_units(const PAttn& a, int tile_rows, int b, int* tiles) {
  const int r_first = __ldg(a.cu + b), n = __ldg(a.cu + b + 1) - r_first;
  int keys = __ldg(a.lens + b);
  *tiles = 0;
  if (r_first < 0 || n <= 0 || n > a.tokens - r_first) return 0;
  keys = keys < 0 ? 0 : (int)min((int64_t)keys, (int64_t)a.max_pages << a.page_shift);
  *tiles = (min(n, a.max_q) * (a.hq / a.hkv) + tile_rows - 1) / tile_rows;
  return max(1, (keys + kTdKeys - 1) / kTdKeys);   // a tile without keys is still written
}
SV_DEV int td_total(const PAttn& a, int tile_rows) {   // units of the call; whole warps
  int sum = 0;
  for (int b0 = 0; b0 < a.seqs; b0 += 32) {
    const int b = b0 + (threadIdx.x & 31);
    int tiles = 0;
    const int per = b < a.seqs ? td_seq_units(a, tile_rows, b, &tiles) : 0;
    sum += per * tiles * a.hkv;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}
SV_DEV int td_runs(int total, int most) { return max(1, min(most, total)); }
SV_DEV int td_begin(int total, int run, int runs) { return (int)((int64_t)total * run / runs); }
struct TdUnit {
  int b, kvh, tile, off, upi;
};
SV_DEV TdUnit td_find(const PAttn& a, int tile_rows, int u) {   // unit u; whole warps
  TdUnit w{};
  int before = 0;
  for (int b0 = 0; b0 < a.seqs; b0 += 32) {
    const int lane = threadIdx.x & 31, b = b0 + lane;
    int tiles = 0;
    const int per = b < a.seqs ? td_seq_units(a, tile_rows, b, &tiles) : 0;
    const int own = per * tiles * a.hkv;
    int sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + sum > u);
    if (past) {
      const int at = __ffs(past) - 1;
      const int in = u - before - __shfl_sync(0xffffffffu, sum - own, at), t = __shfl_sync(0xffffffffu, tiles, at);
      w.upi = __shfl_sync(0xffffffffu, per, at);
      w.b = b0 + at;
      const int item = in / w.upi;
      w.off = in - item * w.upi;
      w.kvh = item / t;
      w.tile = item - w.kvh * t;
      return w;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return w;
}

// A part of a tile that a run holds: units off .. off + seg - 1 of upi.
struct TdPart {
  int b, kvh, tile, tiles, off, seg, upi;
  int r_first, rows, row0, keys, first_pos;
};
SV_DEV void td_seq(const PAttn& a, int tile_rows, TdPart& p) {   // sequence p.b
  p.upi = td_seq_units(a, tile_rows, p.b, &p.tiles);
  p.r_first = __ldg(a.cu + p.b);
  const int n = __ldg(a.cu + p.b + 1) - p.r_first, keys = __ldg(a.lens + p.b);
  p.keys = keys < 0 ? 0 : (int)min((int64_t)keys, (int64_t)a.max_pages << a.page_shift);
  p.rows = min(n, a.max_q) * (a.hq / a.hkv);
  p.first_pos = p.keys - n;
}
// The run's first part (whole warps), and the one that starts at unit u behind p.
SV_DEV TdPart td_first(const PAttn& a, int tile_rows, int u, int u_end) {
  const TdUnit w = td_find(a, tile_rows, u);
  TdPart p;
  p.b = w.b;
  td_seq(a, tile_rows, p);
  p.kvh = w.kvh;
  p.tile = w.tile;
  p.off = w.off;
  p.row0 = p.tile * tile_rows;
  p.seg = min(p.upi - p.off, u_end - u);
  return p;
}
SV_DEV void td_next(const PAttn& a, int tile_rows, TdPart& p, int u, int u_end) {
  if (u >= u_end) return;
  p.off = 0;
  if (++p.tile >= p.tiles) {
    p.tile = 0;
    if (++p.kvh >= a.hkv) {
      p.kvh = 0;
      do {
        ++p.b;                                 // (unit u exists: some sequence holds it)
        td_seq(a, tile_rows, p);
      } while (p.tiles == 0 && p.b + 1 < a.seqs);
    }
  }
  p.row0 = p.tile * tile_rows;
  p.seg = min(p.upi, u_end - u);
}

template <int HD, int R>
__global__ void __launch_bounds__(kTdThreads, 1) pattn_td_kernel(const __grid_constant__ TdArgs ta) {
  using L = TdLayout<HD, R>;
  constexpr int C = L::cols, kHalf = HD / 64;
  constexpr int kSc = 8;                                   // K scales wait for the softmax, behind the ring
  extern __shared__ __align__(1024) unsigned char tsm[];
  __shared__ uint64_t k_full[L::ks], k_empty[L::ks], v_full[L::vs], v_empty[L::vs], b_full[2], b_empty[2];
  __shared__ uint64_t q_full[2], q_empty[2], s_full[4], p_full[4], pv_done[2], drained[2];
  __shared__ __align__(16) unsigned char s_ks[kSc][kTdKeys], s_vs[L::vs][kTdKeys];
  __shared__ float s_qf[2][C], s_red[4][C], s_f[C];
  __shared__ int64_t s_at[C];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ int s_kfill, s_vfill;
  const PAttn& a = ta.a;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int G = a.hq / a.hkv;
  const int total = td_total(a, ta.rows), runs = td_runs(total, ta.runs);
  if ((int)blockIdx.x >= runs || total == 0) return;
  const int u_beg = td_begin(total, blockIdx.x, runs), u_end = td_begin(total, blockIdx.x + 1, runs);
  const uint32_t base = (smem_u32(tsm) + 1023u) & ~1023u;

  if (warp == 4 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&ta.km)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&ta.vm)) : "memory");
    for (int s = 0; s < L::ks; ++s) {
      mbar_init(&k_full[s], 33);             // the tile's bytes, and every lane's scales
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < L::vs; ++s) {
      mbar_init(&v_full[s], 33);
      mbar_init(&v_empty[s], 4);             // converted by four warps
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&b_full[s], 4);
      mbar_init(&b_empty[s], 1);
      mbar_init(&q_full[s], 8);              // staged by the converting warps
      mbar_init(&q_empty[s], 4);             // the softmax warps: their scores and Q's factors are read
      mbar_init(&pv_done[s], 1);
      mbar_init(&drained[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
    }
    s_abort = 0;
    s_kfill = s_vfill = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(smem_u32(&s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  ta_fence_before();
  __syncthreads();
  ta_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  constexpr uint32_t kO = 128;               // columns: scores 0, 32, 64, 96; O^T 128

  // Q of tile k to its buffer: rows first, first + kStagers, ... of one warp
  constexpr int kStagers = 8, kOwn = C / kStagers;
  auto stage = [&](const TdPart& w, int k, int first) {
    const int buf = k & 1;
    if (k >= 2 && !__all_sync(0xffffffffu, ta_wait(&q_empty[buf], (unsigned)((k / 2 - 1) & 1), &s_abort))) return false;
    const uint32_t at = base + L::q_at + buf * L::q;
    constexpr int kPer = HD / 32;           // elements of a lane
    uint32_t raw[kOwn][kPer / 2];             // the loads before the first use
#pragma unroll
    for (int ri = 0; ri < kOwn; ++ri) {
      const int r = first + ri * kStagers, row = w.row0 + r, t = row / G;
      const bool in = r < ta.rows && row < w.rows;
      const bf16* qr = (const bf16*)a.q + (int64_t)(w.r_first + (in ? t : 0)) * a.q_ts +
                       (int64_t)(w.kvh * G + (in ? row - t * G : 0)) * a.q_hs + kPer * lane;
      if constexpr (kPer == 4) {
        const uint2 v = in ? __ldg(reinterpret_cast<const uint2*>(qr)) : make_uint2(0, 0);
        raw[ri][0] = v.x;
        raw[ri][1] = v.y;
      } else {
        raw[ri][0] = in ? __ldg(reinterpret_cast<const uint32_t*>(qr)) : 0u;
      }
    }
#pragma unroll
    for (int ri = 0; ri < kOwn; ++ri) {
      const int r = first + ri * kStagers;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) {
        const uint32_t z = raw[ri][i] & 0x7fff7fffu;
        m = max(m, max(z >> 16, z & 0xffffu));
      }
      m = __reduce_max_sync(0xffffffffu, m) << 16;
      // smallest 2^e with |q| <= 448 * 2^e; a row that is not finite scores NaN
      const bool bad = m >= 0x7f800000u;
      const int e = m == 0 || bad ? 0 : max((int)(m >> 23) - 127 - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0), -100);
      const float f = bad ? 0.f : __uint_as_float((uint32_t)(127 - e) << 23);
      uint32_t hi = 0, lo = 0;
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) {
        uint32_t y, hb;                    // a pair, its first terms and those back as fp16 (exact above 2^-17)
        uint16_t h, l;
        const float y0 = __uint_as_float(raw[ri][i] << 16) * f, y1 = __uint_as_float(raw[ri][i] & 0xffff0000u) * f;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(y1), "f"(y0));
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(y));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hb) : "h"(h));
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(y) : "r"(hb));
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(y));
        hi |= (uint32_t)h << (16 * i);
        lo |= (uint32_t)l << (16 * i);
      }
      if (bad) hi = 0x7f7f7f7fu, lo = 0;     // NaN codes: a masked score is still masked
      // rows r (upper bits) and C + r (the rest) of HD bytes
      const int chunk = (kPer * lane) >> 4, sub = (kPer * lane) & 15;
#pragma unroll
      for (int term = 0; term < 2; ++term) {
        const int rr = r + term * C, sw = HD == 128 ? chunk ^ (rr & 7) : chunk ^ ((rr >> 1) & 3);
        const uint32_t d = at + rr * HD + (sw << 4) + sub, v = term ? lo : hi;
        if constexpr (kPer == 4) asm volatile("st.shared.b32 [%0], %1;" ::"r"(d), "r"(v) : "memory");
        else asm volatile("st.shared.b16 [%0], %1;" ::"r"(d), "h"((uint16_t)v) : "memory");
      }
      if (lane == 0)
        s_qf[buf][r] = fmaxf(__uint_as_float((uint32_t)(127 + e) << 23) * a.scale_log2, 1.2e-38f);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_full[buf]);
    return true;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    // ---- V's codes to bf16 (thread = key row), and Q ----
    const int r = threadIdx.x & 127, s = (warp - 8) >> 2;   // a group of warps takes every other unit
    int i = 0, last = -1;                    // units of all parts, the last of this group
    bool ok = true;
    TdPart w = td_first(a, ta.rows, u_beg, u_end);
    int k = 0;
    ok = stage(w, 0, warp - 8);
    for (int u = u_beg; ok && u < u_end;) {
      u += w.seg;
      for (int j = 0; j < w.seg; ++j, ++i) {
        if ((i & 1) != s) continue;
        const int rs = i % L::vs;
        ok = ta_wait(&v_full[rs], (unsigned)((i / L::vs) & 1), &s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t code = s_vs[rs][r];
        const uint32_t src = base + L::v_at + rs * L::tile + r * HD, dst = base + L::vb_at + s * L::vtile + r * 128;
        uint32_t x[HD / 16][4];
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) {
          const int sw = HD == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[c][0]), "=r"(x[c][1]), "=r"(x[c][2]), "=r"(x[c][3]) : "r"(src + (sw << 4)) : "memory");
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_empty[rs]);
        if (i >= 2) ok = __all_sync(0xffffffffu, ta_wait(&b_empty[s], (unsigned)((i / 2 - 1) & 1), &s_abort));
        if (!ok) break;
        // a row past the length is zero whatever it holds
        const bool dead = (w.off + j) * kTdKeys + r >= w.keys;
        if (__any_sync(0xffffffffu, dead)) {
#pragma unroll
          for (int c = 0; c < HD / 16; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k) x[c][k] = dead ? 0u : x[c][k];
        }
        const float f = dead ? 0.f : row_power(code);
        const uint64_t scale = ta_pair(f, f);
#pragma unroll
        for (int c = 0; c < HD / 16; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) ta_codes(x[c][2 * h + k], scale, o[2 * k], o[2 * k + 1]);
            const int cc = 2 * c + h, col = cc & 7;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                         ::"r"(dst + (cc >> 3) * (L::vtile / kHalf) + ((col ^ (r & 7)) << 4)), "r"(o[0]), "r"(o[1]),
                           "r"(o[2]), "r"(o[3]) : "memory");
          }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_full[s]);
        last = i;
      }
      td_next(a, ta.rows, w, u, u_end);
      if (ok && u < u_end) ok = stage(w, ++k, warp - 8);
    }
    // the last product's signal has landed before the block ends
    if (ok && last >= 0) ta_wait(&b_empty[s], (unsigned)((last / 2) & 1), &s_abort);
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (warp == 4 || warp == 7) {
      // ---- producers: warp 4 of K, warp 7 of V ----
      const bool v = warp == 7;
      const int n = v ? L::vs : L::ks;
      uint64_t *fulls = v ? v_full : k_full, *empties = v ? v_empty : k_empty;
      const unsigned char* scales = v ? a.vs : a.ks;
      const uint32_t ring = base + (v ? L::v_at : L::k_at);
      const void* map = v ? &ta.vm : &ta.km;
      const int box_shift = min(a.page_shift, 7);       // keys of a unit from one page
      int i = 0;
      bool live = true;
      TdPart w = td_first(a, ta.rows, u_beg, u_end);
      for (int u = u_beg; live && u < u_end; td_next(a, ta.rows, w, u, u_end)) {
        u += w.seg;
        const int32_t* table = a.table + w.b * a.table_stride;
        const int npages = (int)(((int64_t)w.keys + (1 << a.page_shift) - 1) >> a.page_shift);
        auto page_of = [&](int j) {   // lane x: page of box x of unit j; -1 (zero rows) past the length or outside the pool
          const int64_t key = (int64_t)(w.off + j) * kTdKeys + (lane << box_shift);
          const int pg = (int)(key >> a.page_shift);
          const int page = lane < kTdKeys >> box_shift && j < w.seg && pg < npages ? __ldg(table + pg) : -1;
          return page >= a.pages ? -1 : page;
        };
        int next = page_of(0);
        for (int j = 0; j < w.seg; ++j, ++i) {
          const int page = next, s = i % n;
          next = page_of(j + 1);
          if (i >= n) live = __all_sync(0xffffffffu, ta_wait(&empties[s], (unsigned)((i / n - 1) & 1), &s_abort));
          if (!live) break;
          const uint32_t dst = ring + s * L::tile;
          const int row0 = (w.kvh << a.page_shift) + (int)(((int64_t)(w.off + j) * kTdKeys) & ((1 << a.page_shift) - 1));
          if (lane == 0) mbar_arrive_expect_tx(&fulls[s], L::tile);
          __syncwarp();
          const int per = kTdKeys >> box_shift;
          for (int b = 0; b < per; ++b) {
            const int pg = __shfl_sync(0xffffffffu, page, b);
            if (ta_elect()) ta_tma_3d(dst + (b << box_shift) * HD, map, 0, row0, pg, &fulls[s]);
          }
          __syncwarp();
          // scales: four keys a lane
          const int pg = __shfl_sync(0xffffffffu, page, (4 * lane) >> box_shift);
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                       ::"r"(smem_u32((v ? s_vs[s] : s_ks[i % kSc]) + 4 * lane)),
                       "l"(scales + (int64_t)max(pg, 0) * a.scale_stride + row0 + ((4 * lane) & ((1 << box_shift) - 1))),
                       "r"(pg < 0 ? 0 : 4) : "memory");
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&fulls[s])) : "memory");
          if (lane == 0) (v ? s_vfill : s_kfill) = i + 1;
        }
      }
      // the last fills are used, and the products' signals have landed, before the block ends
      for (int k = max(0, i - n); live && k < i; ++k)
        live = __all_sync(0xffffffffu, ta_wait(&empties[k % n], (unsigned)((k / n) & 1), &s_abort));
    } else {
      // ---- products: warp 5 the scores, warp 6 O^T (converged, one elected lane issues) ----
      constexpr uint32_t kId = (1u << 4) | ((uint32_t)(128 >> 4) << 24);
      constexpr uint32_t id_s = kId | ((uint32_t)(C >> 3) << 17);
      constexpr uint32_t id_o = ta_idesc(C, 1) | (1u << 15);     // both operands with keys along K, as they lie
      auto wait = [&](uint64_t* bar, unsigned parity) {
        const bool got = __all_sync(0xffffffffu, ta_wait(bar, parity, &s_abort));
        ta_fence_after();
        return got;
      };
      int i = 0, k = 0;                         // units and tiles done
      bool ok = true;
      TdPart w = td_first(a, ta.rows, u_beg, u_end);
      for (int u = u_beg; ok && u < u_end; ++k, td_next(a, ta.rows, w, u, u_end)) {
        u += w.seg;
        if (warp == 5) {
          ok = wait(&q_full[k & 1], (unsigned)((k / 2) & 1));
          const uint32_t q_at = base + L::q_at + (k & 1) * L::q;
          for (int j = 0; ok && j < w.seg; ++j, ++i) {
            // the scores before the last are read
            if (i >= 4) ok = wait(&p_full[i & 3], (unsigned)((i / 4 - 1) & 1));
            if (i + 1 == a.give_up) ok = __all_sync(0xffffffffu, ta_wait(&drained[0], 0, &s_abort, 0));
            ok = ok && wait(&k_full[i % L::ks], (unsigned)((i / L::ks) & 1));
            if (!ok) break;
            const uint32_t k_at = base + L::k_at + (uint32_t)(i % L::ks) * L::tile;
            if (ta_elect()) {
              const uint64_t kd = HD == 128 ? ta_desc(k_at, 1) : ta_desc_narrow(k_at, 4);
              const uint64_t qd = HD == 128 ? ta_desc(q_at, 1) : ta_desc_narrow(q_at, 4);
#pragma unroll
              for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int s = 0; s < HD / 32; ++s)
                  ta_mma_f8(tmem + (i & 3) * 32, kd + 2 * s, qd + t * (C * HD / 16) + 2 * s, id_s, t + s > 0);
              ta_commit(&s_full[i & 3]);
              ta_commit(&k_empty[i % L::ks]);
            }
            __syncwarp();
          }
        } else {
          for (int j = 0; j < w.seg; ++j, ++i) {
            const int s = i & 1;
            ok = wait(&b_full[s], (unsigned)((i / 2) & 1));
            const uint32_t v_at = base + L::vb_at + s * L::vtile;
            ok = ok && wait(&p_full[i & 3], (unsigned)((i / 4) & 1));
            if (!ok) break;
            if (ta_elect()) {
              // head dim 64: the 128 lanes hold the dims twice
              const uint64_t vd = ta_desc(v_at, HD == 64 ? 0 : (L::vtile / kHalf) >> 4);
              const uint64_t pd = ta_desc_narrow(base + L::p_at + (i & 1) * L::p, C / 8);
#pragma unroll
              for (int ks = 0; ks < kTdKeys / 16; ++ks)
                ta_mma_ss(tmem + kO, vd + ks * 128, pd + ks * (16 * C * 2 / 16), id_o, j > 0 || ks > 0);
              ta_commit(&pv_done[i & 1]);
              ta_commit(&b_empty[s]);
            }
            __syncwarp();
          }
        }
      }
    }
  } else {
    // ---- softmax: thread = key of a unit, then dim of O^T ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int tid = threadIdx.x;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    // true when any of the softmax threads says so (a barrier of theirs)
    auto any = [&](bool x) {
      uint32_t y;
      asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
                   : "=r"(y) : "r"((uint32_t)x), "n"(kTdBar) : "memory");
      return y != 0;
    };
    int i = 0, k = 0;
    bool ok = true;                           // the same in all softmax threads
    TdPart w = td_first(a, ta.rows, u_beg, u_end);
    for (int u = u_beg; u < u_end; ++k, td_next(a, ta.rows, w, u, u_end)) {
      const bool whole = w.off == 0 && w.seg == w.upi;
      const int piece = w.off > 0 ? 0 : 1;
      u += w.seg;
      // pairs of rows: minus the reference, the sum, the score's factor
      uint64_t nm[R / 2], l2[R / 2], q2[R / 2];
      bool got = !ok || ta_wait(&q_full[k & 1], (unsigned)((k / 2) & 1), &s_abort);
#pragma unroll
      for (int r = 0; r < R / 2; ++r) {
        nm[r] = ta_pair(-kTdNone, -kTdNone);
        l2[r] = 0;
        q2[r] = ta_pair(s_qf[k & 1][2 * r], s_qf[k & 1][2 * r + 1]);
      }
      const int last_row = min(w.rows, w.row0 + ta.rows) - 1;
      const int see_all = w.first_pos + w.row0 / G + 1;       // keys that every row sees
      for (int j = 0; j < w.seg && ok; ++j, ++i) {
        got = __all_sync(0xffffffffu, got && ta_wait(&s_full[i & 3], (unsigned)((i / 4) & 1), &s_abort));
        ta_fence_after();
        const uint32_t code = s_ks[i % kSc][tid];
        const float kf = row_power(code);
        // scores, -inf where a row does not see the key
        auto scores = [&](float* s) {
#pragma unroll
          for (int c = 0; c < R; c += 8) ta_ld8(tmem + lanes + (i & 3) * 32 + c, s + c);
          ta_wait_ld();
          ta_pin<R>(s);
          const uint64_t kk = ta_pair(kf, kf);
#pragma unroll
          for (int r = 0; r < R; r += 2) ta_split(ta_mul2(ta_pair(s[r], s[r + 1]), kk), s[r], s[r + 1]);
          if ((w.off + j + 1) * kTdKeys > see_all) {
            // row w.row0 + r sees the key from token key - first_pos on
            const int key = (w.off + j) * kTdKeys + tid;
            const int from = key >= w.keys ? 0x7fffffff : (key - w.first_pos) * G - w.row0;
#pragma unroll
            for (int r = 0; r < R; ++r)
              if (r < from) s[r] = neg_inf();
          }
        };
        float x[R];
        float top = kTdNone;
        if (got) {
          scores(x);
#pragma unroll
          for (int r = 0; r < R; r += 2) {
            ta_split(ta_fma2(ta_pair(x[r], x[r + 1]), q2[r / 2], nm[r / 2]), x[r], x[r + 1]);
            top = ta_max3(top, x[r], x[r + 1]);
          }
        }
        const bool move = any(top > kTdLazy || !got);
        if (move) {
          ok = !any(!got);
          if (!ok) break;
        }
        // P's buffer is free (a failure is seen at the next vote)
        if (i >= 2) got = __all_sync(0xffffffffu, ta_wait(&pv_done[i & 1], (unsigned)((i / 2 - 1) & 1), &s_abort));
        ta_fence_after();
        if (move) {
          // new references: the largest over the 128 keys
          scores(x);
#pragma unroll
          for (int r = 0; r < R; r += 2) {
            float t0, t1;
            ta_split(ta_mul2(ta_pair(x[r], x[r + 1]), q2[r / 2]), t0, t1);
            asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(t0));
            asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(t1));
            if (lane == 0) *reinterpret_cast<float2*>(&s_red[warp][r]) = make_float2(t0, t1);
          }
          // O^T holds the units before: the last of them is done
          if (j > 0) got = __all_sync(0xffffffffu, got && ta_wait(&pv_done[(i - 1) & 1], (unsigned)(((i - 1) / 2) & 1), &s_abort));
          ta_fence_after();
          named_sync(kTdBar, 128);
#pragma unroll
          for (int c = 0; c < R; c += 8) {
            float o[8];
            if (j > 0) {
              ta_ld8(tmem + lanes + kO + c, o);
              ta_wait_ld();
              ta_pin<8>(o);
            }
#pragma unroll
            for (int r = c; r < c + 8; r += 2) {
              float n0, n1, t[2];
              ta_split(nm[r / 2], n0, n1);
#pragma unroll
              for (int e = 0; e < 2; ++e)
                t[e] = fminf(fminf(fminf(-s_red[0][r + e], -s_red[1][r + e]), fminf(-s_red[2][r + e], -s_red[3][r + e])), e ? n1 : n0);
              const float f0 = ta_exp2(t[0] - n0), f1 = ta_exp2(t[1] - n1);
              nm[r / 2] = ta_pair(t[0], t[1]);
              l2[r / 2] = ta_mul2(l2[r / 2], ta_pair(f0, f1));
              ta_split(ta_fma2(ta_pair(x[r], x[r + 1]), q2[r / 2], nm[r / 2]), x[r], x[r + 1]);
              o[r - c] *= f0;
              o[r - c + 1] *= f1;
            }
            if (j > 0) ta_st8(tmem + lanes + kO + c, reinterpret_cast<uint32_t*>(o));
          }
          if (j > 0) ta_wait_st();
          named_sync(kTdBar, 128);              // s_red is read
        }
        const uint32_t p_at = base + L::p_at + (i & 1) * L::p + tid * C * 2;
#pragma unroll
        for (int r = 0; r < R; r += 8) {
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p0 = ta_exp2(x[r + 2 * e]), p1 = ta_exp2(x[r + 2 * e + 1]);
            l2[r / 2 + e] = ta_add2(l2[r / 2 + e], ta_pair(p0, p1));
            v[e] = ta_pack(p0, p1);
          }
          const int c = r / 8, sw = C == 32 ? c ^ ((tid >> 1) & 3) : c ^ ((tid >> 2) & 1);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                       ::"r"(p_at + (sw << 4)), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        ta_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[i & 3]);
      }
      // the tile's sums
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[k & 1]);
      if (ok) {
        const bool done = __all_sync(0xffffffffu, ta_wait(&pv_done[(i - 1) & 1], (unsigned)(((i - 1) / 2) & 1), &s_abort));
        ta_fence_after();
        ok = !any(!done || !got);
      }
      float l[C] = {};
#pragma unroll
      for (int r = 0; r < R; r += 2) ta_split(l2[r / 2], l[r], l[r + 1]);
      // sums over the lanes, halving the rows of a lane at each exchange
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const bool up = lane & o;
        const int n = C * o / 32;
        if (n > 0) {
#pragma unroll
          for (int r = 0; r < n; ++r) {
            const float give = up ? l[r] : l[r + n], keep = up ? l[r + n] : l[r];
            l[r] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        } else {
          l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
        }
      }
      s_red[warp][lane / (32 / C)] = l[0];
      float o[R];
      if (ok) {
#pragma unroll
        for (int c = 0; c < R; c += 8) ta_ld8(tmem + lanes + kO + c, o + c);
        ta_wait_ld();
        ta_pin<R>(o);
        ta_fence_before();
      }
      named_sync(kTdBar, 128);
      // row r's sum, reference and place on lane r
      const int lr = lane % C, row = w.row0 + lr, t = row / G, h = w.kvh * G + row - t * G;
      const int live = last_row + 1 - w.row0;
      const float sum = !ok ? __uint_as_float(0x7fffffffu) : (s_red[0][lr] + s_red[1][lr]) + (s_red[2][lr] + s_red[3][lr]);
      float ref = 0.f;
#pragma unroll
      for (int r = 0; r < R; r += 2) {
        float n0, n1;
        ta_split(nm[r / 2], n0, n1);
        ref = r == lr ? -n0 : r + 1 == lr ? -n1 : ref;
      }
      if (whole) {
        const float f = sum > 0.f || !(sum == sum) ? 1.f / sum : 0.f;
        const int64_t at = (int64_t)(w.r_first + t) * a.o_ts + (int64_t)h * a.o_hs;
        if (lane < R) {
          s_at[lane] = at;                    // (the same from all four warps)
          s_f[lane] = f;
        }
        __syncwarp();
        bf16* d = (bf16*)a.out + tid;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float fr = s_f[r];
          const bf16 y = __float2bfloat16_rn(ok ? o[r] * fr : fr);
          if (r < live && tid < HD) d[s_at[r]] = y;
        }
        if (a.lse && warp == 0 && lane < R && lane < live)
          a.lse[(int64_t)(w.r_first + t) * a.hq + h] = sum == 0.f ? neg_inf() : (ref + log2f(sum)) * 0.6931471805599453f;
      } else {
        float* d = a.ws + ((size_t)blockIdx.x * 2 + piece) * R * (HD + 2);
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (r < live && tid < HD) d[r * HD + tid] = ok ? o[r] : 0.f;
        if (warp == 0 && lane < R) {
          d[R * HD + lane] = ref;
          d[R * (HD + 1) + lane] = sum;
        }
      }
      named_sync(kTdBar, 128);                // s_red is read
    }
  }
  __syncthreads();
  // a wait gave up, in whichever warp: products and copies in flight end (bounded) before the space goes
  if (s_abort && (warp == 5 || warp == 6)) ta_drain(&drained[warp - 5]);
  if (s_abort && threadIdx.x == 0) {
    for (int i = max(0, s_kfill - L::ks); i < s_kfill; ++i) {
      long long spins = 0;
      while (!mbar_test(&k_full[i % L::ks], (unsigned)((i / L::ks) & 1)) && ++spins < (1LL << 20)) {
      }
    }
    for (int i = max(0, s_vfill - L::vs); i < s_vfill; ++i) {
      long long spins = 0;
      while (!mbar_test(&v_full[i % L::vs], (unsigned)((i / L::vs) & 1)) && ++spins < (1LL << 20)) {
      }
    }
  }
  __syncthreads();
  if (warp == 5) {
    ta_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem) : "memory");
  }
}

// Joins the parts of the tile that the border before run x + 1 cuts, if it is
// the first border inside that tile.  A warp a row: rows 4 y .. 4 y + 3.
template <int HD>
__global__ void __launch_bounds__(128) pattn_join_kernel(const __grid_constant__ PAttn a, int tile_rows, int cols, int most) {
  const int total = td_total(a, tile_rows), runs = td_runs(total, most), c0 = blockIdx.x;
  if (c0 + 1 >= runs) return;
  const int u = td_begin(total, c0 + 1, runs);
  const TdUnit w = td_find(a, tile_rows, u);
  if (w.off == 0) return;                      // the border lies between tiles
  const int first = u - w.off;
  if (td_begin(total, c0, runs) > first) return;   // an earlier border cuts it too
  int c1 = c0 + 1;                             // the run that ends it
  while (c1 + 1 < runs && td_begin(total, c1 + 1, runs) < first + w.upi) ++c1;
  const int G = a.hq / a.hkv, lane = threadIdx.x & 31, rr = blockIdx.y * 4 + (threadIdx.x >> 5);
  const int r_first = __ldg(a.cu + w.b), rows = min(__ldg(a.cu + w.b + 1) - r_first, a.max_q) * G;
  if (rr >= tile_rows || w.tile * tile_rows + rr >= rows) return;
  constexpr int kPer = HD / 32;                // dims of a lane
  auto part = [&](int c) { return a.ws + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * cols * (HD + 2); };
  float mm = kTdNone;
  for (int c = c0 + lane; c <= c1; c += 32) mm = fmaxf(mm, __ldcg(part(c) + cols * HD + rr));
  mm = warp_max(mm);
  float ll = 0.f, x[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) x[i] = 0.f;
  for (int cb = c0; cb <= c1; cb += 32) {      // the parts' references and sums on the lanes
    float f = 0.f, lv = 0.f;
    if (cb + lane <= c1) {
      const float* d = part(cb + lane);
      f = ta_exp2(__ldcg(d + cols * HD + rr) - mm);
      lv = __ldcg(d + cols * (HD + 1) + rr) * f;
    }
    ll += warp_sum(lv);
    const int np = min(32, c1 - cb + 1);
#pragma unroll 8
    for (int c = 0; c < np; ++c) {
      const float fc = __shfl_sync(0xffffffffu, f, c);
      const float* d = part(cb + c) + rr * HD + kPer * lane;
      if constexpr (kPer == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(d));
        x[0] += v.x * fc; x[1] += v.y * fc; x[2] += v.z * fc; x[3] += v.w * fc;
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(d));
        x[0] += v.x * fc; x[1] += v.y * fc;
      }
    }
  }
  const int row = w.tile * tile_rows + rr, t = row / G, h = w.kvh * G + row - t * G;
  const float f = ll > 0.f || !(ll == ll) ? 1.f / ll : 0.f;
  bf16* d = (bf16*)a.out + (int64_t)(r_first + t) * a.o_ts + (int64_t)h * a.o_hs + kPer * lane;
  if constexpr (kPer == 4) *reinterpret_cast<uint2*>(d) = make_uint2(ta_pack(x[0] * f, x[1] * f), ta_pack(x[2] * f, x[3] * f));
  else *reinterpret_cast<uint32_t*>(d) = ta_pack(x[0] * f, x[1] * f);
  if (a.lse && lane == 0)
    a.lse[(int64_t)(r_first + t) * a.hq + h] = ll == 0.f ? neg_inf() : (mm + log2f(ll)) * 0.6931471805599453f;
}

template <int HD, int R>
cudaError_t launch_td(const TdArgs& ta, cudaStream_t st) {
  using L = TdLayout<HD, R>;
  auto kern = pattn_td_kernel<HD, R>;
  cudaError_t e = launch_rows_smem(std::integral_constant<int, HD * 100 + R>(), kern, dim3((unsigned)ta.runs),
                                   dim3(kTdThreads), L::smem, 1, st, ta);
  if (e != cudaSuccess || ta.runs < 2) return e;
  return launch_rows(pattn_join_kernel<HD>, dim3((unsigned)ta.runs - 1, (ta.rows + 3) / 4), dim3(128), 0, 1, st, ta.a, ta.rows, R,
                     ta.runs);
}

// Rows that a call's tiles are worked on with: even tiles of at most 32.
int td_rows(int64_t rows) {
  const int64_t tiles = (rows + 31) / 32;
  return std::max<int>(16, (int)((rows + tiles - 1) / tiles + 7) / 8 * 8);
}

}  // namespace

bool pattn_td_supported(const PAttn& a) {
  return a.f8 && (a.hd == 64 || a.hd == 128) && a.page_stride > 0 && a.page_stride < 1LL << 38 &&
         (int64_t)a.hkv << a.page_shift <= 0x7fffffffLL;
}
size_t pattn_td_workspace(int64_t rows, int hd, int num_sms) {
  return (size_t)num_sms * 2 * td_rows(rows) * (hd + 2) * sizeof(float);
}

cudaError_t launch_pattn_td(const PAttn& a, int num_sms, cudaStream_t st) {
  TdArgs ta{};
  ta.a = a;
  const int64_t rows = (int64_t)std::min(a.max_q, a.tokens) * (a.hq / a.hkv), tiles = (rows + 31) / 32;
  const int r = td_rows(rows);
  ta.rows = (int)((rows + tiles - 1) / tiles);
  ta.runs = num_sms;
  const int ps = 1 << a.page_shift, box = std::min(ps, kTdKeys);
  if (!ta_map(ta.km, a.k, a.hd, (int64_t)a.hkv * ps, a.pages, a.hd, a.page_stride, box, 1, 1) ||
      !ta_map(ta.vm, a.v, a.hd, (int64_t)a.hkv * ps, a.pages, a.hd, a.page_stride, box, 1, 1))
    return cudaErrorInvalidValue;
  if (a.hd == 128) return r == 16 ? launch_td<128, 16>(ta, st) : r == 24 ? launch_td<128, 24>(ta, st) : launch_td<128, 32>(ta, st);
  return r == 16 ? launch_td<64, 16>(ta, st) : r == 24 ? launch_td<64, 24>(ta, st) : launch_td<64, 32>(ta, st);
}

}  // namespace sv
