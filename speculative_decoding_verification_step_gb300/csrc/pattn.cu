// Attention of a sequence's newest tokens over its keys, for few rows per KV
// head: a verify step's (K + 1) x G, one decoded token's G, a short prompt.
//
// With R = 16 or 32 rows per tile every key costs 4 R head_dim flops and
// 2 head_dim elements of K and V: below ~64 rows the cache's bytes bound the
// time, so a key is read once per tile, straight from its page into shared
// memory, and everything else is arranged around keeping those reads going.
//
// Block = (row tile, KV head, share of the keys), four warps.  The keys are
// walked in 16-key steps, step s on warp s mod 4.  Every warp keeps its own
// ring of kDepth steps filled by 16-byte asynchronous copies (no block
// barrier in the walk), swizzled by row so that ldmatrix finds its eight rows
// in distinct banks; rows past the length are filled with zeros, so whatever
// those slots hold cannot reach a product.
//   S = Q K^T and O += P V are m16n8k16 bf16 MMAs with fp32 sums, rows on the
//   M side: an accumulator of S is, packed to bf16, the A operand of P V, so
//   nothing is exchanged between lanes but the (rare) row maxima.
//   Online softmax with a lazy reference: a row's exponent reference only
//   moves when a score exceeds it by more than 2^8, so the usual step has no
//   shuffles and no rescaling of O; p <= 256 and the sums stay in fp32.
//   Probabilities are rounded to bf16 for P V (relative 2^-9 each, of random
//   sign: the same size as the output's own rounding); the row sum keeps them
//   in fp32.
// 8-bit keys and values: a byte's seven exponent and mantissa bits, moved to
// bits 4..10 of a bf16 with the sign on top, are the bf16 number code *
// 2^-120 exactly (subnormal codes too), two integer operations for two codes
// instead of a conversion.  Q carries 2^60 of it (exact), the rest and the
// row's power of two meet the scores in fp32, and those of V meet the
// probabilities before their rounding.
// The share of the keys: a cluster of up to 16 blocks splits one tile's keys
// and merges through distributed shared memory in a fixed order (no scratch
// memory, no second launch, no atomics): blocks merge their four warps, then
// block j of the cluster finishes the rows j, j + C, ...
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <string>

#include "common.cuh"
#include "paged.h"

namespace sv {

namespace {

constexpr int kPaThreads = 128;
constexpr int kPaWarps = 4;
constexpr int kPaStep = 16;          // keys of a step
constexpr float kPaLazy = 8.f;       // exponent reference moves past 2^8
constexpr float kPaNone = -1e30f;    // reference of a row that has seen nothing

template <int HD, bool F8>
struct PaLayout {
  static constexpr int row = HD * (F8 ? 1 : 2);      // bytes of a key row
  static constexpr int chunks = row / 16;
  static constexpr int tile = kPaStep * row;         // K or V of a step
  static constexpr int stage = 2 * tile + (F8 ? 32 : 0);
  static constexpr int depth = F8 ? 6 : (HD >= 128 ? 3 : 4);
  static constexpr int ring = kPaWarps * depth * stage;
  // Byte offset of 16-byte chunk c of row r: rows of less than 128 bytes
  // share a 128-byte line, so the row bits that vary over eight consecutive
  // lines are the ones to mix in.
  static SV_DEV int at(int r, int c) {
    constexpr int m = chunks >= 8 ? 7 : chunks - 1;
    const int x = chunks >= 8 ? r : r / (8 / chunks);
    return r * row + ((c ^ (x & m)) << 4);
  }
};
template <int HD, bool F8, int MT>
constexpr int pa_smem() {
  const int merge = kPaWarps * MT * 16 * HD * 4;
  return PaLayout<HD, F8>::ring > merge ? PaLayout<HD, F8>::ring : merge;
}

SV_DEV void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
SV_DEV void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
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
// Codes in bytes 0, 2 (even) or 1, 3 (odd) of w as bf16 pairs code * 2^-120.
SV_DEV uint32_t f8_even(uint32_t w) { return ((w << 4) & 0x07f007f0u) | ((w << 8) & 0x80008000u); }
SV_DEV uint32_t f8_odd(uint32_t w) { return ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u); }
// 2^(byte - 127), NaN for 255.
SV_DEV float f8_scale(uint32_t b) { return __uint_as_float(b == 255u ? 0x7fffffffu : b << 23); }

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
template <int HD, bool F8, int MT>
__global__ void __launch_bounds__(kPaThreads, 2) pattn_kernel(const __grid_constant__ PAttn a, int tpq, int C) {
  using L = PaLayout<HD, F8>;
  constexpr int kRows = MT * 16, kKs = HD / 16, kNt = HD / 8, D = L::depth;
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ float s_m[kPaWarps][kRows], s_l[kPaWarps][kRows];
  __shared__ float s_cm[kRows], s_cl[kRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
  const int share = blockIdx.x % C, item = blockIdx.x / C;
  const int b = item / tpq, tile = item - b * tpq, kvh = blockIdx.y;
  const int G = a.hq / a.hkv;

  // the sequence's rows and keys (every block of a cluster sees the same)
  const int r_first = __ldg(a.cu + b);
  const int n = __ldg(a.cu + b + 1) - r_first;
  if (r_first < 0 || n <= 0 || n > a.tokens - r_first || (int64_t)n * G > a.max_rows) return;
  int keys = n;
  if (a.paged) {
    keys = __ldg(a.lens + b);
    const int64_t cap = (int64_t)a.max_pages << a.page_shift;
    keys = keys < 0 ? 0 : (int)min((int64_t)keys, cap);
  }
  const int rows = min(n, a.max_q) * G;       // rows that are computed
  const int row0 = tile * kRows;
  if (row0 >= rows) return;
  const int first_pos = keys - n;             // position of the sequence's row 0
  const int last_row = min(rows, row0 + kRows) - 1;
  const int see_max = min(keys, max(0, first_pos + last_row / G + 1));   // keys that any row of the tile sees
  const int see_all = first_pos + row0 / G + 1;                          // keys that every row sees

  // Q fragments: lane's rows g and g + 8 of every 16-row tile.  8-bit keys:
  // codes come as (even, odd) bytes of four neighbours, so Q's k order is
  // permuted the same way, and carries 2^60.
  uint32_t qa[MT][kKs][4];
  int seen[MT][2];                            // keys seen by the lane's rows
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      const int r = row0 + mt * 16 + g + 8 * hr;
      const bool ok = r < rows;
      const int t = ok ? r / G : 0;
      seen[mt][hr] = ok ? min(keys, first_pos + t + 1) : 0;
      const bf16* qr = (const bf16*)a.q + (int64_t)(r_first + t) * a.q_ts + (int64_t)(kvh * G + (ok ? r - t * G : 0)) * a.q_hs;
#pragma unroll
      for (int ks = 0; ks < kKs; ++ks) {
        uint32_t lo = 0, hi = 0;
        if (ok) {
          if constexpr (F8) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(qr + ks * 16 + 4 * q4));   // k 4q .. 4q + 3
            lo = __byte_perm(w.x, w.y, 0x5410);   // (4q, 4q + 2)
            hi = __byte_perm(w.x, w.y, 0x7632);   // (4q + 1, 4q + 3)
            const __nv_bfloat162 up = __floats2bfloat162_rn(1152921504606846976.f, 1152921504606846976.f);   // 2^60
            __nv_bfloat162 x = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&lo), up);
            __nv_bfloat162 y = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&hi), up);
            lo = *reinterpret_cast<uint32_t*>(&x);
            hi = *reinterpret_cast<uint32_t*>(&y);
          } else {
            lo = __ldg(reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * q4));
            hi = __ldg(reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * q4 + 8));
          }
        }
        qa[mt][ks][hr] = lo;
        qa[mt][ks][2 + hr] = hi;
      }
    }

  float o[MT][kNt][4];
  float m[MT][2], l[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int j = 0; j < kNt; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mt][j][e] = 0.f;
    m[mt][0] = m[mt][1] = kPaNone;
    l[mt][0] = l[mt][1] = 0.f;
  }

  // this block's steps, and the warp's: s0 + 4 j
  const int steps = (see_max + kPaStep - 1) / kPaStep;
  const int s_beg = (int)((int64_t)steps * share / C), s_end = (int)((int64_t)steps * (share + 1) / C);
  const int s0 = s_beg + warp;
  const int nj = s_end > s0 ? (s_end - s0 + kPaWarps - 1) / kPaWarps : 0;
  unsigned char* ring = sm + (size_t)warp * D * L::stage;
  const uint32_t ring_u = smem_u32(ring);
  const int32_t* table = a.paged ? a.table + b * a.table_stride : nullptr;
  const int64_t ps_mask = ((int64_t)1 << a.page_shift) - 1;
  int pid = 0;   // lane i: page of the warp's step (j & ~31) + i

  // copies of the warp's step j into its ring slot
  auto issue = [&](int j) {
    if (a.paged && (j & 31) == 0) {
      const int64_t key = (int64_t)(s0 + kPaWarps * (j + lane)) * kPaStep;
      pid = j + lane < nj ? __ldg(table + (key >> a.page_shift)) : -1;
    }
    if (j < nj) {
      const int key0 = (s0 + kPaWarps * j) * kPaStep;
      int valid = min(kPaStep, keys - key0);
      const unsigned char *kp, *vp;
      int64_t krs, vrs;
      const uint8_t *ksp = nullptr, *vsp = nullptr;
      if (a.paged) {
        const int page = __shfl_sync(0xffffffffu, pid, j & 31);
        const bool in = page >= 0 && page < a.pages;
        if (!in) valid = 0;
        const int64_t row = ((int64_t)kvh << a.page_shift) + (key0 & ps_mask);
        const int64_t off = ((in ? page : 0) * a.page_stride + row * HD) * (F8 ? 1 : 2);
        kp = (const unsigned char*)a.k + off;
        vp = (const unsigned char*)a.v + off;
        krs = vrs = L::row;
        if constexpr (F8) {
          const int64_t so = (in ? page : 0) * a.scale_stride + row;
          ksp = a.ks + so;
          vsp = a.vs + so;
        }
      } else {
        kp = (const unsigned char*)((const bf16*)a.k + (int64_t)(r_first + key0) * a.k_ts + (int64_t)kvh * a.k_hs);
        vp = (const unsigned char*)((const bf16*)a.v + (int64_t)(r_first + key0) * a.v_ts + (int64_t)kvh * a.v_hs);
        krs = a.k_ts * 2;
        vrs = a.v_ts * 2;
      }
      unsigned char* dst = ring + (j % D) * L::stage;
#pragma unroll
      for (int i = 0; i < kPaStep * L::chunks / 32; ++i) {
        const int e = i * 32 + lane, r = e / L::chunks, c = e % L::chunks;
        const bool in = r < valid;
        // rows past the length are not read: the source stays on row 0
        cp_async16(dst + L::at(r, c), kp + (in ? r : 0) * krs + c * 16, in);
        cp_async16(dst + L::tile + L::at(r, c), vp + (in ? r : 0) * vrs + c * 16, in);
      }
      if constexpr (F8) {
        if (lane < 2) cp_async16(dst + 2 * L::tile + 16 * lane, lane ? vsp : ksp, valid > 0);
      }
    }
    cp_async_commit();
  };

  // ldmatrix rows of this lane: K (two key groups x two chunks) and V
  const int lr = lane & 7, l8 = (lane >> 3) & 1, l16 = lane >> 4;
#pragma unroll
  for (int j = 0; j < D - 1; ++j) issue(j);
  for (int j = 0; j < nj; ++j) {
    cp_async_wait<D - 2>();
    __syncwarp();
    const int key0 = (s0 + kPaWarps * j) * kPaStep;
    const uint32_t kt = ring_u + (uint32_t)((j % D) * L::stage), vt = kt + L::tile;
    float s[MT][2][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
    if constexpr (F8) {
#pragma unroll
      for (int c = 0; c < kKs; c += 2) {   // 16 codes a chunk: one k16 slice
        uint32_t w[4];                     // keys 0-7 chunk c, c + 1; keys 8-15 chunk c, c + 1
        ldsm4(w, kt + L::at(lr + 8 * l16, c + l8));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t b0 = f8_even(w[x]), b1 = f8_odd(w[x]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            mma_bf16_16816_acc(s[mt][x >> 1], qa[mt][c + (x & 1)][0], qa[mt][c + (x & 1)][1], qa[mt][c + (x & 1)][2],
                               qa[mt][c + (x & 1)][3], b0, b1);
        }
      }
    } else {
#pragma unroll
      for (int ks = 0; ks < kKs; ++ks) {
        uint32_t w[4];                     // keys 0-7 k 0-7, k 8-15; keys 8-15 k 0-7, k 8-15
        ldsm4(w, kt + L::at(lr + 8 * l16, 2 * ks + l8));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma_bf16_16816_acc(s[mt][0], qa[mt][ks][0], qa[mt][ks][1], qa[mt][ks][2], qa[mt][ks][3], w[0], w[1]);
          mma_bf16_16816_acc(s[mt][1], qa[mt][ks][0], qa[mt][ks][1], qa[mt][ks][2], qa[mt][ks][3], w[2], w[3]);
        }
      }
    }
    // scores in units of log2: key of element (nt, e) is key0 + 8 nt + 2 q4 + (e & 1)
    float vs[2][2];
    if constexpr (F8) {
      const unsigned char* sc = ring + (j % D) * L::stage + 2 * L::tile;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const uint32_t kb = *reinterpret_cast<const uint16_t*>(sc + 8 * nt + 2 * q4);
        const uint32_t vb = *reinterpret_cast<const uint16_t*>(sc + 16 + 8 * nt + 2 * q4);
        const float f = a.scale_log2 * 1152921504606846976.f;   // 2^60: codes carry 2^-120, Q 2^60
        const float k0 = f8_scale(kb & 255u) * f, k1 = f8_scale(kb >> 8) * f;
        vs[nt][0] = f8_scale(vb & 255u) * 1152921504606846976.f;
        vs[nt][1] = f8_scale(vb >> 8) * 1152921504606846976.f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          s[mt][nt][0] *= k0; s[mt][nt][1] *= k1;
          s[mt][nt][2] *= k0; s[mt][nt][3] *= k1;
        }
      }
    } else {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][nt][e] *= a.scale_log2;
    }
    if (key0 + kPaStep > see_all) {        // some row does not see all of the step
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + 8 * nt + 2 * q4 + (e & 1) >= seen[mt][e >> 1]) s[mt][nt][e] = neg_inf();
    }
    float top[MT][2];
    bool move = false;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        top[mt][hr] = fmaxf(fmaxf(s[mt][0][2 * hr], s[mt][0][2 * hr + 1]), fmaxf(s[mt][1][2 * hr], s[mt][1][2 * hr + 1]));
        move |= top[mt][hr] > m[mt][hr] + kPaLazy;
      }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          float t = top[mt][hr];
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
          t = fmaxf(t, m[mt][hr]);
          const float f = exp2_fast(m[mt][hr] - t);
          m[mt][hr] = t;
          l[mt][hr] *= f;
#pragma unroll
          for (int jn = 0; jn < kNt; ++jn) {
            o[mt][jn][2 * hr] *= f;
            o[mt][jn][2 * hr + 1] *= f;
          }
        }
    }
    uint32_t pa[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = exp2_fast(s[mt][nt][e] - m[mt][e >> 1]);
        l[mt][0] += p[0] + p[1];
        l[mt][1] += p[2] + p[3];
        if constexpr (F8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = p[e] == 0.f ? 0.f : p[e] * vs[nt][e & 1];
        }
        pa[mt][2 * nt] = pa_pack(p[0], p[1]);
        pa[mt][2 * nt + 1] = pa_pack(p[2], p[3]);
      }
    }
    if constexpr (F8) {
#pragma unroll
      for (int c = 0; c < kKs; c += 2) {   // chunks of 16 dims; keys 0-7, 8-15 of chunk c, then of c + 1
        uint32_t w[4];
        ldsm4t(w, vt + L::at(lr + 8 * l8, c + l16));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t e0 = f8_even(w[2 * x]), e1 = f8_even(w[2 * x + 1]);
          const uint32_t d0 = f8_odd(w[2 * x]), d1 = f8_odd(w[2 * x + 1]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {   // even dims, odd dims of the chunk
            mma_bf16_16816_acc(o[mt][2 * (c + x)], pa[mt][0], pa[mt][1], pa[mt][2], pa[mt][3], e0, e1);
            mma_bf16_16816_acc(o[mt][2 * (c + x) + 1], pa[mt][0], pa[mt][1], pa[mt][2], pa[mt][3], d0, d1);
          }
        }
      }
    } else {
#pragma unroll
      for (int jn = 0; jn < kNt; jn += 2) {
        uint32_t w[4];                     // keys 0-7, 8-15 of dims 8 jn ..; then of the next eight
        ldsm4t(w, vt + L::at(lr + 8 * l8, jn + l16));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma_bf16_16816_acc(o[mt][jn], pa[mt][0], pa[mt][1], pa[mt][2], pa[mt][3], w[0], w[1]);
          mma_bf16_16816_acc(o[mt][jn + 1], pa[mt][0], pa[mt][1], pa[mt][2], pa[mt][3], w[2], w[3]);
        }
      }
    }
    __syncwarp();
    issue(j + D - 1);
  }
  cp_async_wait<0>();
  __syncthreads();   // the rings become the merge area

  // ---- merge of the four warps: [warp][row][HD] ----
  float* part = reinterpret_cast<float*>(sm);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      float t = l[mt][hr];
      t += __shfl_xor_sync(0xffffffffu, t, 1);
      t += __shfl_xor_sync(0xffffffffu, t, 2);
      const int r = mt * 16 + g + 8 * hr;
      if (q4 == 0) {
        s_m[warp][r] = m[mt][hr];
        s_l[warp][r] = t;
      }
      float* d = part + ((size_t)warp * kRows + r) * HD;
      if constexpr (F8) {
#pragma unroll
        for (int c = 0; c < kKs; ++c)   // dims 4 q4 .. + 3 of chunk c
          *reinterpret_cast<float4*>(d + c * 16 + 4 * q4) =
              make_float4(o[mt][2 * c][2 * hr], o[mt][2 * c + 1][2 * hr], o[mt][2 * c][2 * hr + 1], o[mt][2 * c + 1][2 * hr + 1]);
      } else {
#pragma unroll
        for (int jn = 0; jn < kNt; ++jn)
          *reinterpret_cast<float2*>(d + jn * 8 + 2 * q4) = make_float2(o[mt][jn][2 * hr], o[mt][jn][2 * hr + 1]);
      }
    }
  __syncthreads();
  constexpr int kLpr = HD / 4;                 // lanes of a row, four dims each
  const int col = (tid % kLpr) * 4;
  auto write_row = [&](int r, float4 x, float mm, float ll) {
    const int R = row0 + r, t = R / G, h = kvh * G + R - t * G;
    const float f = ll > 0.f || !(ll == ll) ? (F8 ? 1152921504606846976.f : 1.f) / ll : 0.f;
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
      const float4 y = *reinterpret_cast<const float4*>(part + ((size_t)w * kRows + r) * HD + col);
      ll += s_l[w][r] * f;
      x.x += y.x * f; x.y += y.y * f; x.z += y.z * f; x.w += y.w * f;
    }
    if (C == 1) {
      write_row(r, x, mm, ll);
    } else {
      *reinterpret_cast<float4*>(part + (size_t)r * HD + col) = x;   // warp 0's slot of this element, read above
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
      const float4 y = ld_cluster_f32x4(cluster_map(pu + (uint32_t)(r * HD + col) * 4, c));
      ll += ld_cluster_f32(cluster_map(lu + 4 * r, c)) * f;
      x.x += y.x * f; x.y += y.y * f; x.z += y.z * f; x.w += y.w * f;
    }
    write_row(r, x, mm, ll);
  }
  cluster_arrive_wait();   // a block's memory stays until its peers have read it
}

template <int HD, bool F8, int MT>
cudaError_t launch_pa(const PAttn& a, int num_sms, cudaStream_t st) {
  constexpr int smem = pa_smem<HD, F8, MT>();
  auto kern = pattn_kernel<HD, F8, MT>;
  // attributes are per device and cheap to set again
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int G = a.hq / a.hkv;
  const int64_t rows = std::min<int64_t>((int64_t)std::min(a.max_q, a.tokens) * G, a.max_rows);
  const int tpq = (int)((rows + MT * 16 - 1) / (MT * 16));
  const int64_t items = (int64_t)a.seqs * tpq;
  // blocks of a cluster: until every SM has about one and a half, with at
  // least 64 keys (four steps a block, one per warp) of the longest context each
  const int64_t max_keys = a.paged ? (int64_t)a.max_pages << a.page_shift : rows / G;
  int C = 1;
  while (C < 8 && items * a.hkv * C * 2 < 3LL * num_sms && max_keys >= 128 * C) C *= 2;
  if (items * C > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_rows(kern, dim3((unsigned)(items * C), a.hkv), dim3(kPaThreads), smem, C, st, a, tpq, C);
}
template <int HD>
cudaError_t launch_pa_hd(const PAttn& a, int num_sms, cudaStream_t st) {
  const int64_t rows = std::min<int64_t>((int64_t)std::min(a.max_q, a.tokens) * (a.hq / a.hkv), a.max_rows);
  if (rows <= 16) return a.f8 ? launch_pa<HD, true, 1>(a, num_sms, st) : launch_pa<HD, false, 1>(a, num_sms, st);
  return a.f8 ? launch_pa<HD, true, 2>(a, num_sms, st) : launch_pa<HD, false, 2>(a, num_sms, st);
}

int fail(int code, const std::string& msg) {
  set_thread_error(msg);
  return code;
}
bool row_aligned(const void* p, int64_t ts, int64_t hs) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ts % 8 == 0 && hs % 8 == 0;
}

// Both attention calls, after their own checks.
int run_attention(PAttn& a, const char* who, cudaStream_t st) {
  const std::string w = std::string(who) + ": ";
  if (a.hq < 1 || a.hkv < 1 || a.hq % a.hkv || a.hq > 65535 || a.hkv > 1024)
    return fail(SPEC_E_SHAPE, w + "n_heads must be a multiple of n_kv_heads (at most 1024)");
  if (a.hd != 32 && a.hd != 64 && a.hd != 128) return fail(SPEC_E_SHAPE, w + "head_dim must be 32, 64 or 128");
  if (a.tokens < 0 || a.max_q < 0 || a.seqs < 1) return fail(SPEC_E_ARG, w + "bad tokens, bound or seqs");
  if (!(a.scale_log2 == a.scale_log2) || std::isinf(a.scale_log2) || a.scale_log2 < 0.f)
    return fail(SPEC_E_ARG, w + "scale must be finite and not negative");
  if ((int64_t)a.tokens * (a.hq / a.hkv) > 0x7fffffffLL) return fail(SPEC_E_ARG, w + "too many rows");
  if (a.tokens == 0 || a.max_q == 0) return SPEC_OK;
  if (!a.q || !a.out || !a.cu) return fail(SPEC_E_ARG, w + "null pointer");
  if (!row_aligned(a.q, a.q_ts, a.q_hs) || !row_aligned(a.out, a.o_ts, a.o_hs))
    return fail(SPEC_E_ARG, w + "q and out must be 16-byte aligned with strides multiples of 8");
  if (a.scale_log2 == 0.f) a.scale_log2 = 1.f / std::sqrt((float)a.hd);
  a.scale_log2 *= 1.4426950408889634f;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, w + cudaGetErrorString(e));
  // Sequences of at most kPaMaxRows rows per KV head go to the register-tile
  // kernel, longer chunks to the tensor-memory one where it applies; a batch
  // that may hold both kinds launches both, each skipping the other's.
  const int64_t rows = (int64_t)std::min(a.max_q, a.tokens) * (a.hq / a.hkv);
  a.max_rows = INT_MAX;
  if (rows > kPaMaxRows && pattn_tc_supported(a)) {
    a.max_rows = kPaMaxRows;
    e = launch_pattn_tc(a, sms, st);
    if (e != cudaSuccess) return fail(SPEC_E_CUDA, w + cudaGetErrorString(e));
  }
  e = a.hd == 32 ? launch_pa_hd<32>(a, sms, st) : a.hd == 64 ? launch_pa_hd<64>(a, sms, st) : launch_pa_hd<128>(a, sms, st);
  return e == cudaSuccess ? SPEC_OK : fail(SPEC_E_CUDA, w + cudaGetErrorString(e));
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" {

int spec_attn_paged(const spec_kv_cache* cache, const void* q, int64_t q_tok_stride, int64_t q_head_stride,
                    const int32_t* cu_q, const int32_t* kv_lens, int tokens, int max_q, int n_heads, float scale,
                    void* out, int64_t out_tok_stride, int64_t out_head_stride, float* lse, void* stream) {
  const char* who = "spec_attn_paged";
  const int rc = check_cache(cache, who);
  if (rc) return rc;
  if (tokens > 0 && !kv_lens) return fail(SPEC_E_ARG, std::string(who) + ": null kv_lens");
  PAttn a{};
  a.q = q; a.q_ts = q_tok_stride; a.q_hs = q_head_stride;
  a.cu = cu_q; a.lens = kv_lens; a.seqs = cache->seqs; a.tokens = tokens; a.max_q = max_q;
  a.hq = n_heads; a.hkv = cache->n_kv_heads; a.hd = cache->head_dim; a.scale_log2 = scale;
  a.out = out; a.o_ts = out_tok_stride; a.o_hs = out_head_stride; a.lse = lse;
  a.paged = 1; a.f8 = cache->dtype == SPEC_DTYPE_E4M3;
  a.k = cache->k; a.v = cache->v; a.ks = cache->k_scale; a.vs = cache->v_scale;
  const int64_t row = (int64_t)cache->n_kv_heads * cache->page_size;
  a.page_stride = cache->page_stride ? cache->page_stride : row * cache->head_dim;
  a.scale_stride = cache->scale_page_stride ? cache->scale_page_stride : row;
  a.table = cache->table;
  a.table_stride = cache->table_stride ? cache->table_stride : cache->max_pages;
  a.pages = cache->pages; a.max_pages = cache->max_pages;
  while ((1 << a.page_shift) < cache->page_size) ++a.page_shift;
  return run_attention(a, who, (cudaStream_t)stream);
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
  return run_attention(a, who, (cudaStream_t)stream);
}

}  // extern "C"
