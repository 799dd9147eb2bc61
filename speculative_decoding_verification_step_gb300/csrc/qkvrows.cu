// Norms of queries and keys for each head, with the position rotation and the cache
// write in the same pass.
//
//   y = R(pos) [ x * w / sqrt(mean(x^2) + eps) ]
// of each head of q (to rows) and k (to the cache), and v to the cache as it is: one
// launch where a norm of q, one of k, two rotations and the write were five, and each
// row read and written once.  A row (token, head) is held by head_dim / 16 adjacent
// lanes, two 16-byte chunks each that are rotated together, so the sum of squares and
// an 8-bit row's largest magnitude are shuffles away; sums, norm and rotation in fp32,
// one rounding at the store.  Angles and 8-bit rows as in kvrows.cu.
//
// Bound by HBM for prompts, by launch and dependent loads for a verify step's rows.
// Blocks of q, of k and of v lie side by side in one grid, 1024 threads' work each (512: 2%
// more for 40 heads of 64).
// Measured: 4 x 4000 rows of 32 + 8 + 8 bf16 heads of 128 to an e4m3 cache 65 us (5.5 TB/s,
// 82% of a copy's rate), to a bf16 one 65 us (90%), from fp32 rows 88 us (99%); 16381 rows of
// 40 heads of 64 30 us (5.6 TB/s, 83%); a step's 6 tokens 3.0 us.  Beside its 32 bytes of a
// bf16 row a lane reads 64 of cosines and sines from shared memory and 64 of gains from L1,
// whose pipe was busy for 75% of the time while lanes met in banks and gains came in
// fours (69 and 33 us), and is for 57% now; issue slots are at 68%.  Angles in registers
// over several heads (or gains over several tokens) took 94 registers a thread for 56, and
// with the fewer rows in flight 74 us (69) for 68.5; three rows of a thread in flight 91, the
// compiler held to 48 registers 71; packed fp32 arithmetic in the norm changes nothing.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "common.cuh"
#include "paged.h"
#include "rows_dev.cuh"

namespace sv {

namespace {

constexpr int kMaxAnyDim = 512;      // head_dim of the element-wise form

struct QkvPart {
  const void* x;
  int64_t ts, hs;
  const float* gain;                 // null: no norm
  int64_t gain_hs;
  int heads, rot;                    // rot 0: no rotation
  int tpb, hpb, hblocks, blocks;     // tokens and heads of a block, blocks of a token's heads, blocks
  uint32_t m_heads;                  // quick_div by hpb
};
struct QkvArgs {
  QkvPart part[3];                   // q, k, v
  CacheArgs c;
  void* y;                           // q's rows
  int64_t yt, yh;
  const int32_t* seq;
  const int32_t* pos;
  int tokens, hd;
  float eps;
  spec_rope r;
};

// Sum over `lanes` adjacent lanes (a power of two).
template <int Lanes>
SV_DEV float lanes_sum(float v) {
#pragma unroll
  for (int o = Lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int Lanes>
SV_DEV uint32_t lanes_max(uint32_t m) {
#pragma unroll
  for (int o = Lanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// Rows without a norm turn by the same angles, to the bit, as in rope_rows and kv_append; of normed
// ones those whose rounding is fp32's, or so coarse that its neighbours count (codes), turn by the
// finer ones (16381 rows to fp32 off by 6.4e-8 of their size for 7.6e-8, PyTorch 6.9e-8).
template <typename TO, bool F8>
SV_DEV bool fine_angles(const QkvPart& p, int kind) {
  return p.gain && (kind ? F8 : sizeof(TO) == 4);
}
SV_DEV void row_cos_sin(const spec_rope& r, bool fine, int i, int pos, float* c, float* s) {
  if (fine) turn_cos_sin_fine(r, i, pos, c, s);
  else turn_cos_sin(r, i, pos, 1.f, c, s);
}
// 1 / sqrt(m) with one correction: the function is off by up to two units, as a factor of the
// whole row.
SV_DEV float inverse_root(float m) {
  const float y = rsqrtf(m);
  if (!(y > 0.f && y < 3e38f)) return y;       // of 0, infinity or NaN
  const float h = m * y, l = fmaf(m, y, -h);   // m y, exactly
  return fmaf(0.5f * y, fmaf(-l, y, fmaf(-h, y, 1.f)), y);
}
// Eight gains in one load: two of four, 32 bytes apart from lane to lane, take L1 twice as long.
SV_DEV void load_gain8(float (&x)[8], const float* p) {
  asm("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]) : "l"(p));
}

template <typename T, typename TO, int HD, bool F8>
__global__ void __launch_bounds__(kRowThreads) qkv_kernel(const __grid_constant__ QkvArgs a) {
  constexpr int V = 8, kLanes = HD / (2 * V), kBatch = kRowBatch;
  extern __shared__ __align__(16) float cs[];   // cosines [tpb][pad], sines [tpb][pad]
  __shared__ int2 slot[kMaxTokBlock];
  int blk = blockIdx.x, kind = 0;
  if (blk >= a.part[0].blocks) {
    blk -= a.part[0].blocks;
    kind = 1;
    if (blk >= a.part[1].blocks) {
      blk -= a.part[1].blocks;
      kind = 2;
    }
  }
  const QkvPart& p = a.part[kind];
  const int rot = p.rot, np = rot / 2, pad = (np + 7) & ~7;
  const int tb = blk / p.hblocks, h0 = (blk - tb * p.hblocks) * p.hpb;
  const int t0 = tb * p.tpb, nt = min(p.tpb, a.tokens - t0), nh = min(p.hpb, p.heads - h0);
  float* const si = cs + p.tpb * pad;
  const T* const src = (const T*)p.x + t0 * p.ts + h0 * p.hs;
  const int rows = nt * nh, stride = kRowThreads / kLanes, u = threadIdx.x % kLanes;
  int ca, cb;
  unit_chunks<V>(u, rot, a.r.interleaved, &ca, &cb);
  for (int r0 = (int)threadIdx.x / kLanes, pass = 0;; r0 += kBatch * stride, ++pass) {
    if (pass && !__any_sync(0xffffffffu, r0 < rows)) break;   // whole warps stay together for the shuffles
    RawV<T, V> ra[kBatch], rb[kBatch];          // rows in flight
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int row = min(r0 + q * stride, rows - 1);
      const int t = quick_div(row, p.m_heads), h = row - t * p.hpb;
      const T* x = src + t * p.ts + h * p.hs;
      ra[q].load(x + ca * V);
      rb[q].load(x + cb * V);
    }
    if (pass == 0) {   // the first rows are on their way while slots and angles are worked out
      if (kind && (int)threadIdx.x < nt)
        slot[threadIdx.x] = cache_slot(a.c, __ldg(a.seq + t0 + threadIdx.x), __ldg(a.pos + t0 + threadIdx.x));
      for (int i = threadIdx.x; i < nt * np; i += blockDim.x) {
        const int tt = i / np, k = i - tt * np;
        row_cos_sin(a.r, fine_angles<TO, F8>(p, kind), k, __ldg(a.pos + t0 + tt), cs + tt * pad + angle_at<V>(k, pad),
                    si + tt * pad + angle_at<V>(k, pad));
      }
      __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const bool live = r0 + q * stride < rows;
      const int row = min(r0 + q * stride, rows - 1);
      const int t = quick_div(row, p.m_heads), h = row - t * p.hpb;
      float xa[V], xb[V];
      ra[q].get(xa);
      rb[q].get(xb);
      if (p.gain) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(xa[i], xa[i], fmaf(xb[i], xb[i], ss));
        const float inv = inverse_root(lanes_sum<kLanes>(ss) * (1.f / HD) + a.eps);
        const float* g = p.gain + (h0 + h) * p.gain_hs;
        float ga[V], gb[V];
        load_gain8(ga, g + ca * V);
        load_gain8(gb, g + cb * V);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          xa[i] = xa[i] * inv * ga[i];
          xb[i] = xb[i] * inv * gb[i];
        }
      }
      if (rot) unit_rotate<V>(xa, xb, u, rot, a.r.interleaved, cs + t * pad, si + t * pad, pad);
      if (kind == 0) {
        if (live) {
          TO* y = (TO*)a.y + (t0 + t) * a.yt + (h0 + h) * a.yh;
          store_v<TO, V>(y + ca * V, xa);
          store_v<TO, V>(y + cb * V, xb);
        }
        continue;
      }
      const int2 s = slot[t];
      const size_t base = (size_t)((h0 + h) << a.c.shift) + s.y;
      if constexpr (!F8) {
        if (live && s.x >= 0) {
          bf16* d = (bf16*)(kind == 2 ? a.c.v : a.c.k) + (size_t)s.x * a.c.pstride + base * HD;
          store_v<bf16, V>(d + ca * V, xa);
          store_v<bf16, V>(d + cb * V, xb);
        }
      } else {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) top = abs_max3(top, xa[i], xb[i]);
        const RowScale rs = row_scale(lanes_max<kLanes>(__float_as_uint(top)));
        if (live && s.x >= 0) {
          uint8_t* d = (uint8_t*)(kind == 2 ? a.c.v : a.c.k) + (size_t)s.x * a.c.pstride + base * HD;
          store_codes<V>(d + ca * V, xa, rs);
          store_codes<V>(d + cb * V, xb, rs);
          if (u == 0) ((kind == 2 ? a.c.vs : a.c.ks) + (size_t)s.x * a.c.sstride)[base] = rs.byte;
        }
      }
    }
  }
}

// Any even head_dim up to kMaxAnyDim and any alignment: a warp takes a row, element by element.
template <typename T, typename TO, bool F8>
__global__ void __launch_bounds__(kRowThreads) qkv_any_kernel(const __grid_constant__ QkvArgs a) {
  constexpr int kUnits = kMaxAnyDim / 64;
  const int lane = threadIdx.x & 31, units = a.hd / 2;
  int64_t row = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  int kind = 0;
  for (; kind < 3; ++kind) {
    const int64_t n = (int64_t)a.tokens * a.part[kind].heads;
    if (row < n) break;
    row -= n;
  }
  if (kind == 3) return;
  const QkvPart& p = a.part[kind];
  const int t = (int)(row / p.heads), h = (int)(row - (int64_t)t * p.heads), pos = __ldg(a.pos + t);
  const T* x = (const T*)p.x + t * p.ts + h * p.hs;
  float xa[kUnits], xb[kUnits], ss = 0.f, top = 0.f;
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const int u = lane + 32 * j;
    int ca, cb;
    unit_chunks<1>(u, p.rot, a.r.interleaved, &ca, &cb);
    xa[j] = u < units ? to_f32(x[ca]) : 0.f;
    xb[j] = u < units ? to_f32(x[cb]) : 0.f;
    ss = fmaf(xa[j], xa[j], fmaf(xb[j], xb[j], ss));
  }
  if (p.gain) {
    const float inv = inverse_root(warp_sum(ss) / (float)a.hd + a.eps);
    const float* g = p.gain + h * p.gain_hs;
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int u = lane + 32 * j;
      int ca, cb;
      unit_chunks<1>(u, p.rot, a.r.interleaved, &ca, &cb);
      if (u < units) {
        xa[j] = xa[j] * inv * __ldg(g + ca);
        xb[j] = xb[j] * inv * __ldg(g + cb);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const int u = lane + 32 * j;
    if (u < p.rot / 2) {
      float c, n;
      row_cos_sin(a.r, fine_angles<TO, F8>(p, kind), u, pos, &c, &n);
      const float e = xa[j], f = xb[j];
      xa[j] = e * c - f * n;
      xb[j] = f * c + e * n;
    }
    top = abs_max3(top, xa[j], xb[j]);
  }
  int2 s = make_int2(-1, 0);
  RowScale rs{};
  if (kind) {
    s = cache_slot(a.c, __ldg(a.seq + t), pos);
    if constexpr (F8) rs = row_scale(lanes_max<32>(__float_as_uint(top)));
    if (s.x < 0) return;
  }
  const size_t base = (size_t)(h << a.c.shift) + s.y;
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const int u = lane + 32 * j;
    int ca, cb;
    unit_chunks<1>(u, p.rot, a.r.interleaved, &ca, &cb);
    if (u >= units) break;
    if (kind == 0) {
      TO* y = (TO*)a.y + t * a.yt + h * a.yh;
      y[ca] = from_f32<TO>(xa[j]);
      y[cb] = from_f32<TO>(xb[j]);
    } else {
      const size_t at = (size_t)s.x * a.c.pstride + base * a.hd;
      void* pool = kind == 2 ? a.c.v : a.c.k;
      if constexpr (F8) {
        store_codes<1>((uint8_t*)pool + at + ca, &xa[j], rs);
        store_codes<1>((uint8_t*)pool + at + cb, &xb[j], rs);
      } else {
        ((bf16*)pool)[at + ca] = from_f32<bf16>(xa[j]);
        ((bf16*)pool)[at + cb] = from_f32<bf16>(xb[j]);
      }
    }
  }
  if constexpr (F8) {
    if (kind && lane == 0) ((kind == 2 ? a.c.vs : a.c.ks) + (size_t)s.x * a.c.sstride)[base] = rs.byte;
  }
}

template <typename T, typename TO, bool F8>
cudaError_t launch_qkv_any(const QkvArgs& a, cudaStream_t st) {
  const int64_t rows = (int64_t)a.tokens * ((int64_t)a.part[0].heads + a.part[1].heads + a.part[2].heads);
  const int64_t blocks = (rows + kRowThreads / 32 - 1) / (kRowThreads / 32);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_rows(qkv_any_kernel<T, TO, F8>, dim3((unsigned)blocks), dim3(kRowThreads), 0, 1, st, a);
}

template <typename T, typename TO, bool F8>
cudaError_t launch_qkv(QkvArgs& a, bool vec, cudaStream_t st) {
  if (!vec || (a.hd != 32 && a.hd != 64 && a.hd != 128 && a.hd != 256)) return launch_qkv_any<T, TO, F8>(a, st);
  const int per = a.hd / 16;                                        // threads of a row
  const int64_t all = (int64_t)a.tokens * per * (a.part[0].heads + a.part[1].heads + a.part[2].heads);
  const bool few = all < 1200LL * kRowThreads;                      // few tokens: heads spread over blocks
  int64_t blocks = 0;
  int most = 0;
  for (QkvPart& p : a.part) {
    if (!p.heads) {
      p.tpb = p.hpb = p.hblocks = 1;
      p.blocks = 0;
      continue;
    }
    const int64_t units = (int64_t)p.heads * per;
    p.tpb = few ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(kMaxTokBlock, 8 * kRowThreads / units));
    p.hpb = few ? std::min(p.heads, std::max(1, kRowThreads / per)) : p.heads;
    p.hblocks = (p.heads + p.hpb - 1) / p.hpb;
    const int64_t n = (int64_t)((a.tokens + p.tpb - 1) / p.tpb) * p.hblocks;
    if ((blocks += n) > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    p.blocks = (int)n;
    p.m_heads = div_magic(p.hpb);
    most = std::max(most, p.tpb * ((p.rot / 2 + 7) & ~7));
  }
  const size_t smem = (size_t)most * 2 * sizeof(float);
  const dim3 grid((unsigned)blocks), block(kRowThreads);
  switch (a.hd) {
    case 32: return launch_rows(qkv_kernel<T, TO, 32, F8>, grid, block, smem, 1, st, a);
    case 64: return launch_rows(qkv_kernel<T, TO, 64, F8>, grid, block, smem, 1, st, a);
    case 128: return launch_rows(qkv_kernel<T, TO, 128, F8>, grid, block, smem, 1, st, a);
    default:
      if constexpr (F8) return cudaErrorInvalidValue;               // (no cache holds rows of 256)
      else return launch_rows(qkv_kernel<T, TO, 256, F8>, grid, block, smem, 1, st, a);
  }
}

bool rot_vec(const spec_rope* r) { return !r || r->rot_dim % (r->interleaved ? 8 : 16) == 0; }
bool gain_vec(const float* g, int64_t hs) { return (reinterpret_cast<uintptr_t>(g) & 31u) == 0 && hs % 8 == 0; }
bool eps_ok(float eps) { return eps >= 0.f && std::isfinite(eps); }

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" {

int spec_rope_norm_rows(const void* x, int x_dtype, int64_t x_tok_stride, int64_t x_head_stride, void* y, int y_dtype,
                        int64_t y_tok_stride, int64_t y_head_stride, const int32_t* pos, int tokens, int heads,
                        int head_dim, const float* gain, int64_t gain_head_stride, float eps, const spec_rope* plan,
                        void* stream) {
  const std::string w = "spec_rope_norm_rows: ";
  if (tokens < 0 || heads < 1 || heads > 65535) return fail(SPEC_E_ARG, w + "bad tokens or heads");
  if (head_dim < 2 || head_dim % 2 || head_dim > kMaxAnyDim)
    return fail(SPEC_E_SHAPE, w + "head_dim must be even, in 2..512");
  if (!plan || !plan_ok(plan, head_dim)) return fail(SPEC_E_ARG, w + "null plan, or a rot_dim larger than the head");
  if (!is_io(x_dtype) || !is_io(y_dtype)) return fail(SPEC_E_ARG, w + "rows are fp32 or bf16");
  if (!eps_ok(eps)) return fail(SPEC_E_ARG, w + "eps must be finite and not negative");
  if (tokens == 0) return SPEC_OK;
  if (!x || !y || !pos || !gain) return fail(SPEC_E_ARG, w + "null pointer");
  if (x == y && (x_dtype != y_dtype || x_tok_stride != y_tok_stride || x_head_stride != y_head_stride))
    return fail(SPEC_E_ARG, w + "in place needs equal dtypes and strides");
  QkvArgs a{};
  QkvPart& p = a.part[0];
  p.x = x; p.ts = x_tok_stride; p.hs = x_head_stride; p.gain = gain; p.gain_hs = gain_head_stride;
  p.heads = heads; p.rot = plan->rot_dim;
  a.y = y; a.yt = y_tok_stride; a.yh = y_head_stride; a.pos = pos; a.tokens = tokens; a.hd = head_dim; a.eps = eps;
  a.r = *plan;
  const bool vec = rot_vec(plan) && vec_ok(x, x_tok_stride, x_head_stride, x_dtype) &&
                   vec_ok(y, y_tok_stride, y_head_stride, y_dtype) && gain_vec(gain, gain_head_stride);
  cudaStream_t st = (cudaStream_t)stream;
  const bool xi = x_dtype == SPEC_DTYPE_F32, yi = y_dtype == SPEC_DTYPE_F32;
  cudaError_t e;
  if (xi) e = yi ? launch_qkv<float, float, false>(a, vec, st) : launch_qkv<float, bf16, false>(a, vec, st);
  else e = yi ? launch_qkv<bf16, float, false>(a, vec, st) : launch_qkv<bf16, bf16, false>(a, vec, st);
  return done(e, "spec_rope_norm_rows");
}

int spec_qkv_append(const spec_kv_cache* cache, const void* q, int64_t q_tok_stride, int64_t q_head_stride,
                    const void* k, int64_t k_tok_stride, int64_t k_head_stride, const void* v, int64_t v_tok_stride,
                    int64_t v_head_stride, int dtype, const int32_t* seq, const int32_t* pos, int tokens, int n_heads,
                    const spec_rope* plan, const float* q_gain, const float* k_gain, float eps, void* q_out,
                    int64_t out_tok_stride, int64_t out_head_stride, void* stream) {
  const char* who = "spec_qkv_append";
  const std::string w = std::string(who) + ": ";
  const int rc = check_cache(cache, who);
  if (rc) return rc;
  if (tokens < 0 || !is_io(dtype)) return fail(SPEC_E_ARG, w + "bad tokens, or rows not fp32 or bf16");
  if (n_heads < 1 || n_heads > 65535) return fail(SPEC_E_ARG, w + "bad n_heads");
  if (plan && !plan_ok(plan, cache->head_dim)) return fail(SPEC_E_ARG, w + "the plan's rot_dim does not fit the head");
  if (!eps_ok(eps)) return fail(SPEC_E_ARG, w + "eps must be finite and not negative");
  if (tokens == 0) return SPEC_OK;
  if (!q || !k || !v || !seq || !pos || !q_out) return fail(SPEC_E_ARG, w + "null pointer");
  if (q == q_out && (dtype != SPEC_DTYPE_BF16 || q_tok_stride != out_tok_stride || q_head_stride != out_head_stride))
    return fail(SPEC_E_ARG, w + "in place needs bf16 rows and equal strides");
  QkvArgs a{};
  const int rot = plan ? plan->rot_dim : 0;
  a.part[0] = {q, q_tok_stride, q_head_stride, q_gain, 0, n_heads, rot, 0, 0, 0, 0, 0};
  a.part[1] = {k, k_tok_stride, k_head_stride, k_gain, 0, cache->n_kv_heads, rot, 0, 0, 0, 0, 0};
  a.part[2] = {v, v_tok_stride, v_head_stride, nullptr, 0, cache->n_kv_heads, 0, 0, 0, 0, 0, 0};
  a.c = cache_args(*cache);
  a.y = q_out; a.yt = out_tok_stride; a.yh = out_head_stride;
  a.seq = seq; a.pos = pos; a.tokens = tokens; a.hd = cache->head_dim; a.eps = eps;
  if (plan) a.r = *plan;
  const bool vec = rot_vec(plan) && vec_ok(q, q_tok_stride, q_head_stride, dtype) &&
                   vec_ok(k, k_tok_stride, k_head_stride, dtype) && vec_ok(v, v_tok_stride, v_head_stride, dtype) &&
                   vec_ok(q_out, out_tok_stride, out_head_stride, SPEC_DTYPE_BF16) && gain_vec(q_gain, 0) &&
                   gain_vec(k_gain, 0);
  cudaStream_t st = (cudaStream_t)stream;
  const bool f8 = cache->dtype == SPEC_DTYPE_E4M3;
  cudaError_t e;
  if (dtype == SPEC_DTYPE_F32) e = f8 ? launch_qkv<float, bf16, true>(a, vec, st) : launch_qkv<float, bf16, false>(a, vec, st);
  else e = f8 ? launch_qkv<bf16, bf16, true>(a, vec, st) : launch_qkv<bf16, bf16, false>(a, vec, st);
  return done(e, who);
}

}  // extern "C"
