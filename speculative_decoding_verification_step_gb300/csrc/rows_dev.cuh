// Row helpers of the paged-cache operators (kvrows.cu, qkvrows.cu): rotation by
// turns, wide loads and stores, 8-bit encoding, cache slots, argument checks.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "common.cuh"
#include "paged.h"

namespace sv {

namespace {

constexpr int kRowThreads = 128;
constexpr int kScaleMax = 60;     // |e| of an 8-bit row's power of two
constexpr int kRowBatch = 2;      // rows of a thread in flight
constexpr int kMaxTokBlock = 16;  // tokens of a block

SV_DEV void turn_cos_sin(const spec_rope& r, int i, int pos, float sign, float* cos_out, float* sin_out) {
  const uint64_t ph = r.turn[i] * (uint64_t)(int64_t)pos;
  float s, c;
  sincospif((float)(int32_t)(ph >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31
  *cos_out = c * r.mscale;
  *sin_out = s * r.mscale * sign;
}
// The same with what the fraction's rounding to fp32 leaves (up to 9e-8 of a radian) put back by
// the sine's and cosine's slopes: normed rows, whose 8-bit codes are as often the wrong
// neighbour as the row before the rounding is off.
SV_DEV void turn_cos_sin_fine(const spec_rope& r, int i, int pos, float* cos_out, float* sin_out) {
  const int turn = (int)((r.turn[i] * (uint64_t)(int64_t)pos) >> 32);
  const float f = (float)turn, left = (float)(turn - __float2int_rz(f)) * (4.656612873077393e-10f * 3.1415927f);
  float s, c;
  sincospif(f * 4.656612873077393e-10f, &s, &c);
  *cos_out = fmaf(-s, left, c) * r.mscale;
  *sin_out = fmaf(c, left, s) * r.mscale;
}
// n / d for n * d < 2^32, by m = ceil(2^32 / d) (0 for d = 1).
SV_DEV int quick_div(int n, uint32_t m) { return m ? (int)__umulhi((uint32_t)n, m) : n; }
[[maybe_unused]] uint32_t div_magic(int64_t d) { return d <= 1 ? 0u : (uint32_t)(((1ull << 32) + d - 1) / d); }

// Two fp32 values in a register pair, one instruction for both.
SV_DEV uint64_t pair2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
SV_DEV void split2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
SV_DEV uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
SV_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Largest magnitude; a NaN stays one.
SV_DEV float abs_max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}

// V adjacent elements as they lie (held while their loads are in flight), and
// as fp32.
template <typename T, int V>
struct RawV {
  static constexpr int n = V == 8 ? (int)sizeof(T) / 2 : 1;
  uint4 w[V == 8 ? n : 1];
  T x;
  SV_DEV void load(const T* p) {
    if constexpr (V == 8) {
#pragma unroll
      for (int i = 0; i < n; ++i) w[i] = *(reinterpret_cast<const uint4*>(p) + i);
    } else {
      x = *p;
    }
  }
  SV_DEV void get(float (&y)[V]) const {
    if constexpr (V == 8 && sizeof(T) == 2) {
      y[0] = bf16lo(w[0].x); y[1] = bf16hi(w[0].x); y[2] = bf16lo(w[0].y); y[3] = bf16hi(w[0].y);
      y[4] = bf16lo(w[0].z); y[5] = bf16hi(w[0].z); y[6] = bf16lo(w[0].w); y[7] = bf16hi(w[0].w);
    } else if constexpr (V == 8) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        y[4 * i] = __uint_as_float(w[i].x); y[4 * i + 1] = __uint_as_float(w[i].y);
        y[4 * i + 2] = __uint_as_float(w[i].z); y[4 * i + 3] = __uint_as_float(w[i].w);
      }
    } else {
      y[0] = to_f32(x);
    }
  }
};
SV_DEV uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T, int V>
SV_DEV void store_v(T* p, const float (&x)[V]) {
  if constexpr (V == 8 && sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
  } else if constexpr (V == 8) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = from_f32<T>(x[i]);
  }
}

// Unit u of a head of `dim` elements, in chunks of V: two chunks a, b that
// are rotated together.  Halves: chunk u with chunk u + rot/2V; the rest, and
// interleaved pairs: neighbours 2u, 2u + 1.
template <int V>
SV_DEV void unit_chunks(int u, int rot, int inter, int* a, int* b) {
  const int half = rot / (2 * V);
  if (!inter && u < half) {
    *a = u;
    *b = u + half;
  } else {
    *a = 2 * u;
    *b = 2 * u + 1;
  }
}
// Place of angle k among a token's `pad` in shared memory.  Units of eight read theirs as two
// quads: first quads lie side by side, then the second, so that adjacent lanes find them in
// distinct banks.
template <int V>
SV_DEV int angle_at(int k, int pad) {
  return V == 1 ? k : (k & 4 ? pad / 2 : 0) + ((k >> 3) << 2) + (k & 3);
}
// Rotates the two chunks of unit u (xa, xb) by the token's cosines and sines.
template <int V>
SV_DEV void unit_rotate(float (&xa)[V], float (&xb)[V], int u, int rot, int inter, const float* co, const float* si, int pad) {
  if constexpr (V == 1) {
    if (u >= rot / 2) return;
    const float c = co[u], n = si[u], p = xa[0], q = xb[0];
    xa[0] = p * c - q * n;
    xb[0] = q * c + p * n;
  } else {
    // the unit's eight angles: of elements V u .. (halves), or of pairs 8 u .. (interleaved)
    if (u * 2 * V >= rot) return;
    float c[8], n[8];
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const int at = u * 4 + (i ? pad / 2 : 0);
      const float4 x = *reinterpret_cast<const float4*>(co + at), y = *reinterpret_cast<const float4*>(si + at);
      c[i] = x.x; c[i + 1] = x.y; c[i + 2] = x.z; c[i + 3] = x.w;
      n[i] = y.x; n[i + 1] = y.y; n[i + 2] = y.z; n[i + 3] = y.w;
    }
    if (!inter) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const uint64_t p = pair2(xa[i], xa[i + 1]), q = pair2(xb[i], xb[i + 1]);
        const uint64_t cc = pair2(c[i], c[i + 1]), nn = pair2(n[i], n[i + 1]), mn = pair2(-n[i], -n[i + 1]);
        split2(fma2(q, mn, mul2(p, cc)), xa[i], xa[i + 1]);
        split2(fma2(p, nn, mul2(q, cc)), xb[i], xb[i + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const uint64_t x = pair2(xa[i], xa[i + 1]), y = pair2(xa[i + 1], xa[i]);
        split2(fma2(y, pair2(-n[i / 2], n[i / 2]), mul2(x, pair2(c[i / 2], c[i / 2]))), xa[i], xa[i + 1]);
      }
      if ((2 * u + 1) * V < rot) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const uint64_t x = pair2(xb[i], xb[i + 1]), y = pair2(xb[i + 1], xb[i]);
          const float cc = c[4 + i / 2], nn = n[4 + i / 2];
          split2(fma2(y, pair2(-nn, nn), mul2(x, pair2(cc, cc))), xb[i], xb[i + 1]);
        }
      }
    }
  }
}

// The power of two of an 8-bit row whose largest magnitude has the bits m (infinities
// and NaN sort above every number).
struct RowScale {
  float f;         // 2^-e
  bool bad;        // a row of NaN
  uint8_t byte;    // e + 127, or 255
};
SV_DEV RowScale row_scale(uint32_t m) {
  // 448 = 1.75 * 2^8: smallest e with magnitude <= 448 * 2^e
  int e = m == 0 ? 0 : (int)(m >> 23) - 127 - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
  RowScale r;
  r.bad = m >= 0x7f800000u || e > kScaleMax;
  e = max(e, -kScaleMax);
  r.f = r.bad ? 0.f : __uint_as_float((uint32_t)(127 - e) << 23);
  r.byte = r.bad ? (uint8_t)255 : (uint8_t)(e + 127);
  return r;
}
// V adjacent elements of such a row as codes.
template <int V>
SV_DEV void store_codes(uint8_t* p, const float* y, const RowScale& r) {
  if constexpr (V == 8) {
    const uint64_t ff = pair2(r.f, r.f);
    uint32_t w[2];
#pragma unroll
    for (int w4 = 0; w4 < 2; ++w4) {
      float2 lo, hi;
      split2(mul2(pair2(y[4 * w4], y[4 * w4 + 1]), ff), lo.x, lo.y);
      split2(mul2(pair2(y[4 * w4 + 2], y[4 * w4 + 3]), ff), hi.x, hi.y);
      w[w4] = __nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3) |
              ((uint32_t)__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3) << 16);
      if (r.bad) w[w4] = 0u;
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
    p[0] = r.bad ? (uint8_t)0 : (uint8_t)__nv_cvt_float_to_fp8(y[0] * r.f, __NV_SATFINITE, __NV_E4M3);
  }
}

// ------------------------------------------------------------ cache slots
struct CacheArgs {
  void* k;
  void* v;
  uint8_t* ks;
  uint8_t* vs;
  int pages, shift, hkv, hd, seqs, max_pages;
  int64_t pstride, sstride, tstride;
  const int32_t* table;
};

[[maybe_unused]] CacheArgs cache_args(const spec_kv_cache& c) {
  CacheArgs a{};
  a.k = c.k; a.v = c.v; a.ks = c.k_scale; a.vs = c.v_scale;
  a.pages = c.pages; a.hkv = c.n_kv_heads; a.hd = c.head_dim; a.seqs = c.seqs; a.max_pages = c.max_pages;
  a.shift = 0;
  while ((1 << a.shift) < c.page_size) ++a.shift;
  a.pstride = c.page_stride ? c.page_stride : (int64_t)c.n_kv_heads * c.page_size * c.head_dim;
  a.sstride = c.scale_page_stride ? c.scale_page_stride : (int64_t)c.n_kv_heads * c.page_size;
  a.tstride = c.table_stride ? c.table_stride : c.max_pages;
  a.table = c.table;
  return a;
}

// (page, slot) of a token, or page -1 when it has none.
SV_DEV int2 cache_slot(const CacheArgs& c, int seq, int pos) {
  if (seq < 0 || seq >= c.seqs || pos < 0 || (pos >> c.shift) >= c.max_pages) return make_int2(-1, 0);
  const int page = __ldg(c.table + seq * c.tstride + (pos >> c.shift));
  if (page < 0 || page >= c.pages) return make_int2(-1, 0);
  return make_int2(page, pos & ((1 << c.shift) - 1));
}

[[maybe_unused]] int fail(int code, const std::string& msg) {
  set_thread_error(msg);
  return code;
}
[[maybe_unused]] int done(cudaError_t e, const char* who) {
  return e == cudaSuccess ? SPEC_OK : fail(SPEC_E_CUDA, std::string(who) + ": " + cudaGetErrorString(e));
}
[[maybe_unused]] bool is_io(int dtype) { return dtype == SPEC_DTYPE_F32 || dtype == SPEC_DTYPE_BF16; }
[[maybe_unused]] int esize(int dtype) { return dtype == SPEC_DTYPE_F32 ? 4 : 2; }
// Base and strides that allow 16-byte accesses of 8 elements.
[[maybe_unused]] bool vec_ok(const void* p, int64_t ts, int64_t hs, int dtype) {
  const int64_t m = 16 / esize(dtype);
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ts % m == 0 && hs % m == 0;
}
[[maybe_unused]] bool plan_ok(const spec_rope* r, int hd) {
  return r->rot_dim >= 2 && r->rot_dim % 2 == 0 && r->rot_dim <= hd && r->rot_dim <= SPEC_ROPE_MAX_DIM;
}

}  // namespace

}  // namespace sv
