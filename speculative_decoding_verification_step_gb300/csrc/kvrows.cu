// Row operators of a paged KV cache: rotary positions, the write of new rows
// (with rotation and 8-bit encoding) and their read-back.
//
// All three move each byte once and are bound by HBM for prompts and by
// launch and dependent-load latency for a verify step's few rows; the split
// is (tokens of a block) x (heads), with what belongs to a token (its angles,
// its cache slot) worked out once in shared memory.
//
// Angles.  A pair's turns per position are kept as a 64-bit fraction F of a
// turn; position p turns it by p * F modulo 2^64, exact integer arithmetic,
// so the reduced angle of position 10^6 is as good as that of position 1 (a
// fp32 product p * f would be off by 0.06 rad there) without 64-bit floats.
// The top 32 bits, in units of pi * 2^-31, go to sincospif.
//
// 8-bit rows.  value = e4m3 code * 2^e, one e per row, the smallest that
// keeps the row within 448.  Scaling by a power of two is exact, so a value
// is rounded once, to e4m3 (half a step, 2^-4 relative; below 2^(e-6) the
// step is 2^(e-9) absolute), and code * 2^e is exact in bf16.
//
// Measured.  Rotation of 16381 bf16 rows of 40 heads of 64 30 us (5.7 TB/s, 83%
// of a copy's rate); a step's 6 tokens 2.2 us of the GPU's time.  Append of
// 16000 fp32 rows of 8 heads of 128 to bf16 34 us (86%), of bf16 rows to 8-bit
// 25 us (4.0 TB/s).  The latter fills 56% of the issue slots and 35% of DRAM's
// rate: its 4000 blocks run in 3.3 waves, and each starts with dependent loads
// (sequence and position, then the table), sines and a barrier.  Read-back of
// 16 x 16384 8-bit rows 191 us (6.6 TB/s, 97%).
// Tiles of 4 x 128 units a block, two rows of a thread in flight and the slots
// looked up behind the loads took append from 34 to 24 us and rotation from 33
// to 29; more rows in flight spilled or left fewer blocks (26 and 30 us).
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "common.cuh"
#include "paged.h"
#include "rows_dev.cuh"

namespace sv {

namespace {

// ------------------------------------------------------------------ rotary
struct RopeArgs {
  const void* x;
  void* y;
  int64_t xt, xh, yt, yh;
  const int32_t* pos;
  int tokens, heads, hd, tpb, hpb;
  uint32_t m_per, m_unit;   // quick_div of a block's units by those of a token, of a head
  float sign;
  spec_rope r;
};

// Block (x, y): tokens x * tpb .., heads y * hpb ..; a thread takes units of
// two chunks (V = 8: 16-byte accesses; V = 1 for odd sizes and alignments).
template <typename TI, typename TO, int V>
__global__ void __launch_bounds__(kRowThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ __align__(16) float cs[];   // cosines [tpb][pad], sines [tpb][pad]
  const int rot = a.r.rot_dim, np = rot / 2, pad = (np + 7) & ~7;
  const int t0 = blockIdx.x * a.tpb, nt = min(a.tpb, a.tokens - t0);
  const int h0 = blockIdx.y * a.hpb, nh = min(a.hpb, a.heads - h0);
  float* const si = cs + a.tpb * pad;
  // (a block's last heads may be fewer: units past them are skipped)
  const int U = a.hd / (2 * V), per = a.hpb * U, total = nt * per;
  for (int e = threadIdx.x, pass = 0; pass == 0 || e < total; e += blockDim.x, ++pass) {
    const int t = quick_div(e, a.m_per), w = e - t * per, h = quick_div(w, a.m_unit), u = w - h * U;
    const bool live = e < total && h < nh;
    int ca = 0, cb = 0;
    unit_chunks<V>(u, rot, a.r.interleaved, &ca, &cb);
    RawV<TI, V> ra, rb;
    if (live) {
      const TI* x = (const TI*)a.x + (t0 + t) * a.xt + (h0 + h) * a.xh;
      ra.load(x + ca * V);
      rb.load(x + cb * V);
    }
    if (pass == 0) {   // the first loads are on their way while the angles are worked out
      for (int i = threadIdx.x; i < nt * np; i += blockDim.x) {
        const int tt = i / np, k = i - tt * np;
        turn_cos_sin(a.r, k, __ldg(a.pos + t0 + tt), a.sign, cs + tt * pad + angle_at<V>(k, pad),
                     si + tt * pad + angle_at<V>(k, pad));
      }
      __syncthreads();
    }
    if (live) {
      TO* y = (TO*)a.y + (t0 + t) * a.yt + (h0 + h) * a.yh;
      float xa[V], xb[V];
      ra.get(xa);
      rb.get(xb);
      unit_rotate<V>(xa, xb, u, rot, a.r.interleaved, cs + t * pad, si + t * pad, pad);
      store_v<TO, V>(y + ca * V, xa);
      store_v<TO, V>(y + cb * V, xb);
    }
  }
}

template <typename TI, typename TO>
cudaError_t launch_rope(const RopeArgs& a, bool vec, cudaStream_t st) {
  const dim3 grid((a.tokens + a.tpb - 1) / a.tpb, (a.heads + a.hpb - 1) / a.hpb);
  const size_t smem = (size_t)a.tpb * ((a.r.rot_dim / 2 + 7) & ~7) * 2 * sizeof(float);
  return vec ? launch_rows(rope_kernel<TI, TO, 8>, grid, dim3(kRowThreads), smem, 1, st, a)
             : launch_rows(rope_kernel<TI, TO, 1>, grid, dim3(kRowThreads), smem, 1, st, a);
}

// ------------------------------------------------------------------ append
struct AppendArgs {
  CacheArgs c;
  const void* k;
  const void* v;
  int64_t kt, kh, vt, vh;
  const int32_t* seq;
  const int32_t* pos;
  int tokens, tpb;
  uint32_t m_heads;  // quick_div by the KV heads
  spec_rope r;       // rot_dim 0: no rotation
};

// Blocks of K and of V (z) differ in the rotation only.  A row (token, head) is held by HD / (2 V UPL) adjacent lanes, UPL
// units of two chunks each: the row's largest magnitude is a shuffle away and
// the row is read and written once.  V = 1 serves rotated parts that are no
// multiple of 16 and unaligned inputs.
template <typename T, int HD, int V, bool F8>
__global__ void __launch_bounds__(kRowThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kUnits = HD / (2 * V), kLanes = kUnits < 32 ? kUnits : 32, kUpl = kUnits / kLanes;
  constexpr int kBatch = V == 8 ? kRowBatch : 1;
  extern __shared__ __align__(16) float cs[];   // cosines [tpb][pad], sines [tpb][pad]
  __shared__ int2 slot[kMaxTokBlock];
  const int isv = blockIdx.z;
  const int rot = isv ? 0 : a.r.rot_dim, np = rot / 2, pad = (np + 7) & ~7;
  const int t0 = blockIdx.x * a.tpb, nt = min(a.tpb, a.tokens - t0);
  float* const si = cs + a.tpb * pad;
  const T* const src = (const T*)(isv ? a.v : a.k) + t0 * (isv ? a.vt : a.kt);
  const int64_t ts = isv ? a.vt : a.kt, hs = isv ? a.vh : a.kh;
  // in small calls grid.y blocks share a token's rows
  const int rows = nt * a.c.hkv;
  const int stride = (int)(blockDim.x * gridDim.y) / kLanes;
  const int lane = threadIdx.x % kLanes;
  int ca[kUpl], cb[kUpl];
#pragma unroll
  for (int j = 0; j < kUpl; ++j) unit_chunks<V>(j * kLanes + lane, rot, a.r.interleaved, &ca[j], &cb[j]);
  for (int r0 = (int)(blockIdx.y * blockDim.x + threadIdx.x) / kLanes, pass = 0;; r0 += kBatch * stride, ++pass) {
    // whole warps stay together for the shuffles
    if (pass && !__any_sync(0xffffffffu, r0 < rows)) break;
    RawV<T, V> ra[kBatch][kUpl], rb[kBatch][kUpl];   // rows in flight
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int row = min(r0 + q * stride, rows - 1);
      const int t = quick_div(row, a.m_heads), h = row - t * a.c.hkv;
      const T* x = src + t * ts + h * hs;
#pragma unroll
      for (int j = 0; j < kUpl; ++j) {
        ra[q][j].load(x + ca[j] * V);
        rb[q][j].load(x + cb[j] * V);
      }
    }
    if (pass == 0) {   // the first rows are on their way while slots and angles are worked out
      if ((int)threadIdx.x < nt)
        slot[threadIdx.x] = cache_slot(a.c, __ldg(a.seq + t0 + threadIdx.x), __ldg(a.pos + t0 + threadIdx.x));
      for (int i = threadIdx.x; i < nt * np; i += blockDim.x) {
        const int tt = i / np, k = i - tt * np;
        turn_cos_sin(a.r, k, __ldg(a.pos + t0 + tt), 1.f, cs + tt * pad + angle_at<V>(k, pad),
                     si + tt * pad + angle_at<V>(k, pad));
      }
      __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
    const bool live = r0 + q * stride < rows;
    const int row = min(r0 + q * stride, rows - 1);
    const int t = quick_div(row, a.m_heads), h = row - t * a.c.hkv;
    const int2 s = slot[t];
    float xa[kUpl][V], xb[kUpl][V];
#pragma unroll
    for (int j = 0; j < kUpl; ++j) {
      ra[q][j].get(xa[j]);
      rb[q][j].get(xb[j]);
      if (rot) unit_rotate<V>(xa[j], xb[j], j * kLanes + lane, rot, a.r.interleaved, cs + t * pad, si + t * pad, pad);
    }
    const size_t base = (size_t)(h << a.c.shift) + s.y;
    if constexpr (!F8) {
      if (live && s.x >= 0) {
        bf16* d = (bf16*)(isv ? a.c.v : a.c.k) + (size_t)s.x * a.c.pstride + base * HD;
#pragma unroll
        for (int j = 0; j < kUpl; ++j) {
          store_v<bf16, V>(d + ca[j] * V, xa[j]);
          store_v<bf16, V>(d + cb[j] * V, xb[j]);
        }
      }
    } else {
      float top = 0.f;   // largest magnitude; as bits, infinities and NaN sort above every number
#pragma unroll
      for (int j = 0; j < kUpl; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) top = abs_max3(top, xa[j][i], xb[j][i]);
      uint32_t m = __float_as_uint(top);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const RowScale rs = row_scale(m);
      if (live && s.x >= 0) {
        uint8_t* d = (uint8_t*)(isv ? a.c.v : a.c.k) + (size_t)s.x * a.c.pstride + base * HD;
#pragma unroll
        for (int j = 0; j < kUpl; ++j)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float* y = half ? xb[j] : xa[j];
            uint8_t* p = d + (half ? cb[j] : ca[j]) * V;
            store_codes<V>(p, y, rs);
          }
        if (lane == 0) {
          uint8_t* sc = (isv ? a.c.vs : a.c.ks) + (size_t)s.x * a.c.sstride + base;
          *sc = rs.byte;
        }
      }
    }
    }
  }
}

template <typename T, int HD, int V>
cudaError_t launch_append(const AppendArgs& a, bool f8, int ysplit, cudaStream_t st) {
  const dim3 grid((a.tokens + a.tpb - 1) / a.tpb, ysplit, 2);   // z: K, V
  const size_t smem = (size_t)a.tpb * ((a.r.rot_dim / 2 + 7) & ~7) * 2 * sizeof(float);
  return f8 ? launch_rows(append_kernel<T, HD, V, true>, grid, dim3(kRowThreads), smem, 1, st, a)
            : launch_rows(append_kernel<T, HD, V, false>, grid, dim3(kRowThreads), smem, 1, st, a);
}
template <typename T>
cudaError_t launch_append_t(const AppendArgs& a, bool vec, bool f8, int ysplit, cudaStream_t st) {
  switch (a.c.hd) {
    case 32: return vec ? launch_append<T, 32, 8>(a, f8, ysplit, st) : launch_append<T, 32, 1>(a, f8, ysplit, st);
    case 64: return vec ? launch_append<T, 64, 8>(a, f8, ysplit, st) : launch_append<T, 64, 1>(a, f8, ysplit, st);
    default: return vec ? launch_append<T, 128, 8>(a, f8, ysplit, st) : launch_append<T, 128, 1>(a, f8, ysplit, st);
  }
}

// ------------------------------------------------------------------ gather
struct GatherArgs {
  CacheArgs c;
  const int32_t* seq;
  const int32_t* pos;
  void* k;
  void* v;
  int tokens, tpb;
  uint32_t m_per;    // quick_div of a block's chunks by those of a token
};

// A thread takes 16 bytes of a row (8 bf16 values or 16 codes).
template <typename TO, bool F8>
__global__ void __launch_bounds__(kRowThreads) gather_kernel(const __grid_constant__ GatherArgs a) {
  constexpr int kVals = F8 ? 16 : 8;
  __shared__ int2 slot[kMaxTokBlock];
  const int t0 = blockIdx.x * a.tpb, nt = min(a.tpb, a.tokens - t0);
  if ((int)threadIdx.x < nt)
    slot[threadIdx.x] = cache_slot(a.c, __ldg(a.seq + t0 + threadIdx.x), __ldg(a.pos + t0 + threadIdx.x));
  __syncthreads();
  const bool isv = blockIdx.y == 1 || !a.k;
  const void* pool = isv ? a.c.v : a.c.k;
  const uint8_t* scales = isv ? a.c.vs : a.c.ks;
  TO* out = (TO*)(isv ? a.v : a.k);
  const int nc = a.c.hd / kVals, cshift = 31 - __clz(nc), per = a.c.hkv << cshift;
#pragma unroll 4
  for (int e = threadIdx.x; e < nt * per; e += blockDim.x) {
    const int t = quick_div(e, a.m_per), w = e - t * per, h = w >> cshift, c = w & (nc - 1);
    const int2 s = slot[t];
    const size_t row = (size_t)(h << a.c.shift) + s.y;
    uint4 x = make_uint4(0, 0, 0, 0);
    uint32_t sb = 127;
    if (s.x >= 0) {
      x = ld_stream((const uint8_t*)pool + ((size_t)s.x * a.c.pstride + row * a.c.hd) * (F8 ? 1 : 2) + c * 16);
      if constexpr (F8) sb = __ldg(scales + (size_t)s.x * a.c.sstride + row);
    }
    TO* d = out + ((size_t)(t0 + t) * a.c.hkv + h) * a.c.hd + c * kVals;
    if constexpr (!F8) {
      if constexpr (sizeof(TO) == 2) {
        __stcs(reinterpret_cast<uint4*>(d), x);
      } else {
        __stcs(reinterpret_cast<float4*>(d), make_float4(bf16lo(x.x), bf16hi(x.x), bf16lo(x.y), bf16hi(x.y)));
        __stcs(reinterpret_cast<float4*>(d) + 1, make_float4(bf16lo(x.z), bf16hi(x.z), bf16lo(x.w), bf16hi(x.w)));
      }
    } else {
      const float f = row_power(sb);
      const uint32_t in[4] = {x.x, x.y, x.z, x.w};
      float y[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(in[i / 2] >> (16 * (i & 1))), __NV_E4M3);
        const float2 v2 = __half22float2(*reinterpret_cast<const __half2*>(&hr));
        y[2 * i] = v2.x * f;
        y[2 * i + 1] = v2.y * f;
      }
      if constexpr (sizeof(TO) == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          __stcs(reinterpret_cast<uint4*>(d) + i,
                 make_uint4(pack2(y[8 * i], y[8 * i + 1]), pack2(y[8 * i + 2], y[8 * i + 3]),
                            pack2(y[8 * i + 4], y[8 * i + 5]), pack2(y[8 * i + 6], y[8 * i + 7])));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __stcs(reinterpret_cast<float4*>(d) + i, make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]));
      }
    }
  }
}

}  // namespace

int check_cache(const spec_kv_cache* c, const char* who) {
  const std::string w = std::string(who) + ": ";
  if (!c || !c->k || !c->v || !c->table) return fail(SPEC_E_ARG, w + "null cache, pool or table");
  if (c->dtype != SPEC_DTYPE_BF16 && c->dtype != SPEC_DTYPE_E4M3)
    return fail(SPEC_E_ARG, w + "the cache is bf16 or e4m3");
  const bool f8 = c->dtype == SPEC_DTYPE_E4M3;
  if (f8 && (!c->k_scale || !c->v_scale)) return fail(SPEC_E_ARG, w + "an e4m3 cache needs k_scale and v_scale");
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128)
    return fail(SPEC_E_SHAPE, w + "head_dim must be 32, 64 or 128");
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    return fail(SPEC_E_SHAPE, w + "page_size must be a power of two in 16..256");
  if (c->pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 1024 || c->seqs < 1 || c->max_pages < 1)
    return fail(SPEC_E_ARG, w + "pages, n_kv_heads (at most 1024), seqs and max_pages must be positive");
  if ((int64_t)c->max_pages * c->page_size > 0x7fffff00LL)
    return fail(SPEC_E_ARG, w + "max_pages * page_size exceeds 2^31 positions");
  const int64_t row = (int64_t)c->n_kv_heads * c->page_size;
  if ((c->page_stride && c->page_stride < row * c->head_dim) || (c->scale_page_stride && c->scale_page_stride < row) ||
      (c->table_stride && c->table_stride < c->max_pages))
    return fail(SPEC_E_ARG, w + "a stride is smaller than what it steps over");
  if ((reinterpret_cast<uintptr_t>(c->k) & 15u) || (reinterpret_cast<uintptr_t>(c->v) & 15u) ||
      (c->page_stride * (f8 ? 1 : 2)) % 16 != 0)
    return fail(SPEC_E_ARG, w + "pools and page strides must be 16-byte aligned");
  if (f8 && ((reinterpret_cast<uintptr_t>(c->k_scale) & 15u) || (reinterpret_cast<uintptr_t>(c->v_scale) & 15u) ||
             c->scale_page_stride % 16 != 0))
    return fail(SPEC_E_ARG, w + "scales and their page stride must be 16-byte aligned");
  return SPEC_OK;
}

}  // namespace sv

using namespace sv;

extern "C" {

int spec_rope_plan(const spec_rope_desc* d, spec_rope* out) {
  if (!d || !out) return fail(SPEC_E_ARG, "spec_rope_plan: null argument");
  if (d->rot_dim < 2 || d->rot_dim % 2 || d->rot_dim > SPEC_ROPE_MAX_DIM)
    return fail(SPEC_E_ARG, "spec_rope_plan: rot_dim must be even, in 2..256");
  if (!(d->theta > 0.0) || !std::isfinite(d->theta)) return fail(SPEC_E_ARG, "spec_rope_plan: theta must be positive");
  if (d->scaling < SPEC_ROPE_PLAIN || d->scaling > SPEC_ROPE_PARTS)
    return fail(SPEC_E_ARG, "spec_rope_plan: unknown scaling");
  if (d->scaling != SPEC_ROPE_PLAIN && !(d->factor > 0.0 && std::isfinite(d->factor)))
    return fail(SPEC_E_ARG, "spec_rope_plan: factor must be positive");
  if (d->scaling == SPEC_ROPE_NTK && d->rot_dim < 4)
    return fail(SPEC_E_ARG, "spec_rope_plan: the grown theta needs rot_dim >= 4");
  if (d->scaling == SPEC_ROPE_PARTS && !(d->orig_ctx > 0.0 && d->high > d->low))
    return fail(SPEC_E_ARG, "spec_rope_plan: scaling by parts needs orig_ctx > 0 and high > low");
  if (!(d->mscale >= 0.0) || !std::isfinite((float)d->mscale)) return fail(SPEC_E_ARG, "spec_rope_plan: bad mscale");
  const double kTurn = 6.283185307179586476925286766559;
  spec_rope r{};
  r.rot_dim = d->rot_dim;
  r.interleaved = d->interleaved ? 1 : 0;
  r.mscale = d->mscale == 0.0 ? 1.f : (float)d->mscale;
  double theta = d->theta;
  if (d->scaling == SPEC_ROPE_NTK) theta *= std::pow(d->factor, (double)d->rot_dim / (d->rot_dim - 2));
  for (int i = 0; i < d->rot_dim / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / d->rot_dim);
    if (d->scaling == SPEC_ROPE_LINEAR) f /= d->factor;
    if (d->scaling == SPEC_ROPE_PARTS) {
      const double turns = d->orig_ctx * f / kTurn;
      const double keep = std::min(1.0, std::max(0.0, (turns - d->low) / (d->high - d->low)));
      f *= keep + (1.0 - keep) / d->factor;
    }
    double whole;
    const double frac = std::modf(f / kTurn, &whole);   // whole turns turn nothing
    // 2^64 * frac in two halves: a double holds 53 of the 64 bits
    const double hi = std::floor(frac * 4294967296.0);
    const double lo = std::floor((frac * 4294967296.0 - hi) * 4294967296.0 + 0.5);
    r.turn[i] = ((uint64_t)hi << 32) + (uint64_t)lo;
  }
  *out = r;
  return SPEC_OK;
}

int spec_rope_rows(const void* x, int x_dtype, int64_t x_tok_stride, int64_t x_head_stride, void* y, int y_dtype,
                   int64_t y_tok_stride, int64_t y_head_stride, const int32_t* pos, int tokens, int heads,
                   int head_dim, const spec_rope* plan, int inverse, void* stream) {
  const char* who = "spec_rope_rows";
  if (tokens < 0 || heads < 1 || heads > 65535 || head_dim < 2 || head_dim > 4096)
    return fail(SPEC_E_ARG, std::string(who) + ": bad tokens, heads or head_dim");
  if (!plan || !plan_ok(plan, head_dim))
    return fail(SPEC_E_ARG, std::string(who) + ": null plan, or a rot_dim larger than the head");
  if (!is_io(x_dtype) || !is_io(y_dtype)) return fail(SPEC_E_ARG, std::string(who) + ": rows are fp32 or bf16");
  if (tokens == 0) return SPEC_OK;
  if (!x || !y || !pos) return fail(SPEC_E_ARG, std::string(who) + ": null pointer");
  if (x == y && (x_dtype != y_dtype || x_tok_stride != y_tok_stride || x_head_stride != y_head_stride))
    return fail(SPEC_E_ARG, std::string(who) + ": in place needs equal dtypes and strides");
  // odd head sizes leave one element over the pairs of chunks
  if (head_dim % 2) return fail(SPEC_E_SHAPE, std::string(who) + ": head_dim must be even");
  RopeArgs a{};
  a.x = x; a.y = y; a.xt = x_tok_stride; a.xh = x_head_stride; a.yt = y_tok_stride; a.yh = y_head_stride;
  a.pos = pos; a.tokens = tokens; a.heads = heads; a.hd = head_dim; a.sign = inverse ? -1.f : 1.f;
  a.r = *plan;
  const bool vec = head_dim % 16 == 0 && plan->rot_dim % (plan->interleaved ? 8 : 16) == 0 &&
                   vec_ok(x, x_tok_stride, x_head_stride, x_dtype) && vec_ok(y, y_tok_stride, y_head_stride, y_dtype);
  // about a thousand units a block where there are many tokens; for few, the
  // heads of a token are spread over blocks of one unit a thread
  const int upt = head_dim / (vec ? 16 : 2);
  a.hpb = std::min(heads, std::max(1, 8192 / upt));
  a.tpb = std::max(1, std::min(kMaxTokBlock, 4 * kRowThreads / (a.hpb * upt)));
  if ((int64_t)tokens * heads * upt < 1200LL * kRowThreads) {
    a.tpb = 1;
    a.hpb = std::max(1, std::min(a.hpb, kRowThreads / upt));
  }
  a.m_per = div_magic((int64_t)a.hpb * upt);
  a.m_unit = div_magic(upt);
  cudaStream_t st = (cudaStream_t)stream;
  const bool xi = x_dtype == SPEC_DTYPE_F32, yi = y_dtype == SPEC_DTYPE_F32;
  cudaError_t e;
  if (xi) e = yi ? launch_rope<float, float>(a, vec, st) : launch_rope<float, bf16>(a, vec, st);
  else e = yi ? launch_rope<bf16, float>(a, vec, st) : launch_rope<bf16, bf16>(a, vec, st);
  return done(e, who);
}

int spec_kv_append(const spec_kv_cache* cache, const void* k, int64_t k_tok_stride, int64_t k_head_stride,
                   const void* v, int64_t v_tok_stride, int64_t v_head_stride, int dtype, const int32_t* seq,
                   const int32_t* pos, int tokens, const spec_rope* plan, void* stream) {
  const char* who = "spec_kv_append";
  int rc = check_cache(cache, who);
  if (rc) return rc;
  if (tokens < 0 || !is_io(dtype)) return fail(SPEC_E_ARG, std::string(who) + ": bad tokens, or rows not fp32 or bf16");
  if (plan && !plan_ok(plan, cache->head_dim))
    return fail(SPEC_E_ARG, std::string(who) + ": the plan's rot_dim does not fit the head");
  if (tokens == 0) return SPEC_OK;
  if (!k || !v || !seq || !pos) return fail(SPEC_E_ARG, std::string(who) + ": null pointer");
  AppendArgs a{};
  a.c = cache_args(*cache);
  a.k = k; a.v = v; a.kt = k_tok_stride; a.kh = k_head_stride; a.vt = v_tok_stride; a.vh = v_head_stride;
  a.seq = seq; a.pos = pos; a.tokens = tokens;
  if (plan) a.r = *plan;
  const bool vec = vec_ok(k, k_tok_stride, k_head_stride, dtype) && vec_ok(v, v_tok_stride, v_head_stride, dtype) &&
                   (!plan || plan->rot_dim % (plan->interleaved ? 8 : 16) == 0);
  const int64_t per = (int64_t)cache->n_kv_heads * (cache->head_dim / (vec ? 16 : 2));   // threads a token's K or V
  a.tpb = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxTokBlock, 4 * kRowThreads / per));
  a.m_heads = div_magic(cache->n_kv_heads);
  int ysplit = 1;
  if (tokens * per < 1200LL * kRowThreads) {
    a.tpb = 1;
    ysplit = (int)std::max<int64_t>(1, std::min<int64_t>(8, per / kRowThreads));
  }
  const bool f8 = cache->dtype == SPEC_DTYPE_E4M3;
  cudaStream_t st = (cudaStream_t)stream;
  return done(dtype == SPEC_DTYPE_F32 ? launch_append_t<float>(a, vec, f8, ysplit, st)
                                      : launch_append_t<bf16>(a, vec, f8, ysplit, st), who);
}

int spec_kv_gather(const spec_kv_cache* cache, const int32_t* seq, const int32_t* pos, int tokens, void* k_out,
                   void* v_out, int out_dtype, void* stream) {
  const char* who = "spec_kv_gather";
  int rc = check_cache(cache, who);
  if (rc) return rc;
  if (tokens < 0 || !is_io(out_dtype)) return fail(SPEC_E_ARG, std::string(who) + ": bad tokens, or rows not fp32 or bf16");
  if (tokens == 0 || (!k_out && !v_out)) return SPEC_OK;
  if (!seq || !pos) return fail(SPEC_E_ARG, std::string(who) + ": null pointer");
  if ((reinterpret_cast<uintptr_t>(k_out) & 15u) || (reinterpret_cast<uintptr_t>(v_out) & 15u))
    return fail(SPEC_E_ARG, std::string(who) + ": outputs must be 16-byte aligned");
  GatherArgs a{};
  a.c = cache_args(*cache);
  a.seq = seq; a.pos = pos; a.k = k_out; a.v = v_out; a.tokens = tokens;
  const bool f8 = cache->dtype == SPEC_DTYPE_E4M3;
  const int64_t per = (int64_t)cache->n_kv_heads * (cache->head_dim / (f8 ? 16 : 8));
  a.tpb = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxTokBlock, 4 * kRowThreads / per));
  if (tokens * per < 1200LL * kRowThreads) a.tpb = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxTokBlock, kRowThreads / per));
  a.m_per = div_magic(per);
  const dim3 grid((tokens + a.tpb - 1) / a.tpb, k_out && v_out ? 2 : 1);
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (out_dtype == SPEC_DTYPE_F32)
    e = f8 ? launch_rows(gather_kernel<float, true>, grid, dim3(kRowThreads), 0, 1, st, a)
           : launch_rows(gather_kernel<float, false>, grid, dim3(kRowThreads), 0, 1, st, a);
  else
    e = f8 ? launch_rows(gather_kernel<bf16, true>, grid, dim3(kRowThreads), 0, 1, st, a)
           : launch_rows(gather_kernel<bf16, false>, grid, dim3(kRowThreads), 0, 1, st, a);
  return done(e, who);
}

}  // extern "C"
