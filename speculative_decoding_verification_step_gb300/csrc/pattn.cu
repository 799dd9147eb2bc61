// The attention calls: checks, choice of kernel, and the register-tile kernel
// (pattn_dev.cuh) of plain causal attention.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "common.cuh"
#include "paged.h"
#include "pattn_dev.cuh"

namespace sv {

std::atomic<int> g_attn_give_up{0};

namespace {

int fail(int code, const std::string& msg) {
  set_thread_error(msg);
  return code;
}
bool row_aligned(const void* p, int64_t ts, int64_t hs) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ts % 8 == 0 && hs % 8 == 0;
}

// A window that holds every position of the call is none.
void settle_window(PAttn& a) {
  const int64_t most = a.paged ? (int64_t)a.max_pages << a.page_shift : std::min(a.max_q, a.tokens);
  if (a.window >= most) a.window = 0;
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
  int64_t keys = (int64_t)a.max_pages << a.page_shift;
  if (a.window > 0) keys = std::min(keys, (int64_t)a.window + a.sinks + a.max_q);
  const int64_t items = (int64_t)a.seqs * a.hkv * ((rows + 31) / 32);
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

// Workspace of launch_pattn_shared where it is taken, else 0.  What is fixed in its four
// launches is some 25 us, 20 more than in the one launch of the other way, and sequences
// that read the same pages one by one find them in L2: it is taken where they would
// read 800 thousand rows of keys (positions x KV heads) again, for more than 8 rows per
// KV head, whose walk costs more, 260 thousand, 450 at head dim 64, and beyond 32 rows,
// where what lies behind the prefix weighs more, 2048 positions at least.
// The lengths being on the device, a table's width stands for them, so over a table much
// wider than its contexts (8 KV heads, 131072 positions: from two sequences on) sharing is
// taken where one by one would be faster: 4 x 6 behind 512 then take 18 us for 9, 2 x 1
// behind 2048 20 for 8.  One by one / shared, us, tables as wide as the contexts, 8 KV
// heads, 100 positions behind the prefix.  4 rows, bf16, head dim 128: 8 sequences x 8192
// 26 / 29, 16 x 8192 39 / 29, 64 x 2048 51 / 28, 64 x 8192 168 / 37, 4 x
// 32768 45 / 50; e4m3: 8 x 8192 29 / 36, 16 x 8192 50 / 35; head dim 64, bf16: 8 x 8192
// 16 / 28, 16 x 8192 26 / 26.  24 rows, bf16, head dim 128: 4 x 8192 28 / 35, 8 x 8192
// 47 / 39, 64 x 512 36 / 42, 64 x 2048 90 / 50; e4m3: 8 x 8192 58 / 42, 64 x 8192
// 288 / 92; head dim 64, bf16: 8 x 8192 27 / 30, 16 x 8192 38 / 36.  64 rows, bf16: 4 x
// 8192 46 / 43, 16 x 2048 36 / 38, 64 x 512 45 / 77, 64 x 2048 125 / 98.
size_t shared_bytes(const PAttn& a, int sms) {
  const int64_t rows = (int64_t)std::min(a.max_q, a.tokens) * (a.hq / a.hkv), keys = (int64_t)a.max_pages << a.page_shift;
  if (rows < 1 || rows > kPaMaxRows || a.seqs <= a.n_groups || (rows > 32 && keys < 2048)) return 0;
  const int64_t least = rows <= 8 ? 800000 : a.hd == 128 ? 260000 : 450000;
  return (double)(a.seqs - a.n_groups) * (double)keys * a.hkv < (double)least ? 0 : pattn_shared_workspace(a, sms);
}

// All attention calls, after their own checks.
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
  settle_window(a);
  if (a.scale_log2 == 0.f) a.scale_log2 = 1.f / std::sqrt((float)a.hd);
  a.scale_log2 *= kLog2e;
  a.give_up = g_attn_give_up.load(std::memory_order_relaxed);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(SPEC_E_CUDA, w + cudaGetErrorString(e));
  if (const size_t need = a.shared ? shared_bytes(a, sms) : 0; need && a.ws && ws_bytes >= need) {
    e = launch_pattn_shared(a, sms, st);
    return e == cudaSuccess ? SPEC_OK : fail(SPEC_E_CUDA, w + cudaGetErrorString(e));
  }
  const Way way = choose_way(a, sms);
  if (way.tc) e = a.window > 0 ? launch_pattn_tc_window(a, sms, st) : launch_pattn_tc(a, sms, st);
  else if (way.td_ws && a.ws && ws_bytes >= way.td_ws) e = launch_pattn_td(a, sms, st);
  else if (a.window > 0) e = launch_pa_window(a, sms, st);
  else e = a.hd == 32 ? launch_pa_hd<32, kPaCausal>(a, sms, st) : a.hd == 64 ? launch_pa_hd<64, kPaCausal>(a, sms, st) : launch_pa_hd<128, kPaCausal>(a, sms, st);
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

// Workspace of a call of these sizes (queries and outputs with strides that the kernels take:
// others go to the register tiles).  a: the window, or the number of groups.
int64_t asked_workspace(PAttn a, const char* who, const spec_kv_cache* cache, int tokens, int max_q, int n_heads) {
  if (check_cache(cache, who) || tokens < 1 || max_q < 1 || n_heads < 1 || n_heads % cache->n_kv_heads) return 0;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  cache_fields(a, cache);
  a.hq = n_heads; a.tokens = tokens; a.max_q = max_q;
  a.q_hs = a.o_hs = a.hd; a.q_ts = a.o_ts = (int64_t)n_heads * a.hd;
  settle_window(a);
  const size_t own = a.n_groups > 0 ? shared_bytes(a, sms) : 0;
  return own ? (int64_t)own : (int64_t)choose_way(a, sms).td_ws;
}

int window_fields(PAttn& a, int window, int sinks, const char* who) {
  if (window < 0 || sinks < 0) return fail(SPEC_E_ARG, std::string(who) + ": window and sinks must not be negative");
  a.window = window;
  a.sinks = sinks;
  return SPEC_OK;
}

// The calls over a cache (a: what sets them apart) and over packed prompts.
int paged_attention(PAttn a, const char* who, const spec_kv_cache* cache, const void* q, int64_t q_tok_stride,
                    int64_t q_head_stride, const int32_t* cu_q, const int32_t* kv_lens, int tokens, int max_q, int n_heads,
                    float scale, void* out, int64_t out_tok_stride, int64_t out_head_stride, float* lse, void* workspace,
                    int64_t workspace_bytes, void* stream) {
  const int rc = check_cache(cache, who);
  if (rc) return rc;
  if (tokens > 0 && !kv_lens) return fail(SPEC_E_ARG, std::string(who) + ": null kv_lens");
  if (workspace_bytes < 0 || (reinterpret_cast<uintptr_t>(workspace) & 15u))
    return fail(SPEC_E_ARG, std::string(who) + ": workspace must be 16-byte aligned");
  cache_fields(a, cache);
  a.q = q; a.q_ts = q_tok_stride; a.q_hs = q_head_stride;
  a.cu = cu_q; a.lens = kv_lens; a.tokens = tokens; a.max_q = max_q;
  a.hq = n_heads; a.scale_log2 = scale;
  a.out = out; a.o_ts = out_tok_stride; a.o_hs = out_head_stride; a.lse = lse;
  a.ws = (float*)workspace;
  return run_attention(a, workspace ? (size_t)workspace_bytes : 0, who, (cudaStream_t)stream);
}
int prompt_attention(PAttn a, const char* who, const void* q, int64_t q_tok_stride, int64_t q_head_stride, const void* k,
                     int64_t k_tok_stride, int64_t k_head_stride, const void* v, int64_t v_tok_stride, int64_t v_head_stride,
                     const int32_t* cu, int seqs, int tokens, int max_len, int n_heads, int n_kv_heads, int head_dim,
                     float scale, void* out, int64_t out_tok_stride, int64_t out_head_stride, float* lse, void* stream) {
  if (tokens > 0 && max_len > 0) {
    if (!k || !v) return fail(SPEC_E_ARG, std::string(who) + ": null pointer");
    if (!row_aligned(k, k_tok_stride, k_head_stride) || !row_aligned(v, v_tok_stride, v_head_stride))
      return fail(SPEC_E_ARG, std::string(who) + ": k and v must be 16-byte aligned with strides multiples of 8");
  }
  a.q = q; a.q_ts = q_tok_stride; a.q_hs = q_head_stride;
  a.cu = cu; a.seqs = seqs; a.tokens = tokens; a.max_q = max_len;
  a.hq = n_heads; a.hkv = n_kv_heads; a.hd = head_dim; a.scale_log2 = scale;
  a.out = out; a.o_ts = out_tok_stride; a.o_hs = out_head_stride; a.lse = lse;
  a.k = k; a.v = v; a.k_ts = k_tok_stride; a.k_hs = k_head_stride; a.v_ts = v_tok_stride; a.v_hs = v_head_stride;
  return run_attention(a, 0, who, (cudaStream_t)stream);
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" {

int spec_attn_paged(const spec_kv_cache* cache, const void* q, int64_t q_tok_stride, int64_t q_head_stride,
                    const int32_t* cu_q, const int32_t* kv_lens, int tokens, int max_q, int n_heads, float scale,
                    void* out, int64_t out_tok_stride, int64_t out_head_stride, float* lse, void* workspace,
                    int64_t workspace_bytes, void* stream) {
  return paged_attention(PAttn{}, "spec_attn_paged", cache, q, q_tok_stride, q_head_stride, cu_q, kv_lens, tokens, max_q,
                         n_heads, scale, out, out_tok_stride, out_head_stride, lse, workspace, workspace_bytes, stream);
}

int spec_attn_paged_window(const spec_kv_cache* cache, const void* q, int64_t q_tok_stride, int64_t q_head_stride,
                           const int32_t* cu_q, const int32_t* kv_lens, int tokens, int max_q, int n_heads, float scale,
                           int window, int sinks, void* out, int64_t out_tok_stride, int64_t out_head_stride, float* lse,
                           void* workspace, int64_t workspace_bytes, void* stream) {
  PAttn a{};
  const char* who = "spec_attn_paged_window";
  const int rc = window_fields(a, window, sinks, who);
  return rc ? rc : paged_attention(a, who, cache, q, q_tok_stride, q_head_stride, cu_q, kv_lens, tokens, max_q, n_heads, scale,
                                   out, out_tok_stride, out_head_stride, lse, workspace, workspace_bytes, stream);
}

int spec_attn_shared(const spec_kv_cache* cache, const void* q, int64_t q_tok_stride, int64_t q_head_stride,
                     const int32_t* cu_q, const int32_t* kv_lens, const int32_t* groups, int n_groups,
                     const int32_t* shared, int tokens, int max_q, int n_heads, float scale, void* out,
                     int64_t out_tok_stride, int64_t out_head_stride, float* lse, void* workspace,
                     int64_t workspace_bytes, void* stream) {
  const char* who = "spec_attn_shared";
  if (n_groups < 1 || (!groups && n_groups != 1))
    return fail(SPEC_E_ARG, std::string(who) + ": n_groups must be positive, and 1 without groups");
  if (tokens > 0 && !shared) return fail(SPEC_E_ARG, std::string(who) + ": null shared");
  PAttn a{};
  a.groups = groups; a.n_groups = n_groups; a.shared = shared;
  return paged_attention(a, who, cache, q, q_tok_stride, q_head_stride, cu_q, kv_lens, tokens, max_q, n_heads, scale, out,
                         out_tok_stride, out_head_stride, lse, workspace, workspace_bytes, stream);
}

int64_t spec_attn_paged_workspace(const spec_kv_cache* cache, int tokens, int max_q, int n_heads) {
  return asked_workspace(PAttn{}, "spec_attn_paged_workspace", cache, tokens, max_q, n_heads);
}

int64_t spec_attn_paged_window_workspace(const spec_kv_cache* cache, int tokens, int max_q, int n_heads, int window,
                                         int sinks) {
  PAttn a{};
  const char* who = "spec_attn_paged_window_workspace";
  return window_fields(a, window, sinks, who) ? 0 : asked_workspace(a, who, cache, tokens, max_q, n_heads);
}

int64_t spec_attn_shared_workspace(const spec_kv_cache* cache, int n_groups, int tokens, int max_q, int n_heads) {
  PAttn a{};
  a.n_groups = n_groups;
  return n_groups < 1 ? 0 : asked_workspace(a, "spec_attn_shared_workspace", cache, tokens, max_q, n_heads);
}

int spec_attn_prompt(const void* q, int64_t q_tok_stride, int64_t q_head_stride, const void* k, int64_t k_tok_stride,
                     int64_t k_head_stride, const void* v, int64_t v_tok_stride, int64_t v_head_stride,
                     const int32_t* cu, int seqs, int tokens, int max_len, int n_heads, int n_kv_heads, int head_dim,
                     float scale, void* out, int64_t out_tok_stride, int64_t out_head_stride, float* lse,
                     void* stream) {
  return prompt_attention(PAttn{}, "spec_attn_prompt", q, q_tok_stride, q_head_stride, k, k_tok_stride, k_head_stride, v,
                          v_tok_stride, v_head_stride, cu, seqs, tokens, max_len, n_heads, n_kv_heads, head_dim, scale, out,
                          out_tok_stride, out_head_stride, lse, stream);
}

int spec_attn_prompt_window(const void* q, int64_t q_tok_stride, int64_t q_head_stride, const void* k, int64_t k_tok_stride,
                            int64_t k_head_stride, const void* v, int64_t v_tok_stride, int64_t v_head_stride,
                            const int32_t* cu, int seqs, int tokens, int max_len, int n_heads, int n_kv_heads,
                            int head_dim, float scale, int window, int sinks, void* out, int64_t out_tok_stride,
                            int64_t out_head_stride, float* lse, void* stream) {
  PAttn a{};
  const char* who = "spec_attn_prompt_window";
  const int rc = window_fields(a, window, sinks, who);
  return rc ? rc : prompt_attention(a, who, q, q_tok_stride, q_head_stride, k, k_tok_stride, k_head_stride, v, v_tok_stride,
                                    v_head_stride, cu, seqs, tokens, max_len, n_heads, n_kv_heads, head_dim, scale, out,
                                    out_tok_stride, out_head_stride, lse, stream);
}

}  // extern "C"
