// Internal interface of the paged-cache operators (kvrows.cu: rotary
// positions, cache write and read-back; pattn.cu, pattn_tc.cu: attention).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <string>
#include <utility>

#include "common.cuh"
#include "specverify.h"

namespace sv {

void set_thread_error(const std::string& msg);  // engine.cu

// A launch in plain stream order (these kernels take no part in programmatic
// dependent launch), optionally in clusters of `cluster` blocks along x.
// (`early`: may start before the kernel in front of it ends; it waits for that one itself.)
template <typename... KArgs, typename... Args>
inline cudaError_t launch_rows_early(bool early, void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster,
                                     cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  if (early) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}
template <typename... KArgs, typename... Args>
inline cudaError_t launch_rows(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster,
                               cudaStream_t st, Args&&... args) {
  return launch_rows_early(false, kernel, grid, block, smem, cluster, st, std::forward<Args>(args)...);
}

// launch_rows of a kernel that needs `smem` bytes of dynamic shared memory.
// The kernel's limit is a property of the device's context and is raised at
// the first launch there (a call of about half the launch's own cost); a
// launch that fails, as after a device reset, raises it again.
template <bool Early = false, typename Tag, typename... KArgs, typename... Args>
inline cudaError_t launch_rows_smem(Tag, void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster,
                                    cudaStream_t st, Args&&... args) {
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (raised.load(std::memory_order_relaxed) & bit) {
    e = launch_rows_early(Early, kernel, grid, block, smem, cluster, st, args...);
    if (e != cudaErrorInvalidValue) return e;
    (void)cudaGetLastError();
  }
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  raised.fetch_or(bit, std::memory_order_relaxed);
  return launch_rows_early(Early, kernel, grid, block, smem, cluster, st, args...);
}

// Power of two of an 8-bit row: 2^(byte - 127), of which byte 0 is below fp32's
// normal numbers; 255 marks a row of NaN.
SV_DEV float row_power(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fffffffu : max(byte << 23, 0x00400000u));
}

// Checks of a cache description shared by the entry points; SPEC_OK or the
// code to return, with the message set.
int check_cache(const spec_kv_cache* c, const char* who);

// One attention call.  Row r of sequence b's KV head g is token r / G, query
// head g * G + r % G (G = hq / hkv).  Keys come from pages (paged = 1) or
// from packed rows (kcu = cu, the rows of the sequence itself).
struct PAttn {
  const void* q;
  int64_t q_ts, q_hs;            // strides in elements between tokens and heads
  const int32_t* cu;             // [seqs + 1] rows of q of each sequence
  const int32_t* lens;           // [seqs] keys (paged); packed: the rows themselves
  int seqs, tokens, max_q;
  int hq, hkv, hd;
  float scale_log2;              // softmax scale * log2(e)
  void* out;
  int64_t o_ts, o_hs;
  float* lse;                    // [tokens][hq] or null
  int paged, f8;
  const void* k;                 // pools, or packed rows
  const void* v;
  int64_t k_ts, k_hs, v_ts, v_hs;   // packed: strides of k and v
  const uint8_t* ks;
  const uint8_t* vs;
  int64_t page_stride, scale_stride;
  const int32_t* table;
  int64_t table_stride;
  int pages, page_shift, max_pages;
  float* ws;                     // workspace of launch_pattn_td or launch_pattn_shared, or null
  int window, sinks;             // a row sees the last `window` keys up to its own (0: all) and keys below `sinks`
  const int32_t* groups;         // shared prefixes: [n_groups + 1] first sequences (null: one group of all)
  const int32_t* shared;         // [n_groups] positions whose pages a group's rows of the table all name
  int n_groups, runs;            // most runs that share a prefix's units
  float* rest;                   // [tokens][hq] sums of head_dim, then references and sums of what lies behind the prefixes
  int give_up;                   // test hook: the step of a tensor-memory block that waits for what never comes (0: none)
};
// What a row of the attention kernels sees of the keys up to its own position.
enum PaMode {
  kPaCausal = 0,   // all
  kPaWindow = 1,   // the last `window`, and those below `sinks`
  kPaRest = 2,     // those behind its group's shared prefix, to be joined with the prefix's parts
  kPaPrefix = 3    // tensor memory only: parts of a group's shared prefix, seen whole by all of the group's rows
};
// A group of sequences as the prefix's kernels see it (worked out on the device).
struct __align__(16) ShGroup {
  int eff;         // shared positions that all rows of the group see
  int unit0;       // its first unit: 128 keys of one (KV head, pair of row tiles)
  int tile0;       // its first (KV head, pair of row tiles)
  int row0, toks;  // first row, rows
  int seq0;        // the sequence whose table row is read: the group's first with rows
  int pairs, steps;
};
// What a sequence shares with its group (eff 0: nothing), for the rest and the join.
struct __align__(16) ShSeq {
  int eff, row0, unit0, tile0, pairs, steps, pad[2];
};
// The prefix's workspace: the units and the runs that share them, the groups, the sequences,
// then slots [256 rows][head_dim] of sums, [256] of a reference and a sum.  Run r's part of
// (KV head, pair) tile i lies in slot r + i: along the runs either grows by one.
struct __align__(16) ShPlan {
  int units, runs, pad[6];
};
__host__ __device__ inline size_t sh_slots_at(int n_groups, int seqs) {
  return (sizeof(ShPlan) + (size_t)n_groups * sizeof(ShGroup) + (size_t)seqs * sizeof(ShSeq) + 255) & ~(size_t)255;
}
SV_DEV int sh_begin(int run, int units, int runs) {
  const uint64_t n = (uint64_t)units * run;
  return n >> 32 ? (int)(n / (uint32_t)runs) : (int)((uint32_t)n / (uint32_t)runs);
}
SV_DEV int sh_run(int unit, int units, int runs) {   // the run of a unit; run r begins at units * r / runs
  const uint64_t n = ((uint64_t)unit + 1) * runs - 1;
  return n >> 32 ? (int)(n / (uint32_t)units) : (int)((uint32_t)n / (uint32_t)units);
}
SV_DEV ShGroup* sh_groups(const float* ws) {
  return reinterpret_cast<ShGroup*>(reinterpret_cast<ShPlan*>(const_cast<float*>(ws)) + 1);
}
SV_DEV ShSeq* sh_seqs(const float* ws, int n_groups) { return reinterpret_cast<ShSeq*>(sh_groups(ws) + n_groups); }
SV_DEV float* sh_slot(const float* ws, int n_groups, int seqs, int hd, int slot) {
  return const_cast<float*>(ws) + sh_slots_at(n_groups, seqs) / sizeof(float) + (size_t)slot * 256 * (hd + 2);
}
// SPEC_FAULT_ATTN_TIMEOUT: give_up of the calls from now on.
extern std::atomic<int> g_attn_give_up;
// Rows per KV head of the longest sequence beyond which the tensor-memory
// kernel takes every call that both can.
constexpr int kPaMaxRows = 64;
// Tensor-memory kernel: bf16 or e4m3 keys, head dim 64 or 128.
bool pattn_tc_supported(const PAttn& a);
cudaError_t launch_pattn_tc(const PAttn& a, int num_sms, cudaStream_t st);
// The same, and the register tiles, for a window.
cudaError_t launch_pattn_tc_window(const PAttn& a, int num_sms, cudaStream_t st);
cudaError_t launch_pa_window(const PAttn& a, int num_sms, cudaStream_t st);
// Sequences behind shared prefixes: the prefixes on tensor memory in equal runs over all SMs,
// each sequence's rest in register tiles, and a join of the parts.  Head dim 64 or 128, up to
// kPaMaxRows rows per KV head of a sequence, a.ws of pattn_shared_workspace bytes (0: not supported).
size_t pattn_shared_workspace(const PAttn& a, int num_sms);
cudaError_t launch_pattn_shared(const PAttn& a, int num_sms, cudaStream_t st);
cudaError_t launch_pa_rest(const PAttn& a, int num_sms, cudaStream_t st);
// Few rows over paged 8-bit keys on tensor memory (head dim 64 or 128), with
// a.ws of pattn_td_workspace bytes for `rows` rows per KV head.
bool pattn_td_supported(const PAttn& a);
size_t pattn_td_workspace(int64_t rows, int hd, int num_sms);
cudaError_t launch_pattn_td(const PAttn& a, int num_sms, cudaStream_t st);

}  // namespace sv
