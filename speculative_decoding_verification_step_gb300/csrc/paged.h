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
template <typename... KArgs, typename... Args>
inline cudaError_t launch_rows(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster,
                               cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// launch_rows of a kernel that needs `smem` bytes of dynamic shared memory.
// The kernel's limit is a property of the device's context and is raised at
// the first launch there (a call of about half the launch's own cost); a
// launch that fails, as after a device reset, raises it again.
template <typename Tag, typename... KArgs, typename... Args>
inline cudaError_t launch_rows_smem(Tag, void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster,
                                    cudaStream_t st, Args&&... args) {
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (raised.load(std::memory_order_relaxed) & bit) {
    e = launch_rows(kernel, grid, block, smem, cluster, st, args...);
    if (e != cudaErrorInvalidValue) return e;
    (void)cudaGetLastError();
  }
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  raised.fetch_or(bit, std::memory_order_relaxed);
  return launch_rows(kernel, grid, block, smem, cluster, st, args...);
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
  float* ws;                     // workspace of launch_pattn_td, or null
  int give_up;                   // test hook: the step of a tensor-memory block that waits for what never comes (0: none)
};
// SPEC_FAULT_ATTN_TIMEOUT: give_up of the calls from now on.
extern std::atomic<int> g_attn_give_up;
// Rows per KV head of the longest sequence beyond which the tensor-memory
// kernel takes every call that both can.
constexpr int kPaMaxRows = 64;
// Tensor-memory kernel: bf16 or e4m3 keys, head dim 64 or 128.
bool pattn_tc_supported(const PAttn& a);
cudaError_t launch_pattn_tc(const PAttn& a, int num_sms, cudaStream_t st);
// Few rows over paged 8-bit keys on tensor memory (head dim 64 or 128), with
// a.ws of pattn_td_workspace bytes for `rows` rows per KV head.
bool pattn_td_supported(const PAttn& a);
size_t pattn_td_workspace(int64_t rows, int hd, int num_sms);
cudaError_t launch_pattn_td(const PAttn& a, int num_sms, cudaStream_t st);

}  // namespace sv
