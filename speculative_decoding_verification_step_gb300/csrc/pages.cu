// Pages and index arrays of a step, worked out on the GPU: kv_reserve gives every
// sequence the pages of its new tokens and writes the arrays that the row and attention
// calls read, kv_release takes back the pages of positions that are dropped (rejected
// drafts, finished sequences).
//
// A sequence of length L holds ceil(L / page_size) pages.  Both calls are prefix sums
// over the sequences (pages and tokens in 64 bits), then writes of what the sums place:
//   reserve  the i-th page needed, in order of sequences and positions, is the i-th from
//            the top of the free stack; token i of the step finds its sequence by a
//            search in the sums, four tokens a thread.
//   release  the i-th page dropped goes to place n_free + i of the stack.  Entries that a
//            program has cleared itself (negative: the pages in front of a window) are no
//            pages, so the places follow from what the table holds: a block takes its run of
//            the dropped entries into shared memory, and the blocks of a cluster tell each
//            other how many pages are among them (64 prompts' release 1.3 us of 11.4; a step's
//            few entries are the first block's, 0.3).
// Sequences come in chunks of kPgThreads, a chunk's sums in shared memory.  One block is
// enough for a verify step; where there is more to write, a cluster of eight shares the
// writes: every block sums for itself (the inputs are a few KB and lie in L2), and the
// stack's count changes behind a barrier of the cluster, when all have read it.  Beyond
// 64 thousand tokens the blocks are as many as the writes need, and the count changes in a
// launch behind them (960 thousand tokens and the release of their pages 61 -> 21 us).
// No atomics: the pages that a sequence gets depend on the arguments alone.
// Bound by latency: loads, two scans, searches, stores.  64 sequences x 6 tokens and their
// release 8.2 us replayed from a graph; as calls 21 us of host time, 6 of them the results.
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "common.cuh"
#include "paged.h"
#include "rows_dev.cuh"

namespace sv {

namespace {

constexpr int kPgThreads = 512;
constexpr int kPgCluster = 8;
constexpr int kPgMost = 296;       // blocks of a step of many tokens (304, two an SM: 21.7 us for 21.4)
constexpr int kPgBatch = 4;        // dropped entries of a thread on their way
constexpr int kPgHeld = 8192;      // dropped entries of a block at a time

struct Sums {
  int64_t pages, toks;
};
// Inclusive sums of the block's values in thread order; total: those of all.
SV_DEV Sums block_sums(Sums v, Sums (&warps)[kPgThreads / 32], Sums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t p = __shfl_up_sync(0xffffffffu, v.pages, o), t = __shfl_up_sync(0xffffffffu, v.toks, o);
    if (lane >= o) {
      v.pages += p;
      v.toks += t;
    }
  }
  __syncthreads();                             // the last sums are read
  if (lane == 31) warps[warp] = v;
  __syncthreads();
  Sums before{0, 0};
  total = Sums{0, 0};
#pragma unroll
  for (int w = 0; w < kPgThreads / 32; ++w) {
    const Sums x = warps[w];
    if (w < warp) {
      before.pages += x.pages;
      before.toks += x.toks;
    }
    total.pages += x.pages;
    total.toks += x.toks;
  }
  return Sums{v.pages + before.pages, v.toks + before.toks};
}
// The last of at[0 .. n] (ascending) that is not above i, at most n - 1.
SV_DEV int find_run(const int* at, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}
SV_DEV void pg_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// *at of block `rank` of the cluster.
SV_DEV int pg_peer(const int* at, int rank) {
  int v;
  asm volatile("{\n .reg .u32 p;\n mapa.shared::cluster.u32 p, %1, %2;\n ld.shared::cluster.u32 %0, [p];\n}"
               : "=r"(v) : "r"(smem_u32(at)), "r"(rank) : "memory");
  return v;
}

struct PageArgs {
  int32_t* table;
  int64_t tstride;
  int seqs, max_pages, shift;
  const int32_t* lens;
  const int32_t* change;         // reserve: new tokens; release: kept length
  int32_t* free_pages;
  int32_t* n_free;
  int free_cap;
  int tokens;                    // reserve: capacity of seq and pos
  int32_t* cu;
  int32_t* lens_out;
  int32_t* seq;
  int32_t* pos;
  int32_t* lacking;
  int blocks;                    // 1, the cluster's, or more without a cluster
  int vec;                       // seq and pos take 16-byte stores
};

__global__ void __launch_bounds__(kPgThreads) reserve_kernel(const __grid_constant__ PageArgs a) {
  __shared__ Sums warps[kPgThreads / 32];
  __shared__ int s_tok[kPgThreads + 1], s_page[kPgThreads + 1], s_len[kPgThreads], s_had[kPgThreads];
  const int tid = threadIdx.x, rank = (int)blockIdx.x;
  const int me = rank * kPgThreads + tid, all = a.blocks * kPgThreads;
  const int left = max(0, min(ld_volatile_i32(a.n_free), a.free_cap)), ps1 = (1 << a.shift) - 1;
  const int64_t cap = (int64_t)a.max_pages << a.shift;
  Sums asked{0, 0}, given{0, 0};               // of the chunks before
  for (int b0 = 0; b0 < a.seqs; b0 += kPgThreads) {
    const int b = b0 + tid, n = min(kPgThreads, a.seqs - b0);
    const int len = b < a.seqs ? __ldg(a.lens + b) : -1, want = b < a.seqs ? max(0, __ldg(a.change + b)) : 0;
    const bool fits = len >= 0 && (int64_t)len + want <= cap;
    const int had = fits ? (int)(((int64_t)len + ps1) >> a.shift) : 0;
    Sums ask{0, 0}, total;
    if (fits) ask = Sums{(((int64_t)len + want + ps1) >> a.shift) - had, want};
    const Sums sum = block_sums(ask, warps, total);
    const bool served = fits && (ask.pages == 0 || asked.pages + sum.pages <= left) && asked.toks + sum.toks <= a.tokens;
    asked.pages += total.pages;
    asked.toks += total.toks;
    if (!served) ask = Sums{0, 0};
    const Sums at = block_sums(ask, warps, total);
    s_tok[tid + 1] = (int)(given.toks + at.toks);
    s_page[tid + 1] = (int)(given.pages + at.pages);
    s_len[tid] = len;
    s_had[tid] = had;
    if (tid == 0) {
      s_tok[0] = (int)given.toks;
      s_page[0] = (int)given.pages;
    }
    __syncthreads();
    if (rank == 0 && b < a.seqs) {
      a.lens_out[b] = len + (int)ask.toks;
      a.cu[b + 1] = s_tok[tid + 1];
    }
    given.pages += total.pages;
    given.toks += total.toks;
    // tokens of the chunk, four at a time
    const int t_beg = s_tok[0], t_end = (int)given.toks;
    for (int64_t i0 = (int64_t)(t_beg & ~3) + 4LL * me; i0 < t_end; i0 += 4LL * all) {
      const int i = (int)i0;
      int r = find_run(s_tok, n, max(i, t_beg)), sq[4], po[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        while (r + 1 < n && i + e >= s_tok[r + 1]) ++r;
        sq[e] = b0 + r;
        po[e] = s_len[r] + i + e - s_tok[r];
      }
      if (a.vec && i >= t_beg && i + 3 < t_end) {
        *reinterpret_cast<int4*>(a.seq + i) = make_int4(sq[0], sq[1], sq[2], sq[3]);
        *reinterpret_cast<int4*>(a.pos + i) = make_int4(po[0], po[1], po[2], po[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e >= t_beg && i + e < t_end) {
            a.seq[i + e] = sq[e];
            a.pos[i + e] = po[e];
          }
      }
    }
    // pages of the chunk
    const int p_end = (int)given.pages;
    for (int64_t i = (int64_t)s_page[0] + me; i < p_end; i += all) {
      const int r = find_run(s_page, n, (int)i);
      a.table[(b0 + r) * a.tstride + s_had[r] + ((int)i - s_page[r])] = a.free_pages[left - 1 - (int)i];
    }
    __syncthreads();                           // the chunk's sums are read
  }
  for (int64_t i = given.toks + me; i < a.tokens; i += all) a.seq[i] = a.pos[i] = -1;
  if (a.blocks == kPgCluster) pg_cluster_sync();   // all have read the count
  else __syncthreads();
  if (rank == 0 && tid == 0) {
    a.cu[0] = 0;
    if (a.blocks <= kPgCluster) *a.n_free = left - (int)given.pages;
    *a.lacking = (int)min((int64_t)0x7fffffff, max((int64_t)0, asked.pages - left));
  }
}

// The stack's count behind blocks that share no barrier: less the pages that the lengths grew by.
__global__ void __launch_bounds__(kPgThreads) reserve_end_kernel(const __grid_constant__ PageArgs a) {
  __shared__ Sums warps[kPgThreads / 32];
  const int ps1 = (1 << a.shift) - 1;
  Sums mine{0, 0}, total;
  for (int b = threadIdx.x; b < a.seqs; b += kPgThreads)
    mine.pages += (((int64_t)__ldg(a.lens_out + b) + ps1) >> a.shift) - (((int64_t)__ldg(a.lens + b) + ps1) >> a.shift);
  block_sums(mine, warps, total);
  if (threadIdx.x == 0) *a.n_free = max(0, min(*a.n_free, a.free_cap)) - (int)total.pages;
}

__global__ void __launch_bounds__(kPgThreads) release_kernel(const __grid_constant__ PageArgs a) {
  __shared__ Sums warps[kPgThreads / 32];
  __shared__ int s_page[kPgThreads + 1], s_beg[kPgThreads], s_held[kPgHeld], s_kept[2];
  const int tid = threadIdx.x, rank = (int)blockIdx.x;
  const int left = max(0, min(ld_volatile_i32(a.n_free), a.free_cap)), ps1 = (1 << a.shift) - 1, room = a.free_cap - left;
  const int64_t cap = (int64_t)a.max_pages << a.shift;
  int64_t done = 0, solo = 0;                  // pages that went before: of runs that all know of, of the block's since
  for (int b0 = 0, odd = 0; b0 < a.seqs; b0 += kPgThreads) {
    const int b = b0 + tid, n = min(kPgThreads, a.seqs - b0);
    const int64_t len = b < a.seqs ? min(cap, (int64_t)max(0, __ldg(a.lens + b))) : 0;
    const int64_t keep = b < a.seqs ? min(len, (int64_t)max(0, __ldg(a.change + b))) : 0;
    const int beg = (int)((keep + ps1) >> a.shift), end = (int)((len + ps1) >> a.shift);
    Sums total;
    const Sums at = block_sums(Sums{end - beg, 0}, warps, total);
    s_page[tid + 1] = (int)min((int64_t)0x7fffffff, at.pages);
    s_beg[tid] = beg;
    if (tid == 0) s_page[0] = 0;
    __syncthreads();
    const unsigned count = (unsigned)min((int64_t)0x7fffffff, total.pages), most = (unsigned)a.blocks * kPgHeld;
    for (unsigned t0 = 0; t0 < count; t0 += most) {
      // the block's run of the next entries (few of them are the first block's): out of the table, and counted
      const unsigned in = min(most, count - t0);
      const bool split = a.blocks == kPgCluster && in > kPgThreads;
      const unsigned i_beg = t0 + (split ? in * rank >> 3 : rank ? in : 0), i_end = t0 + (split ? in * (rank + 1) >> 3 : in);
      const unsigned run = i_end - i_beg;
      int sound = 0, mine = 0;
      for (unsigned i0 = tid; i0 < run; i0 += kPgBatch * kPgThreads) {
        int32_t* e[kPgBatch];
        int page[kPgBatch];
#pragma unroll
        for (int k = 0; k < kPgBatch; ++k) {   // (all on their way: the entries written are not those read)
          const unsigned i = i0 + k * kPgThreads;
          e[k] = nullptr;
          if (i < run) {
            const int at = (int)(i_beg + i), r = find_run(s_page, n, at);
            e[k] = a.table + (b0 + r) * a.tstride + s_beg[r] + (at - s_page[r]);
            page[k] = *e[k];
          }
        }
#pragma unroll
        for (int k = 0; k < kPgBatch; ++k)
          if (e[k]) {
            *e[k] = -1;
            s_held[i0 + k * kPgThreads] = page[k];
            sound += page[k] >= 0;
            ++mine;
          }
      }
      unsigned kept = run;
      if (!__syncthreads_and(sound == mine)) {
        block_sums(Sums{sound, 0}, warps, total);
        kept = (unsigned)total.pages;
      }
      int64_t place = done + solo;             // of the run's first page in the stack, from n_free on
      solo += kept;
      if (split) {
        if (tid == 0) s_kept[odd] = (int)solo;
        __syncwarp();
        pg_cluster_sync();
        for (int c = 0; c < kPgCluster; ++c) {
          const int k = pg_peer(&s_kept[odd], c);
          if (c < rank) place += k;
          done += k;
        }
        solo = 0;
        odd ^= 1;
      }
      // (a stack cannot hold more than free_cap: what would lie past it is dropped)
      if (kept == run) {
        for (unsigned i = tid; i < run; i += kPgThreads)
          if (place + i < room) a.free_pages[left + place + i] = s_held[i];
      } else {
        for (unsigned i0 = 0; i0 < run; i0 += kPgThreads) {
          const int page = i0 + tid < run ? s_held[i0 + tid] : -1;
          const Sums before = block_sums(Sums{page >= 0, 0}, warps, total);
          const int64_t to = place + before.pages - 1;
          if (page >= 0 && to < room) a.free_pages[left + to] = page;
          place += total.pages;
        }
      }
      __syncthreads();                         // s_held is read
    }
  }
  if (a.blocks == kPgCluster) pg_cluster_sync();   // all have read the count, and each other's
  if (rank == 0 && tid == 0) *a.n_free = left + (int)min((int64_t)room, done + solo);
}

// The checks that both calls share.
int page_args(PageArgs& a, const spec_kv_cache* cache, const int32_t* lens, const int32_t* change, int32_t* free_pages,
              int32_t* n_free, int free_cap, const char* who) {
  const std::string w = std::string(who) + ": ";
  const int rc = check_cache(cache, who);
  if (rc) return rc;
  if (!lens || !change || (!free_pages && free_cap > 0) || !n_free) return fail(SPEC_E_ARG, w + "null pointer");
  if (cache->seqs > 1 << 30) return fail(SPEC_E_ARG, w + "too many sequences");
  if (free_cap < 0) return fail(SPEC_E_ARG, w + "bad capacity of the free stack");
  a.table = const_cast<int32_t*>(cache->table);
  a.tstride = cache->table_stride ? cache->table_stride : cache->max_pages;
  a.seqs = cache->seqs;
  a.max_pages = cache->max_pages;
  while ((1 << a.shift) < cache->page_size) ++a.shift;
  a.lens = lens; a.change = change; a.free_pages = free_pages; a.n_free = n_free; a.free_cap = free_cap;
  return SPEC_OK;
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" {

int spec_kv_reserve(const spec_kv_cache* cache, const int32_t* kv_lens, const int32_t* counts, int32_t* free_pages,
                    int32_t* n_free, int free_cap, int tokens, int32_t* cu_q, int32_t* kv_lens_out, int32_t* seq,
                    int32_t* pos, int32_t* lacking, void* stream) {
  const char* who = "spec_kv_reserve";
  PageArgs a{};
  const int rc = page_args(a, cache, kv_lens, counts, free_pages, n_free, free_cap, who);
  if (rc) return rc;
  if (tokens < 0 || tokens > 0x7fffff00) return fail(SPEC_E_ARG, std::string(who) + ": bad tokens");
  if (!cu_q || !kv_lens_out || !lacking || (tokens > 0 && (!seq || !pos)))
    return fail(SPEC_E_ARG, std::string(who) + ": null pointer");
  if (kv_lens_out == kv_lens) return fail(SPEC_E_ARG, std::string(who) + ": kv_lens_out must not be kv_lens");
  a.tokens = tokens; a.cu = cu_q; a.lens_out = kv_lens_out; a.seq = seq; a.pos = pos; a.lacking = lacking;
  a.vec = ((reinterpret_cast<uintptr_t>(seq) | reinterpret_cast<uintptr_t>(pos)) & 15u) == 0;
  const bool many = tokens > 65536;
  a.blocks = many ? std::min(kPgMost, tokens / 1024) : tokens > 8 * kPgThreads ? kPgCluster : 1;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = launch_rows(reserve_kernel, dim3(a.blocks), dim3(kPgThreads), 0, many ? 1 : a.blocks, st, a);
  if (e == cudaSuccess && many) e = launch_rows(reserve_end_kernel, dim3(1), dim3(kPgThreads), 0, 1, st, a);
  return done(e, who);
}

int spec_kv_release(const spec_kv_cache* cache, const int32_t* kv_lens, const int32_t* keep, int32_t* free_pages,
                    int32_t* n_free, int free_cap, void* stream) {
  const char* who = "spec_kv_release";
  PageArgs a{};
  const int rc = page_args(a, cache, kv_lens, keep, free_pages, n_free, free_cap, who);
  if (rc) return rc;
  a.blocks = (int64_t)a.seqs * a.max_pages > 16 * kPgThreads ? kPgCluster : 1;
  return done(launch_rows(release_kernel, dim3(a.blocks), dim3(kPgThreads), 0, a.blocks, (cudaStream_t)stream, a), who);
}

}  // extern "C"
