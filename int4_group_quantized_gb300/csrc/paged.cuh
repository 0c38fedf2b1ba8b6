// Shared by the paged-cache kernels: the pool and table as kernel arguments,
// host-side checks, and the bounds checks every device-read index goes through
// (FlexGen notes, "背景知识": KV Concat; "5. 近似方法": KV stored in 4-bit
// groups of 64 along the hidden dimension).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "fg_internal.cuh"

namespace fg {
namespace paged {

struct Pool {
  uint8_t* codes[2];    // K, V: [pages][heads][ps][D/2]
  float* mins[2];       // [pages][heads][ps][D/64]
  float* scales[2];
  int pages, heads, ps_log2;
};

struct Table {
  int32_t* table;       // [seqs][stride]
  int32_t* lens;
  int32_t* refs;
  int seqs, pages, ps_log2;
  int64_t stride;
};

// A ragged batch: rows cu[i] .. cu[i+1]-1 belong to sequence i.
struct Batch {
  const int32_t* cu;
  int ntok;
  unsigned int* err;    // device error word
};

inline int log2_of(int ps) {
  int l = 0;
  while ((1 << l) < ps) ++l;
  return l;
}

// Rows [row0, row0 + n) of sequence i and its tokens in the cache (at most
// what a table row can name).  Offsets outside the batch give n = 0 and raise
// DEV_ERR_BATCH.
struct Seq {
  int row0, n, len, keys;   // len as stored; keys = min(len, stride * ps)
};
__device__ __forceinline__ Seq seq_of(const Table& t, const Batch& b, int i) {
  Seq s;
  const int a = b.cu[i], e = b.cu[i + 1];
  const int len = t.lens[i];
  const bool ok = a >= 0 && e >= a && e <= b.ntok && len >= 0;
  if (!ok) atomicOr(b.err, DEV_ERR_BATCH);
  s.row0 = ok ? a : 0;
  s.n = ok ? e - a : 0;
  s.len = ok ? len : 0;
  const int64_t cap = t.stride << t.ps_log2;
  s.keys = s.len > cap ? static_cast<int>(cap) : s.len;
  if (s.n > 0 && s.len > cap) atomicOr(b.err, DEV_ERR_PAGE);
  return s;
}

// The sequence that row `r` of the batch belongs to: the last i with cu[i] <= r
// (seqs when r lies outside every sequence).  With offsets that decrease the
// answer is some sequence; callers check r against seq_of's range.
__device__ __forceinline__ int seq_of_row(const int32_t* cu, int seqs, int r) {
  int lo = 0, hi = seqs;   // cu[lo] <= r < cu[hi] is sought
  if (r < cu[0] || r >= cu[seqs]) return seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Page of token `pos` of sequence i, or -1 where the row is too short or the
// entry is no page.
__device__ __forceinline__ int page_of(const Table& t, int i, int pos) {
  const int64_t j = pos >> t.ps_log2;
  if (j >= t.stride) return -1;
  const int p = t.table[i * t.stride + j];
  return (p >= 0 && p < t.pages) ? p : -1;
}
// Row of the pool's arrays that holds token `pos` of head h in page `page`.
__device__ __forceinline__ int64_t slot_of(const Pool& p, int page, int h, int pos) {
  return ((static_cast<int64_t>(page) * p.heads + h) << p.ps_log2) + (pos & ((1 << p.ps_log2) - 1));
}

// A launch; an `early` one may be set up while the one before it in the stream still runs: every kernel launched so waits for
// that one (griddepcontrol.wait) before it reads or writes anything.  Calls outside a graph gain the 2 us between kernels
// (a small step's attention 10.8 us from 13.1, an append of a step 7.9 from 10.2).
template <class... P, class... A>
fg_status launch(const char* what, bool early, void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st, A&&... args) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = early ? 1 : 0;
  cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  return check_launch(what);
}

fg_status check_pool(const fg_page_pool* p);
fg_status check_table(const fg_page_table* t);
fg_status check_pool_table(const fg_page_pool* p, const fg_page_table* t);
Pool pool_of(const fg_page_pool& p);
Table table_of(const fg_page_table& t);

}  // namespace paged
}  // namespace fg
