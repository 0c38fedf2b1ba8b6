// Which sequences of a batch share leading pages (forks of one another), for
// attention that reads a shared prefix once (FlexGen notes, "4. 卸载策略": one
// read serves every sequence of the block, here of the cache).
//
// Two launches.  The first compares table rows, a warp a sequence: its leader,
// the lowest-numbered sequence that begins with the same page, and the number of
// leading entries the two have in common.  The second, one CTA, picks every
// leader's number of shared pages, numbers the groups and lists their rows.
// Bound by launch latency and two chains of dependent reads; the rows' entries are
// read once and compared with the leader's, which stay in L2.  256 sequences over
// seven prefixes of 100 to 1,500 pages: 17 us (each launch by itself, cold: comparing
// 11, picking 13); 12 sequences 7.  Picking counts followers pair by pair in one CTA,
// so it grows with the square: 1,024 sequences over one prefix 72 us, 4,096 0.96 ms,
// 16,384 14 ms, made once when a batch changes.
#include <algorithm>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace fg {
namespace paged {
namespace {

constexpr int kWarps = 8;
constexpr int kPickThreads = 1024;
constexpr unsigned long long kMostSeqs = 16384;   // the picking compares all followers pair by pair; c * count * kMostSeqs is below 2^54

struct ShareArgs {
  Table tab;
  Batch batch;
  int min_pages;
  int32_t *group, *tokens, *first, *leader, *begin, *rows;
  // workspace: of sequence i its leader (-1: it takes no part), the entries in common with it, its rows; of a leader the
  // pages that its group shares, the group's number and its rows
  int32_t *lead, *common, *n, *pick, *number, *size;
  unsigned long long* best;   // (page reads saved, followers counted down) of a leader's best number of pages
};

// Rows and usable pages of sequence i: full pages that end before its rows.
__device__ __forceinline__ int usable_pages(const Table& t, const Batch& b, int i, int& n) {
  const Seq s = seq_of(t, b, i);
  n = s.n;
  if (s.n == 0 || s.len <= s.n) return 0;
  const int64_t full = (s.len - s.n) >> t.ps_log2;
  return static_cast<int>(full < t.stride ? full : t.stride);
}
// The first page of a sequence that takes part, or -1.
__device__ __forceinline__ int first_page(const Table& t, const Batch& b, int i) {
  int n;
  if (usable_pages(t, b, i, n) == 0) return -1;
  const int p = t.table[i * t.stride];
  return p >= 0 && p < t.pages ? p : -1;
}

__global__ void __launch_bounds__(32 * kWarps) compare_kernel(const ShareArgs a) {
  tc::griddep_launch();
  tc::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= a.tab.seqs) return;
  int n;
  const int mine = usable_pages(a.tab, a.batch, i, n), page = first_page(a.tab, a.batch, i);
  int lead = page < 0 ? -1 : i, common = mine;
  if (page >= 0) {
    for (int j0 = 0; j0 < i; j0 += 32) {
      const int j = j0 + lane;
      const uint32_t same = __ballot_sync(0xffffffffu, j < i && first_page(a.tab, a.batch, j) == page);
      if (same) {
        lead = j0 + __ffs(same) - 1;
        break;
      }
    }
    int other;
    const int end = min(mine, lead == i ? mine : usable_pages(a.tab, a.batch, lead, other));
    const int32_t* x = a.tab.table + i * a.tab.stride;
    const int32_t* y = a.tab.table + lead * a.tab.stride;
    common = end;
    constexpr int kAhead = 16;
    for (int j0 = 0; j0 < end; j0 += 32 * kAhead) {   // the first entry that differs or is no page
      int at = end;
#pragma unroll
      for (int e = kAhead - 1; e >= 0; --e) {
        const int j = j0 + 32 * e + lane;
        if (j < end) {
          const int p = x[j];
          if (p != y[j] || p < 0 || p >= a.tab.pages) at = j;
        }
      }
      at = __reduce_min_sync(0xffffffffu, at);
      if (at < end) {
        common = at;
        break;
      }
    }
  }
  if (lane == 0) {
    a.lead[i] = lead;
    a.common[i] = common;
    a.n[i] = n;
    a.best[i] = 0;
  }
}

// Prefix sum of one value a thread over the CTA, and the total (three barriers).
__device__ __forceinline__ int cta_prefix(int v, int* slots, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  __syncthreads();
  if (lane == 31) slots[warp] = inc;
  __syncthreads();
  int w = slots[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += up;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return inc - v + (warp > 0 ? before : 0);
}

// SMALL: up to kSmall sequences, whose numbers then stay in shared memory (256 sequences: the call 17 us for 22).
constexpr int kSmall = 1024;
template <bool SMALL>
__global__ void __launch_bounds__(kPickThreads) pick_kernel(const ShareArgs a) {
  __shared__ int slots[32];
  __shared__ int groups, listed;
  __shared__ int32_t own[SMALL ? 8 * kSmall + 1 : 1];
  __shared__ unsigned long long own_best[SMALL ? kSmall : 1];
  tc::griddep_launch();
  tc::griddep_wait();
  const int seqs = a.tab.seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* const lead = SMALL ? own : a.lead;
  int32_t* const common = SMALL ? own + kSmall : a.common;
  int32_t* const rows_of = SMALL ? own + 2 * kSmall : a.n;
  int32_t* const pick = SMALL ? own + 3 * kSmall : a.pick;
  int32_t* const number = SMALL ? own + 4 * kSmall : a.number;   // of a leader's group; then a group's rows
  int32_t* const group = SMALL ? own + 5 * kSmall : a.group;
  int32_t* const first = SMALL ? own + 6 * kSmall : a.first;
  int32_t* const begin = SMALL ? own + 7 * kSmall : a.begin;     // [seqs + 1]
  int32_t* const size = SMALL ? number : a.size;
  unsigned long long* const best = SMALL ? own_best : a.best;
  if (SMALL) {
    if (tid < seqs) {
      lead[tid] = a.lead[tid];
      common[tid] = a.common[tid];
      rows_of[tid] = a.n[tid];
      best[tid] = 0;
    }
    __syncthreads();
  }
  // The pages of a leader's group: c pages shared by the leader and every follower with c or more in common save c times
  // their number page reads; the most of these, the larger c (the fewer followers) of two.  A warp a follower.
  for (int i = warp; i < seqs; i += kPickThreads / 32) {
    const int L = lead[i], c = common[i];
    if (L < 0 || L == i || c < a.min_pages) continue;
    int count = 0;
#pragma unroll 4
    for (int j = lane; j < seqs; j += 32) count += lead[j] == L && j != L && common[j] >= c ? 1 : 0;
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) atomicMax(best + L, (static_cast<unsigned long long>(c) * count) * kMostSeqs + (kMostSeqs - 1 - count));
  }
  if (tid == 0) groups = listed = 0;
  __syncthreads();
  for (int i = tid; i < seqs; i += kPickThreads) {
    const unsigned long long key = SMALL ? best[i] : __ldcg(best + i);   // atomics act in L2
    pick[i] = key == 0 ? 0 : static_cast<int>(key / kMostSeqs / (kMostSeqs - 1 - key % kMostSeqs));
  }
  __syncthreads();
  // groups in the order of their leaders
  for (int i0 = 0; i0 < seqs; i0 += kPickThreads) {
    const int i = i0 + tid;
    const bool head = i < seqs && pick[i] > 0;
    int total;
    const int at = groups + cta_prefix(head ? 1 : 0, slots, total);
    if (head) {
      number[i] = at;
      a.leader[at] = i;
    }
    __syncthreads();
    if (tid == 0) groups += total;
    __syncthreads();
  }
  for (int i = tid; i < seqs; i += kPickThreads) {
    const int L = lead[i];
    const bool in = L >= 0 && pick[L] > 0 && (L == i || common[i] >= pick[L]);
    group[i] = in ? number[L] : -1;
    if (SMALL) a.group[i] = in ? number[L] : -1;
    a.tokens[i] = in ? pick[L] << a.tab.ps_log2 : 0;
    first[i] = 0;
    if (i >= groups) a.leader[i] = -1;
  }
  __syncthreads();
  // a group's rows, and the rows of its members before each: a warp a group
  for (int g = warp; g < groups; g += kPickThreads / 32) {
    int at = 0;
    for (int i0 = 0; i0 < seqs; i0 += 32) {
      const int i = i0 + lane;
      const bool in = i < seqs && group[i] == g;
      if (!__any_sync(0xffffffffu, in)) continue;
      int inc = in ? rows_of[i] : 0;
      const int n = inc;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
      }
      if (in) first[i] = at + inc - n;
      at += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) size[g] = at;
  }
  __syncthreads();
  for (int g0 = 0; g0 < groups; g0 += kPickThreads) {
    const int g = g0 + tid;
    int total;
    const int at = listed + cta_prefix(g < groups ? size[g] : 0, slots, total);
    if (g < groups) begin[g] = at;
    __syncthreads();
    if (tid == 0) listed += total;
    __syncthreads();
  }
  for (int g = groups + tid; g <= seqs; g += kPickThreads) begin[g] = listed;
  __syncthreads();
  if (SMALL) {
    for (int i = tid; i <= seqs; i += kPickThreads) {
      a.begin[i] = begin[i];
      if (i < seqs) a.first[i] = first[i];
    }
  }
  for (int i = warp; i < seqs; i += kPickThreads / 32) {
    const int g = group[i];
    if (g < 0) continue;
    const int to = begin[g] + first[i], from = a.batch.cu[i], n = rows_of[i];
    for (int r = lane; r < n; r += 32)
      if (static_cast<uint32_t>(to) + r < static_cast<uint32_t>(a.batch.ntok)) a.rows[to + r] = from + r;   // ranges that overlap (refused offsets) stay inside the array
  }
  for (int r = max(0, listed) + tid; r < a.batch.ntok; r += kPickThreads) a.rows[r] = -1;
}

inline size_t up(size_t x) { return (x + 255) / 256 * 256; }
size_t share_bytes(int64_t seqs) { return 256 + 6 * up(4 * static_cast<size_t>(seqs)) + up(8 * static_cast<size_t>(seqs)); }

}  // namespace

fg_status check_share(const fg_page_share* s, const fg_page_table* t, int64_t ntok) {
  if (!s) return fail(FG_ERR_ARG, "null share");
  if (s->seqs != t->seqs || s->ntok != ntok)
    return fail(FG_ERR_SHAPE, "share of %lld sequences and %lld rows, batch of %lld and %lld", (long long)s->seqs, (long long)s->ntok,
                (long long)t->seqs, (long long)ntok);
  if (!s->group || !s->tokens || !s->first || !s->leader || !s->begin || (!s->rows && ntok > 0)) return fail(FG_ERR_ARG, "share: null arrays");
  if (!aligned(s->group, 4) || !aligned(s->tokens, 4) || !aligned(s->first, 4) || !aligned(s->leader, 4) || !aligned(s->begin, 4) ||
      !aligned(s->rows, 4))
    return fail(FG_ERR_ALIGN, "share: arrays need 4-byte alignment");
  return FG_OK;
}

}  // namespace paged
}  // namespace fg

using namespace fg;
using namespace fg::paged;

extern "C" {

size_t fg_pages_share_workspace_bytes(const fg_page_table* t) {
  if (check_table(t) != FG_OK) return 0;
  return share_bytes(t->seqs);
}

fg_status fg_pages_share(const fg_page_table* t, const int32_t* cu, int64_t min_tokens, const fg_page_share* s, void* ws, size_t ws_bytes,
                         cudaStream_t stream) {
  FG_TRY(check_table(t));
  if (t->seqs > static_cast<int64_t>(kMostSeqs)) return fail(FG_ERR_UNSUPPORTED, "sharing among more than %llu sequences", kMostSeqs);
  if (min_tokens < 1) return fail(FG_ERR_ARG, "min_tokens below 1");
  if (!s) return fail(FG_ERR_ARG, "null share");
  if (s->ntok < 0) return fail(FG_ERR_ARG, "negative row count");
  if (s->ntok > INT32_MAX - 256) return fail(FG_ERR_UNSUPPORTED, "more than 2^31 rows");
  if (t->seqs == 0) return s->seqs == 0 ? FG_OK : fail(FG_ERR_SHAPE, "share of other sequences");
  FG_TRY(check_share(s, t, s->ntok));
  if (!cu) return fail(FG_ERR_ARG, "null pointer");
  if (!aligned(cu, 4)) return fail(FG_ERR_ALIGN, "offsets need 4-byte alignment");
  if (!ws || ws_bytes < share_bytes(t->seqs)) return fail(FG_ERR_WORKSPACE, "sharing needs %zu workspace bytes", share_bytes(t->seqs));
  if (!aligned(ws, 256)) return fail(FG_ERR_ALIGN, "workspace needs 256-byte alignment");
  unsigned int* err = device_error_word();
  if (!err) return fail(FG_ERR_CUDA, "device error word");
  ShareArgs a;
  a.tab = table_of(*t);
  a.batch = Batch{cu, static_cast<int>(s->ntok), err};
  const int64_t pages = (min_tokens + t->page_size - 1) / t->page_size;
  a.min_pages = static_cast<int>(std::min<int64_t>(pages, INT32_MAX));
  a.group = s->group;
  a.tokens = s->tokens;
  a.first = s->first;
  a.leader = s->leader;
  a.begin = s->begin;
  a.rows = s->rows;
  char* p = static_cast<char*>(ws);
  for (int32_t** x : {&a.lead, &a.common, &a.n, &a.pick, &a.number, &a.size}) {
    *x = reinterpret_cast<int32_t*>(p);
    p += up(4 * static_cast<size_t>(t->seqs));
  }
  a.best = reinterpret_cast<unsigned long long*>(p);
  Trace tr(KC_PAGES_PLAN, stream);
  FG_TRY(paged::launch("compare_kernel", true, compare_kernel, static_cast<unsigned>((t->seqs + kWarps - 1) / kWarps), 32 * kWarps, 0, stream, a));
  trace_extra_launch();
  return paged::launch("pick_kernel", true, t->seqs <= kSmall ? pick_kernel<true> : pick_kernel<false>, 1, kPickThreads, 0, stream, a);
}

}  // extern "C"
