// Page bookkeeping of the paged 4-bit cache: growth, forking, freeing and
// compaction, decided on the device so that a serving step can be captured
// into a graph (FlexGen notes, "背景知识": the cache grows by Concat; the pages
// follow the sequences instead of one fixed block).
//
// A decision is a scan over refs (one int per page) and the sequences: a few
// hundred KB at most, so one CTA of 1024 threads makes it in two passes over
// contiguous warp segments (count, then write the lists), with one barrier
// between them.  The data then moves in one launch over all layers, reading
// the list of pages from the workspace.
#include <algorithm>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace fg {
namespace paged {

fg_status check_pool(const fg_page_pool* p) {
  if (!p) return fail(FG_ERR_ARG, "null page pool");
  if (p->dtype != FG_F16 && p->dtype != FG_F32) return fail(FG_ERR_ARG, "page pool dtype");
  if (p->pages <= 0 || p->heads <= 0) return fail(FG_ERR_ARG, "page pool sizes");
  if (p->pages > (1 << 25) || p->heads > 65535)
    return fail(FG_ERR_UNSUPPORTED, "page pool: more than 2^25 pages or 65535 heads");
  if (p->head_dim != 64 && p->head_dim != 128) return fail(FG_ERR_UNSUPPORTED, "head_dim %d (64 or 128)", p->head_dim);
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128 && p->page_size != 256)
    return fail(FG_ERR_SHAPE, "page_size %d (16, 32, 64, 128 or 256)", p->page_size);
  if (!p->k_codes || !p->v_codes || !p->k_mins || !p->k_scales || !p->v_mins || !p->v_scales)
    return fail(FG_ERR_ARG, "page pool: null arrays");
  if (!aligned(p->k_codes, 16) || !aligned(p->v_codes, 16) || !aligned(p->k_mins, 16) || !aligned(p->k_scales, 16) ||
      !aligned(p->v_mins, 16) || !aligned(p->v_scales, 16))
    return fail(FG_ERR_ALIGN, "page pool: arrays need 16-byte alignment");
  return FG_OK;
}

fg_status check_table(const fg_page_table* t) {
  if (!t) return fail(FG_ERR_ARG, "null page table");
  if (t->seqs < 0 || t->stride <= 0 || t->pages <= 0) return fail(FG_ERR_ARG, "page table sizes");
  if (t->page_size != 16 && t->page_size != 32 && t->page_size != 64 && t->page_size != 128 && t->page_size != 256)
    return fail(FG_ERR_SHAPE, "page_size %d (16, 32, 64, 128 or 256)", t->page_size);
  if (t->seqs > (1 << 20) || t->pages > (1 << 25) || t->stride > (int64_t(1) << 30) / t->page_size)
    return fail(FG_ERR_UNSUPPORTED, "page table: more than 2^20 sequences, 2^25 pages or 2^30 tokens of a sequence");
  if (!t->table || !t->lens || !t->refs) return fail(FG_ERR_ARG, "page table: null arrays");
  if (!aligned(t->table, 4) || !aligned(t->lens, 4) || !aligned(t->refs, 4))
    return fail(FG_ERR_ALIGN, "page table: arrays need 4-byte alignment");
  return FG_OK;
}

fg_status check_pool_table(const fg_page_pool* p, const fg_page_table* t) {
  FG_TRY(check_pool(p));
  FG_TRY(check_table(t));
  if (p->pages != t->pages || p->page_size != t->page_size)
    return fail(FG_ERR_SHAPE, "pool has %lld pages of %d, table %lld of %d", (long long)p->pages, p->page_size,
                (long long)t->pages, t->page_size);
  return FG_OK;
}

Pool pool_of(const fg_page_pool& p) {
  Pool a;
  a.codes[0] = p.k_codes;
  a.codes[1] = p.v_codes;
  a.mins[0] = p.k_mins;
  a.mins[1] = p.v_mins;
  a.scales[0] = p.k_scales;
  a.scales[1] = p.v_scales;
  a.pages = static_cast<int>(p.pages);
  a.heads = p.heads;
  a.ps_log2 = log2_of(p.page_size);
  return a;
}

Table table_of(const fg_page_table& t) {
  Table a;
  a.table = t.table;
  a.lens = t.lens;
  a.refs = t.refs;
  a.seqs = static_cast<int>(t.seqs);
  a.pages = static_cast<int>(t.pages);
  a.ps_log2 = log2_of(t.page_size);
  a.stride = t.stride;
  return a;
}

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// ---- workspace ----------------------------------------------------------------
// head[0]: pages to copy.  src, dst: their numbers [pages].  row: an int per
// sequence, fork: an int per fork.
struct Plan {
  int* head;
  int* src;
  int* dst;
  int* row;
  int* fork;
};
inline size_t up(size_t x) { return (x + 255) / 256 * 256; }
size_t plan_bytes(const fg_page_table& t, int64_t n) {
  return 256 + 2 * up(4 * static_cast<size_t>(t.pages)) + up(4 * static_cast<size_t>(t.seqs)) +
         up(4 * static_cast<size_t>(n));
}
Plan plan_of(const fg_page_table& t, void* ws) {
  Plan p;
  char* c = static_cast<char*>(ws);
  p.head = reinterpret_cast<int*>(c);
  c += 256;
  p.src = reinterpret_cast<int*>(c);
  c += up(4 * static_cast<size_t>(t.pages));
  p.dst = reinterpret_cast<int*>(c);
  c += up(4 * static_cast<size_t>(t.pages));
  p.row = reinterpret_cast<int*>(c);
  c += up(4 * static_cast<size_t>(t.seqs));
  p.fork = reinterpret_cast<int*>(c);
  return p;
}

// ---- scans over the CTA -----------------------------------------------------------
// A warp's share of n items: [begin, end).
__device__ __forceinline__ void warp_share(int n, int warp, int& begin, int& end) {
  const int per = (n + kPlanWarps - 1) / kPlanWarps;
  const int64_t b = static_cast<int64_t>(warp) * per;
  begin = b < n ? static_cast<int>(b) : n;
  end = b + per < n ? static_cast<int>(b + per) : n;
}
// Exclusive prefix of one value per warp over the CTA's warps, and the total.
// Holds two barriers; `slots` is shared memory of kPlanWarps ints.
__device__ __forceinline__ int warps_prefix(int value, int* slots, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) slots[warp] = value;
  __syncthreads();
  int v = slots[lane];   // kPlanWarps == 32
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  total = __shfl_sync(0xffffffffu, inc, 31);
  return __shfl_sync(0xffffffffu, inc - v, warp);
}
// Writes the ascending numbers x < n with pred(x) to list[0 .. limit) and
// returns how many there are (list may be null: count only).
template <class Pred>
__device__ __forceinline__ int list_where(int n, Pred pred, int* list, int limit, int* slots) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int begin, end;
  warp_share(n, warp, begin, end);
  int mine = 0;
#pragma unroll 4
  for (int x = begin + lane; x < end; x += 32) mine += pred(x) ? 1 : 0;
  mine = __reduce_add_sync(0xffffffffu, mine);
  int total;
  int at = warps_prefix(mine, slots, total);
  if (list != nullptr && at < limit) {
#pragma unroll 4
    for (int x0 = begin; x0 < end; x0 += 32) {
      const int x = x0 + lane;
      const bool on = x < end && pred(x);
      const uint32_t m = __ballot_sync(0xffffffffu, on);
      const int k = at + __popc(m & ((1u << lane) - 1));
      if (on && k < limit) list[k] = x;
      at += __popc(m);
    }
  }
  __syncthreads();   // the list is written
  return total;
}

__device__ __forceinline__ int pages_for(int64_t tokens, int ps_log2) {
  return static_cast<int>((tokens + (1 << ps_log2) - 1) >> ps_log2);
}

// ---- growth ------------------------------------------------------------------------
// Pages that sequence i lacks once its n new tokens are counted, cut at the
// row's end (`cut` then).
struct Growth {
  int have, add;
  int64_t len;
  bool bad, cut;
};
__device__ __forceinline__ Growth growth_of(const Table& t, const int32_t* cu, int i) {
  Growth g;
  const int64_t n = static_cast<int64_t>(cu[i + 1]) - cu[i];
  const int len = t.lens[i];
  g.bad = n < 0 || len < 0;
  g.len = g.bad ? len : len + n;
  if (g.len > INT32_MAX) {
    g.bad = true;
    g.len = len;
  }
  const int64_t have = g.bad ? 0 : pages_for(len, t.ps_log2), want = g.bad ? 0 : pages_for(g.len, t.ps_log2);
  g.cut = want > t.stride;
  const int64_t h = have < t.stride ? have : t.stride, w = want < t.stride ? want : t.stride;
  g.have = static_cast<int>(h);
  g.add = static_cast<int>(w - h);
  return g;
}

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const Table t, const int32_t* cu, Plan p,
                                                               unsigned int* err) {
  __shared__ int slots[kPlanWarps];
  tc::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int begin, end;
  warp_share(t.seqs, warp, begin, end);
  // how many pages the sequences lack: a warp's share counts as at most all
  // pages (2^25 of them), so the 32 shares add up in an int, and a warp that
  // begins past the last free page begins past it in the clipped sum too
  int64_t mine = 0;
  for (int i = begin + lane; i < end; i += 32) mine += growth_of(t, cu, i).add;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  int need;
  int64_t at = warps_prefix(static_cast<int>(mine < t.pages ? mine : t.pages), slots, need);
  const int limit = need < t.pages ? need : t.pages;
  const int nfree = need > 0 ? list_where(t.pages, [&](int x) { return t.refs[x] == 0; }, p.src, limit, slots) : 0;
  const int have_pages = nfree < limit ? nfree : limit;   // entries of p.src
  for (int i0 = begin; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    Growth g{0, 0, 0, false, false};
    if (i < end) {
      g = growth_of(t, cu, i);
      t.lens[i] = static_cast<int32_t>(g.len);
      if (g.bad) atomicOr(err, DEV_ERR_BATCH);
      if (g.cut) atomicOr(err, DEV_ERR_PAGE);
    }
    // the sequences that grow into new pages, one after another, the warp's
    // lanes along the entries
    uint32_t todo = __ballot_sync(0xffffffffu, g.add > 0);
    while (todo) {
      const int w = __ffs(todo) - 1;
      todo &= todo - 1;
      const int add = __shfl_sync(0xffffffffu, g.add, w), have = __shfl_sync(0xffffffffu, g.have, w);
      int32_t* row = t.table + (i0 + w) * t.stride + have;
      for (int k = lane; k < add; k += 32) {
        const bool got = at + k < have_pages;
        const int page = got ? p.src[at + k] : -1;
        row[k] = page;
        if (got) t.refs[page] = 1;
        else atomicOr(err, DEV_ERR_PAGE);
      }
      at += add;
    }
  }
}

// ---- freeing --------------------------------------------------------------------------
// One warp per named row; the exchange of the length decides which of two
// mentions of a row ends it.
__global__ void free_kernel(const Table t, const int32_t* rows, int n, unsigned int* err) {
  tc::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int k = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (k >= n) return;
  const int i = rows[k];
  if (i < 0 || i >= t.seqs) {
    if (lane == 0) atomicOr(err, DEV_ERR_BATCH);
    return;
  }
  int len = 0;
  if (lane == 0) len = atomicExch(t.lens + i, 0);
  len = __shfl_sync(0xffffffffu, len, 0);
  if (len <= 0) return;
  const int64_t held = pages_for(len, t.ps_log2);
  const int np = static_cast<int>(held < t.stride ? held : t.stride);
  for (int j = lane; j < np; j += 32) {
    int32_t* e = t.table + i * t.stride + j;
    const int page = *e;
    *e = -1;
    if (page >= 0 && page < t.pages) atomicSub(t.refs + page, 1);
  }
}

// ---- forking ---------------------------------------------------------------------------
// p.row[dst] = the first fork that names it; p.fork[k] = the source's length,
// -1 for a fork that is refused.  The copied page of fork k is entry k' of
// (src, dst), k' counting the forks with a page to copy before it: a source
// whose partly filled page is missing is refused first and takes none.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const Table t, const int32_t* src, const int32_t* dst,
                                                                 int n, Plan p, unsigned int* err) {
  __shared__ int slots[kPlanWarps];
  tc::griddep_launch();
  tc::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part_mask = (1 << t.ps_log2) - 1;
  auto in_range = [&](int x) { return x >= 0 && x < t.seqs; };
  for (int k = threadIdx.x; k < n; k += kPlanThreads)
    if (in_range(dst[k])) p.row[dst[k]] = INT32_MAX;
  __syncthreads();
  for (int k = threadIdx.x; k < n; k += kPlanThreads)
    if (in_range(dst[k])) atomicMin(p.row + dst[k], k);
  __syncthreads();
  int begin, end;
  warp_share(n, warp, begin, end);
  int mine = 0;
  for (int k = begin + lane; k < end; k += 32) {
    const int a = src[k], b = dst[k];
    const bool ok = in_range(a) && in_range(b) && a != b && p.row[b] == k && t.lens[b] == 0 && t.lens[a] >= 0 &&
                    pages_for(t.lens[a], t.ps_log2) <= t.stride;
    int len = ok ? t.lens[a] : -1;
    if (!ok) atomicOr(err, DEV_ERR_BATCH);
    if (ok && (len & part_mask)) {
      const int page = t.table[a * t.stride + (len >> t.ps_log2)];
      if (page >= 0 && page < t.pages) {
        ++mine;
      } else {
        atomicOr(err, DEV_ERR_PAGE);
        len = -1;
      }
    }
    p.fork[k] = len;
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  int need;
  int at = warps_prefix(mine, slots, need);
  const int limit = need < t.pages ? need : t.pages;
  const int nfree = need > 0 ? list_where(t.pages, [&](int x) { return t.refs[x] == 0; }, p.dst, limit, slots) : 0;
  // the rows' entries: lens and entries of a source are read as they were (a
  // source that is also a destination is empty), refs change by sums alone
  for (int k0 = begin; k0 < end; k0 += 32) {
    const int k = k0 + lane;
    const int len = k < end ? p.fork[k] : -1;
    const bool part = len > 0 && (len & part_mask);
    const uint32_t m = __ballot_sync(0xffffffffu, part);
    const int kk = at + __popc(m & ((1u << lane) - 1));
    at += __popc(m);
    if (len >= 0) {
      const int full = len >> t.ps_log2;
      const int32_t* from = t.table + src[k] * t.stride;
      int page = -1, fresh = -1;
      bool ok = true;
      if (part) {
        page = from[full];
        ok = kk < nfree && kk < limit;
        fresh = ok ? p.dst[kk] : -1;
        if (ok) p.src[kk] = page;
      }
      if (!ok) {
        p.fork[k] = -1;
        atomicOr(err, DEV_ERR_PAGE);
      } else if (part) {
        t.table[dst[k] * t.stride + full] = fresh;
        t.refs[fresh] = 1;
      }
    }
  }
  if (threadIdx.x == 0) p.head[0] = need < nfree ? need : (need > 0 ? nfree : 0);
  __syncthreads();
  // full pages: a warp per fork copies the entries and counts them
  for (int k = warp; k < n; k += kPlanWarps) {
    const int len = p.fork[k];
    if (len < 0) continue;
    const int full = len >> t.ps_log2;
    const int32_t* from = t.table + src[k] * t.stride;
    int32_t* to = t.table + dst[k] * t.stride;
    for (int j = lane; j < full; j += 32) {
      const int page = from[j];
      to[j] = page;
      if (page >= 0 && page < t.pages) atomicAdd(t.refs + page, 1);
    }
    if (lane == 0) t.lens[dst[k]] = len;
  }
}

// ---- compaction ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const Table t, Plan p) {
  __shared__ int slots[kPlanWarps];
  tc::griddep_launch();
  tc::griddep_wait();
  const int32_t* refs = t.refs;
  const int live = list_where(t.pages, [&](int x) { return refs[x] > 0; }, nullptr, 0, slots);
  const int moves = list_where(t.pages - live, [&](int x) { return refs[live + x] > 0; }, p.src, t.pages, slots);
  list_where(live, [&](int x) { return refs[x] <= 0; }, p.dst, t.pages, slots);
  if (threadIdx.x == 0) {
    p.head[0] = moves;
    p.head[1] = live;
  }
  for (int k = threadIdx.x; k < moves; k += kPlanThreads) {
    const int a = p.src[k] + live, b = p.dst[k];
    p.src[k] = a;
    t.refs[b] = t.refs[a];
    t.refs[a] = 0;
  }
}

// ---- the pages' data ------------------------------------------------------------------------
constexpr int kCopyLayers = 64;   // pools per launch (48 bytes of pointers each)
constexpr int kCopyUnits = 1024;  // 16-byte units of a piece
struct CopyArgs {
  void* base[kCopyLayers][6];
  const int* head;
  const int* src;
  const int* dst;
  int layers;
  int pages;
  int codes16, meta16;     // 16-byte units of a page in a codes / (min or scale) array
  int codes_n, meta_n;     // pieces of them
  Table tab;               // compaction: the table whose entries follow the moves (seqs 0: none)
};

// The table after the moves: an entry at or past the pages in use was moved;
// its place among the (ascending) sources is found by bisection.
__device__ __forceinline__ void move_entries(const CopyArgs& a, int moves) {
  const Table& t = a.tab;
  const int live = a.head[1];
  const int64_t n = t.seqs * t.stride;
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; x < n;
       x += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int i = static_cast<int>(x / t.stride);
    const int64_t j = x - i * t.stride;
    const int len = t.lens[i];
    if (len <= 0 || j >= pages_for(len, t.ps_log2)) continue;
    const int page = t.table[x];
    if (page < live || page >= t.pages) continue;
    int lo = 0, hi = moves;   // src[lo] <= page < src[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.src[mid] <= page) lo = mid;
      else hi = mid;
    }
    if (a.src[lo] == page) t.table[x] = a.dst[lo];
  }
}

// Pieces of at most 16 KB of (move, layer, array), dealt over the CTAs; a
// thread holds four units of a piece at once.  A source is never a
// destination, so the order does not matter.  Bound by the memory: 48 forks
// with a partly filled page in 8 layers (236 MB) 41 us by graph replay with
// their plan and the growth after it (5.8 TB/s), a compaction of 415 MB 72 us
// with the frees before it (5.8 TB/s); one unit in flight took 46 and 85.
__global__ void __launch_bounds__(256) copy_pages_kernel(const __grid_constant__ CopyArgs a) {
  tc::griddep_launch();
  tc::griddep_wait();
  const int moves = a.head[0];
  if (moves == 0) return;
  if (a.tab.seqs > 0) move_entries(a, moves);
  const int per = 2 * a.codes_n + 4 * a.meta_n;   // pieces of a page of a layer
  const int64_t items = static_cast<int64_t>(moves) * a.layers * per;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t ml = it / per;
    int c = static_cast<int>(it - ml * per);
    const int m = static_cast<int>(ml / a.layers), l = static_cast<int>(ml - static_cast<int64_t>(m) * a.layers);
    const int s = a.src[m], d = a.dst[m];
    if (s < 0 || s >= a.pages || d < 0 || d >= a.pages) continue;
    int arr, n;
    if (c < 2 * a.codes_n) {
      arr = c / a.codes_n;
      c -= arr * a.codes_n;
      n = a.codes16;
    } else {
      c -= 2 * a.codes_n;
      arr = c / a.meta_n;
      c -= arr * a.meta_n;
      arr += 2;
      n = a.meta16;
    }
    const uint4* from = static_cast<const uint4*>(a.base[l][arr]) + static_cast<int64_t>(s) * n;
    uint4* to = static_cast<uint4*>(a.base[l][arr]) + static_cast<int64_t>(d) * n;
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int x = c * kCopyUnits + u * 256 + threadIdx.x;
      if (x < n) v[u] = from[x];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int x = c * kCopyUnits + u * 256 + threadIdx.x;
      if (x < n) to[x] = v[u];
    }
  }
}

// Copies the plan's pages in all pools, and (tab given) moves the table's
// entries.
fg_status copy_pages(const fg_page_pool* pools, int l, const Plan& p, const fg_page_table* tab, cudaStream_t st) {
  for (int l0 = 0; l0 < l || l0 == 0; l0 += kCopyLayers) {
    CopyArgs a = {};
    a.layers = std::min(kCopyLayers, l - l0);
    for (int i = 0; i < a.layers; ++i) {
      const fg_page_pool& q = pools[l0 + i];
      a.base[i][0] = q.k_codes;
      a.base[i][1] = q.v_codes;
      a.base[i][2] = q.k_mins;
      a.base[i][3] = q.k_scales;
      a.base[i][4] = q.v_mins;
      a.base[i][5] = q.v_scales;
    }
    a.head = p.head;
    a.src = p.src;
    a.dst = p.dst;
    if (l > 0) {
      a.pages = static_cast<int>(pools[0].pages);
      const int64_t rows = static_cast<int64_t>(pools[0].heads) * pools[0].page_size;
      a.codes16 = static_cast<int>(rows * pools[0].head_dim / 32);
      a.meta16 = static_cast<int>(rows * pools[0].head_dim / 256);
      a.codes_n = (a.codes16 + kCopyUnits - 1) / kCopyUnits;
      a.meta_n = (a.meta16 + kCopyUnits - 1) / kCopyUnits;
    }
    if (tab && l0 == 0) a.tab = table_of(*tab);
    if (a.layers == 0 && a.tab.seqs == 0) break;
    Trace tr(KC_PAGES_COPY, st);
    FG_TRY(paged::launch("copy_pages_kernel", true, copy_pages_kernel, static_cast<unsigned>(num_sms() * 8), 256, 0, st, a));
  }
  return FG_OK;
}

fg_status check_pools(const fg_page_table* t, const fg_page_pool* pools, int32_t l) {
  if (l < 0) return fail(FG_ERR_ARG, "negative pool count");
  if (l > 0 && !pools) return fail(FG_ERR_ARG, "null pools");
  for (int32_t i = 0; i < l; ++i) {
    FG_TRY(check_pool_table(&pools[i], t));
    if (pools[i].heads != pools[0].heads || pools[i].head_dim != pools[0].head_dim)
      return fail(FG_ERR_SHAPE, "pool %d has other heads or head_dim than pool 0", i);
  }
  return FG_OK;
}

fg_status check_ws(const fg_page_table& t, int64_t n, const void* ws, size_t ws_bytes) {
  const size_t need = plan_bytes(t, n);
  if (!ws || ws_bytes < need) return fail(FG_ERR_WORKSPACE, "page bookkeeping needs %zu workspace bytes", need);
  if (!aligned(ws, 256)) return fail(FG_ERR_ALIGN, "workspace needs 256-byte alignment");
  return FG_OK;
}

}  // namespace
}  // namespace paged
}  // namespace fg

using namespace fg;
using namespace fg::paged;

extern "C" {

size_t fg_pages_workspace_bytes(const fg_page_table* t, int64_t n) {
  if (check_table(t) != FG_OK || n < 0 || n > INT32_MAX) return 0;
  return plan_bytes(*t, n);
}

fg_status fg_pages_reserve(const fg_page_table* t, const int32_t* cu, void* ws, size_t ws_bytes, cudaStream_t stream) {
  FG_TRY(check_table(t));
  if (!cu) return fail(FG_ERR_ARG, "null offsets");
  if (!aligned(cu, 4)) return fail(FG_ERR_ALIGN, "offsets need 4-byte alignment");
  FG_TRY(check_ws(*t, 0, ws, ws_bytes));
  if (t->seqs == 0) return FG_OK;
  unsigned int* err = device_error_word();
  if (!err) return fail(FG_ERR_CUDA, "device error word");
  Trace tr(KC_PAGES_PLAN, stream);
  return paged::launch("reserve_kernel", true, reserve_kernel, 1, kPlanThreads, 0, stream, table_of(*t), cu, plan_of(*t, ws), err);
}

fg_status fg_pages_free(const fg_page_table* t, const int32_t* rows, int64_t n, cudaStream_t stream) {
  FG_TRY(check_table(t));
  if (n < 0) return fail(FG_ERR_ARG, "negative count");
  if (n > (1 << 24)) return fail(FG_ERR_UNSUPPORTED, "more than 2^24 rows in a call");
  if (n == 0) return FG_OK;
  if (!rows) return fail(FG_ERR_ARG, "null rows");
  if (!aligned(rows, 4)) return fail(FG_ERR_ALIGN, "rows need 4-byte alignment");
  unsigned int* err = device_error_word();
  if (!err) return fail(FG_ERR_CUDA, "device error word");
  Trace tr(KC_PAGES_PLAN, stream);
  return paged::launch("free_kernel", true, free_kernel, static_cast<unsigned>((n + 3) / 4), 128, 0, stream, table_of(*t), rows,
                      static_cast<int>(n), err);
}

fg_status fg_pages_fork(const fg_page_table* t, const fg_page_pool* pools, int32_t l, const int32_t* src,
                        const int32_t* dst, int64_t n, void* ws, size_t ws_bytes, cudaStream_t stream) {
  FG_TRY(check_table(t));
  FG_TRY(check_pools(t, pools, l));
  if (n < 0) return fail(FG_ERR_ARG, "negative count");
  if (n > (1 << 20)) return fail(FG_ERR_UNSUPPORTED, "more than 2^20 forks in a call");
  if (n == 0) return FG_OK;
  if (!src || !dst) return fail(FG_ERR_ARG, "null lists");
  if (!aligned(src, 4) || !aligned(dst, 4)) return fail(FG_ERR_ALIGN, "lists need 4-byte alignment");
  FG_TRY(check_ws(*t, n, ws, ws_bytes));
  unsigned int* err = device_error_word();
  if (!err) return fail(FG_ERR_CUDA, "device error word");
  const Plan p = plan_of(*t, ws);
  {
    Trace tr(KC_PAGES_PLAN, stream);
    FG_TRY(paged::launch("fork_plan_kernel", true, fork_plan_kernel, 1, kPlanThreads, 0, stream, table_of(*t), src, dst,
                        static_cast<int>(n), p, err));
  }
  return copy_pages(pools, l, p, nullptr, stream);
}

fg_status fg_pages_compact(const fg_page_table* t, const fg_page_pool* pools, int32_t l, void* ws, size_t ws_bytes,
                           cudaStream_t stream) {
  FG_TRY(check_table(t));
  FG_TRY(check_pools(t, pools, l));
  FG_TRY(check_ws(*t, 0, ws, ws_bytes));
  const Plan p = plan_of(*t, ws);
  {
    Trace tr(KC_PAGES_PLAN, stream);
    FG_TRY(paged::launch("compact_plan_kernel", true, compact_plan_kernel, 1, kPlanThreads, 0, stream, table_of(*t), p));
  }
  return copy_pages(pools, l, p, t, stream);
}

}  // extern "C"
