// Attention of a ragged batch of chunks over the paged 4-bit cache (FlexGen
// notes, "背景知识": Softmax(x_Q x_K^T / sqrt(h1)) x_V per head, causal; "5.
// 近似方法": K and V stored in 4-bit groups of 64).
//
// Here: the plan that deals the work out, the joining of partials, the
// workspace and the entry point.  The kernels: paged_step.cu (fp16, sequences
// of few rows), paged_tile.cu (fp16, longer chunks), paged_f32.cu.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "paged_attn.cuh"
#include "paged_prefix.cuh"
#include "tc_ptx.cuh"

namespace fg {
namespace paged {
namespace {

__device__ __forceinline__ void put4(float* p, const float4& v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void put4(__half* p, const float4& v) {
  const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// ---- the plan -------------------------------------------------------------------
// One CTA: the tiles of every sequence, class by class, as prefix sums, and
// the size of a share.  A warp takes a run of sequences, a lane one of them; a
// chunk's units are counted by the warp's lanes together, one chunk after
// another, in the first of two passes (which leaves the counts where the prefix
// sums go).
constexpr int kPlanThreads = 1024;

struct PlanArgs {
  Table tab;
  Batch batch;
  AttnShape shape;
  int heads;
  ClassPlan step, tile;   // a class with no workers is not used
};

template <int TRU, int TKTL, bool SKIP>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
  __shared__ int64_t warp_sum[2][32];
  __shared__ int warp_max[2][32];
  tc::griddep_launch();
  tc::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nwarps = blockDim.x >> 5;
  const int seqs = a.tab.seqs, per = (seqs + nwarps - 1) / nwarps;
  const int begin = min(seqs, warp * per), end = min(seqs, begin + per);
  int64_t sum[2] = {0, 0};
  int longest[2] = {0, 0};
  for (int pass = 0; pass < 2; ++pass) {
    int64_t at[2] = {0, 0};
    if (pass == 1) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (lane == 0) {
          warp_sum[c][warp] = sum[c];
          warp_max[c][warp] = longest[c];
        }
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        int64_t v = lane < nwarps ? warp_sum[c][lane] : 0, inc = v;
        int mx = lane < nwarps ? warp_max[c][lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += up;
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        }
        const int64_t total = __shfl_sync(0xffffffffu, inc, 31);
        at[c] = __shfl_sync(0xffffffffu, inc - v, warp);
        const ClassPlan& p = c ? a.tile : a.step;
        if (threadIdx.x == 0 && p.workers > 0) {
          p.head[0] = total;
          p.head[1] = share_of(total, mx, p.workers, c ? 1 : kStepFew);
          p.pre[seqs] = total;
        }
      }
    }
    for (int i0 = begin; i0 < end; i0 += 32) {
      const int i = i0 + lane;
      int64_t cost[2] = {0, 0};
      bool tall = false;
      Seq s{0, 0, 0, 0, 0};
      if (pass == 1 && i < end) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const ClassPlan& p = c ? a.tile : a.step;
          if (p.workers > 0) cost[c] = p.pre[i];
        }
      }
      if (pass == 0 && i < end) {
        s = seq_of<SKIP>(a.tab, a.batch, i);
        if (s.n > a.shape.max_q) {
          atomicOr(a.batch.err, DEV_ERR_BATCH);
          s.n = 0;
        }
        const int64_t rows = static_cast<int64_t>(s.n) * a.shape.group;
        if (rows > 0 && a.step.workers > 0 && rows <= kStepRows) {
          const int tiles = step_tiles(s, a.shape);
          cost[0] = static_cast<int64_t>(tiles) * a.heads;
          longest[0] = max(longest[0], tiles);
        } else if (rows > 0 && a.tile.workers > 0) {
          tall = true;
          longest[1] = max(longest[1], longest_unit<TRU, TKTL>(s, a.shape));
        }
      }
      uint32_t todo = __ballot_sync(0xffffffffu, tall);
      while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        Seq t{0, 0, 0, 0, 0};
        t.n = __shfl_sync(0xffffffffu, s.n, src);
        t.len = __shfl_sync(0xffffffffu, s.len, src);
        t.keys = __shfl_sync(0xffffffffu, s.keys, src);
        int64_t c = units_tiles<TRU, TKTL>(t, a.shape, lane, 32);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
        if (lane == src) cost[1] = c * a.heads;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        int64_t inc = cost[c];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += up;
        }
        const ClassPlan& p = c ? a.tile : a.step;
        if (i < end && p.workers > 0) p.pre[i] = pass == 0 ? cost[c] : at[c] + inc - cost[c];
        const int64_t all = __shfl_sync(0xffffffffu, inc, 31);
        at[c] += all;
        if (pass == 0) sum[c] += all;
      }
    }
    if (pass == 0)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) longest[c] = max(longest[c], __shfl_xor_sync(0xffffffffu, longest[c], o));
  }
}

// ---- joining the partials of items that cross shares ------------------------------
// A block joins 16 rows of the item that begins in share w and ends later: the partials
// lie in slot 1 of w and slot 0 of the shares after it.  Up to four shares are
// loaded at once, four columns a lane.  Of more the factors of all (share, row)
// first, then the sums: a warp per row and part of the shares, the parts added
// in order (the same bits every time).
constexpr int kJoinWarps = 8;
constexpr int kJoinRows = 16;

template <typename T, int D, int RU>
__device__ __forceinline__ void join_rows(const AttnArgs<T>& a, const ClassPlan& pl, int w, int n0) {
  constexpr int kRows = kJoinRows;
  constexpr int kCols = D / 4;                // lanes of a row
  __shared__ float fac[(kMaxSplits + 2) * kRows];
  __shared__ float norm[kRows];
  __shared__ float4 sums[kJoinWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 rec = pl.rec[w];
  if (rec.x < 0) return;
  const Seq s = seq_of(a.tab, a.batch, rec.x);
  const Unit x = unit_of<RU>(s, a.shape.group, rec.z);
  const int shares = rec.w - w + 1;
  auto slot = [&](int k, int n) { return (static_cast<int64_t>(w + k) * 2 + (k == 0 ? 1 : 0)) * pl.rows + n; };
  auto write = [&](int n, int col, const float4& o, float f) {   // four columns of row n0 + n
    const int row = x.r0 + n0 + n, t = row / a.shape.group;
    T* dst = a.out + static_cast<int64_t>(s.row0 + t) * a.ldo +
             static_cast<int64_t>(rec.y * a.shape.group + row - t * a.shape.group) * D + 4 * col;
    put4(dst, make_float4(o.x * f, o.y * f, o.z * f, o.w * f));
  };
  if (n0 >= x.rows) return;
  constexpr int kFew = 4;
  if (shares <= kFew) {   // the usual case: everything is loaded at once
    constexpr int kAtOnce = kJoinWarps * 32 / kCols;   // rows
    const int col = threadIdx.x % kCols;
#pragma unroll
    for (int r = 0; r < kRows; r += kAtOnce) {
      const int n = r + threadIdx.x / kCols;
      if (n0 + n >= x.rows) continue;
      float2 st[kFew];
      float4 v[kFew];
#pragma unroll
      for (int k = 0; k < kFew; ++k) {
        st[k] = make_float2(-INFINITY, 0.0f);
        v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (k < shares) {
          st[k] = pl.stat[slot(k, n0 + n)];
          v[k] = *reinterpret_cast<const float4*>(pl.part + slot(k, n0 + n) * D + 4 * col);
        }
      }
      const float m = fmaxf(fmaxf(st[0].x, st[1].x), fmaxf(st[2].x, st[3].x)), base = m == -INFINITY ? 0.0f : m;
      float l = 0.0f;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kFew; ++k) {
        const float f = exp2f(st[k].x - base);
        l += f * st[k].y;
        o.x = fmaf(f, v[k].x, o.x);
        o.y = fmaf(f, v[k].y, o.y);
        o.z = fmaf(f, v[k].z, o.z);
        o.w = fmaf(f, v[k].w, o.w);
      }
      write(n, col, o, l == 0.0f ? 0.0f : 1.0f / l);
    }
    return;
  }
  {
    const int rows = min(kRows, x.rows - n0);
    for (int n = warp; n < rows; n += kJoinWarps) {
      float m = -INFINITY;
      for (int k = lane; k < shares; k += 32) m = fmaxf(m, pl.stat[slot(k, n0 + n)].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float base = m == -INFINITY ? 0.0f : m;
      float l = 0.0f;
      for (int k = lane; k < shares; k += 32) {
        const float2 st = pl.stat[slot(k, n0 + n)];
        const float f = exp2f(st.x - base);
        fac[k * kRows + n] = f;
        l += f * st.y;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (lane == 0) norm[n] = l == 0.0f ? 0.0f : 1.0f / l;
    }
    __syncthreads();
    // (row, part) pairs over half warps (D = 64) or warps (D = 128)
    constexpr int kTeams = kJoinWarps * 32 / kCols;
    const int team = threadIdx.x / kCols, col = threadIdx.x % kCols;
    int parts = 1;
    while (parts * 2 * rows <= kTeams && parts * 2 <= shares) parts *= 2;
    for (int r0 = 0; r0 < rows; r0 += kTeams / parts) {
      const int n = r0 + team / parts, part = team % parts;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (n < rows) {
#pragma unroll 8
        for (int k = part; k < shares; k += parts) {
          const float4 v = *reinterpret_cast<const float4*>(pl.part + slot(k, n0 + n) * D + 4 * col);
          const float f = fac[k * kRows + n];
          o.x = fmaf(f, v.x, o.x);
          o.y = fmaf(f, v.y, o.y);
          o.z = fmaf(f, v.z, o.z);
          o.w = fmaf(f, v.w, o.w);
        }
      }
      if (parts > 1) {
        sums[warp][lane] = o;
        __syncthreads();
        if (part == 0)
          for (int q = 1; q < parts; ++q) {
            const int tid = threadIdx.x + q * kCols;
            const float4 v = sums[tid >> 5][tid & 31];
            o.x += v.x;
            o.y += v.y;
            o.z += v.z;
            o.w += v.w;
          }
        __syncthreads();
      }
      if (n < rows && part == 0) write(n, col, o, norm[n]);
    }
  }
}

// Blocks 0 .. step.workers - 1: the steps' shares; then 16 rows of each of the
// chunks' shares.
template <typename T, int D, int RU>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const AttnArgs<T> a, const ClassPlan step, const ClassPlan tile) {
  tc::griddep_launch();
  tc::griddep_wait();
  const int b = static_cast<int>(blockIdx.x) - step.workers;
  if (b < 0) {
    join_rows<T, D, kStepRows>(a, step, blockIdx.x, 0);
  } else {
    constexpr int kParts = RU / kJoinRows;
    join_rows<T, D, RU>(a, tile, b / kParts, b % kParts * kJoinRows);
  }
}

template <typename T, int D, int RU>
fg_status join(const AttnArgs<T>& a, const ClassPlan& step, const ClassPlan& tile, cudaStream_t st) {
  Trace tr(KC_ATTN_COMBINE, st);
  return paged::launch("join_kernel", true, join_kernel<T, D, RU>, static_cast<unsigned>(step.workers + tile.workers * (RU / kJoinRows)),
                      32 * kJoinWarps, 0, st, a, step, tile);
}

// ---- when a call shares ------------------------------------------------------------------
// By min_saved, the reads that the header counts: a chunk's four times a step's, a group's unit once or four times, 8 tokens for
// a row's parts.  By the library's own rule, what the launches take, in reads of one token of one K/V head (64 dims take as long
// as 128), from 880 calls of 2 to 256 sequences of 1 to 400 rows over one prefix of 128 to 32,768 tokens, with 32 heads of 128,
// 32 on 8, 64 on 8, 16, and 12 of 64, over inputs larger than L2, each timed by fg_paged_attention and shared:
//   class 0: 256 rows of a chunk as three steps, a group's unit as two and a 24th of one for each row, a row's parts as 32 tokens,
//     the launches as 500 thousand reads.  Of 290 calls of steps 7 are more than 5% slower than the faster way, in all 0.5%, of 102
//     with a few chunks none.  By fg_paged_attention and shared, us: 16 sequences, 32 heads, 1,024 tokens 33 and 38 (goes alone),
//     2,048 60 and 41; 64 sequences 512 tokens 66 and 65, 1,024 94 and 66; 4 sequences 8,192 tokens 44 and 55 (alone), 32,768 160
//     and 133.
//   class 1: 256 rows of a chunk as four, of a group as five, parts as 32 tokens, the launches as 900 thousand.  Of 492 calls 13, in
//     all 0.5%.  16 sequences, 32 heads, 20 rows over 1,024 tokens 102 and 108 (alone), 1,536 126 and 112; 128 rows over 2,048 161
//     and 203 (alone), 8,192 458 and 371; 48 of 32 rows over 512 186 and 221 (alone), 1,024 262 and 241.
// A call that goes alone by it takes 6 us (steps) or 7 to 19 (chunks) more than fg_paged_attention: the launches that find it out.
// (One limit of 64 MB by the header's count for both took calls that are up to 1.7 times as slow.)
constexpr SharePrices kCounted = {{4 * kStepPrice, 4 * kStepPrice}, {kStepPrice, 4 * kStepPrice}, 0, 8 * kStepPrice, {0, 0}};
constexpr SharePrices kMeasured = {{3 * kStepPrice, 4 * kStepPrice}, {2 * kStepPrice, 5 * kStepPrice}, 1, 32 * kStepPrice, {500000, 900000}};

// ---- workspace ------------------------------------------------------------------------
constexpr int kMaxSms = 160;   // a workspace fits this many SMs; launches use no more
inline size_t up(size_t x) { return (x + 255) / 256 * 256; }

struct Layout {
  ClassPlan step, tile;
  Prefix prefix;     // of a call beside shared prefixes
  ClassPlan tall;    // its groups of many rows of chunks
  int32_t* skip;
  size_t bytes;
};
void carve_class(ClassPlan& c, char*& p, int64_t seqs, int head_dim, int workers, int most, int rows) {
  c.workers = workers;
  c.rows = rows;
  if (workers == 0) return;
  c.head = reinterpret_cast<int64_t*>(p);
  p += 256;
  c.pre = reinterpret_cast<int64_t*>(p);
  p += up(8 * static_cast<size_t>(seqs + 1));
  c.rec = reinterpret_cast<int4*>(p);
  p += up(16 * static_cast<size_t>(most));
  c.stat = reinterpret_cast<float2*>(p);
  p += up(16 * static_cast<size_t>(most) * rows);
  c.part = reinterpret_cast<float*>(p);
  p += up(8 * static_cast<size_t>(most) * rows * head_dim);
}
// The classes that a call of at most max_q rows a sequence can need.
Layout layout_of(const fg_page_pool& pool, const fg_page_table& t, int32_t q_heads, int64_t max_q, void* ws, int sms, int64_t shared_rows = -1) {
  Layout l;
  const int64_t group = q_heads / pool.heads, most = std::min<int64_t>(max_q, INT32_MAX) * group;
  char* p = static_cast<char*>(ws);
  memset(&l.step, 0, sizeof(l.step));
  memset(&l.tile, 0, sizeof(l.tile));
  if (pool.dtype == FG_F16 && group <= kStepRows) {
    const int rows = most <= 8 ? 8 : kStepRows;
    carve_class(l.step, p, t.seqs, pool.head_dim, step_workers(rows, sms), step_workers(rows, kMaxSms), rows);
  }
  if (pool.dtype == FG_F32)
    carve_class(l.tile, p, t.seqs, pool.head_dim, f32_workers(pool.head_dim, sms), f32_workers(pool.head_dim, kMaxSms), kF32Rows);
  else if (most > (l.step.workers ? kStepRows : 0))
    carve_class(l.tile, p, t.seqs, pool.head_dim, sms, kMaxSms, kTileRows);
  memset(&l.prefix, 0, sizeof(l.prefix));
  memset(&l.tall, 0, sizeof(l.tall));
  l.skip = nullptr;
  if (shared_rows >= 0) {
    const size_t pairs = static_cast<size_t>(shared_rows) * q_heads, d = pool.head_dim;
    auto take = [&](auto*& x, size_t bytes) {
      x = reinterpret_cast<std::remove_reference_t<decltype(x)>>(p);
      p += up(bytes);
    };
    take(l.skip, 4 * static_cast<size_t>(t.seqs));
    take(l.prefix.info, sizeof(PrefixGroup) * static_cast<size_t>(t.seqs) * (l.tile.workers ? 2 : 1));
    take(l.prefix.home_row, 4 * static_cast<size_t>(t.seqs));
    take(l.prefix.planned, 4);
    const size_t extra = static_cast<size_t>(kMaxSms) * (kPrefixRows + (l.tile.workers ? kTileRows : 0));
    if (l.tile.workers) {
      l.tall.workers = l.tile.workers;
      l.tall.rows = kTileRows;
      take(l.tall.head, 256);
      take(l.tall.pre, 8 * static_cast<size_t>(t.seqs + 1));
      for (int32_t** x : {&l.prefix.steps, &l.prefix.chunks, &l.prefix.member, &l.prefix.before}) take(*x, 4 * static_cast<size_t>(t.seqs));
      take(l.prefix.order, 4 * static_cast<size_t>(shared_rows));
      take(l.prefix.head, 16);
    }
    take(l.prefix.home_stat, 8 * pairs);
    take(l.prefix.extra_stat, 8 * extra);
    take(l.prefix.home, 4 * pairs * d);
    take(l.prefix.extra, 4 * extra * d);
  }
  l.bytes = static_cast<size_t>(p - static_cast<char*>(ws)) + 256;
  return l;
}

template <typename T>
fg_status launch_attn(const fg_page_pool& pool, const fg_page_table& t, const int32_t* cu, const void* q, int64_t ldq,
                      int32_t q_heads, int64_t ntok, int64_t max_q, int64_t window, int64_t sinks, void* out,
                      int64_t ldo, void* ws, unsigned int* err, cudaStream_t st, const fg_page_share* share = nullptr, const SharePrices& price = kCounted) {
  AttnArgs<T> a;
  a.pool = pool_of(pool);
  a.tab = table_of(t);
  a.batch = Batch{cu, static_cast<int>(ntok), err};
  a.q = static_cast<const T*>(q);
  a.out = static_cast<T*>(out);
  a.ldq = ldq;
  a.ldo = ldo;
  a.q_heads = q_heads;
  const double scale = 1.0 / sqrt(static_cast<double>(pool.head_dim));
  a.scale = static_cast<float>(scale);
  a.scale_log2 = static_cast<float>(scale * 1.4426950408889634074);
  a.shape.group = q_heads / pool.heads;
  a.shape.max_q = static_cast<int>(std::min<int64_t>(max_q, ntok));
  // positions are below 2^31: a wider window hides nothing
  a.shape.window = window > (int64_t(1) << 30) ? 0 : static_cast<int>(window);
  a.shape.sinks = static_cast<int>(std::min<int64_t>(sinks, int64_t(1) << 30));
  const Layout l = layout_of(pool, t, q_heads, max_q, ws, std::min(num_sms(), kMaxSms), share ? ntok : -1);
  constexpr bool half = sizeof(T) == 2;
  a.prefix = l.prefix;
  if constexpr (half) {
    if (share) {
      a.prefix.group = share->group;
      a.prefix.tokens = share->tokens;
      a.prefix.first = share->first;
      a.prefix.leader = share->leader;
      a.prefix.begin = share->begin;
      a.prefix.rows = share->rows;
      const PrefixArgs p{a, l.skip, l.tall, std::min(num_sms(), kMaxSms), price};
      if (l.tall.workers > 0) FG_TRY(paged_prefix_plan(p, st));
      FG_TRY(paged_prefix(p, pool.head_dim, st));
      if (l.tall.workers > 0) FG_TRY(paged_prefix_tile(a, l.tall, pool.head_dim, st));
      FG_TRY(paged_prefix_join(p, pool.head_dim, st));
      a.tab.skip = l.skip;
    }
  }
  const bool wide = pool.head_dim == 128;
  const bool own_plan = t.seqs <= kOwnPlan;
  if (!own_plan) {
    PlanArgs p{a.tab, a.batch, a.shape, pool.heads, l.step, l.tile};
    Trace tr(KC_ATTN_PAGED_PLAN, st);
    // all warps where there are chunks to count (129 of 20 rows: the call 107 us, 122 with a lane a sequence and no more);
    // for steps alone a lane a sequence (129: 33.1 us, 34.5 with all)
    const unsigned lanes = static_cast<unsigned>(std::min<int64_t>(kPlanThreads, (t.seqs + 31) / 32 * 32));
    const unsigned threads = l.tile.workers > 0 ? kPlanThreads : lanes;
    const auto plan = !half ? plan_kernel<kF32Rows, kF32KeysLog2, false> : a.tab.skip ? plan_kernel<kTileRows, 7, true> : plan_kernel<kTileRows, 7, false>;
    FG_TRY(paged::launch("plan_kernel", true, plan, 1, threads, 0, st, p));
  }
  if constexpr (half) {
    // One after the other: a kernel reads nothing before those before it are complete.  (Steps that were set up beside the
    // chunks' last shares and read the plan and the lengths without that wait: 63 single tokens beside a chunk of 512 rows
    // 355 us for 362, with shared heads 141.5 for 142.5, 100 beside 28 chunks of 20 rows 83.7 for 81; chunks first and the
    // steps behind them 372, 157 and 95.)
    if (l.step.workers > 0) FG_TRY(paged_attention_step(a, l.step, pool.head_dim, own_plan, st));
    if (l.tile.workers > 0) FG_TRY(paged_attention_tile(a, l.tile, pool.head_dim, own_plan, l.step.workers == 0, st));
    return wide ? join<T, 128, kTileRows>(a, l.step, l.tile, st) : join<T, 64, kTileRows>(a, l.step, l.tile, st);
  } else {
    FG_TRY(paged_attention_f32(a, l.tile, pool.head_dim, own_plan, st));
    return wide ? join<T, 128, kF32Rows>(a, l.step, l.tile, st) : join<T, 64, kF32Rows>(a, l.step, l.tile, st);
  }
}

fg_status check_attn(const fg_page_pool* pool, const fg_page_table* t, int32_t q_heads, int64_t ntok, int64_t max_q) {
  FG_TRY(check_pool_table(pool, t));
  if (q_heads <= 0 || ntok < 0 || max_q < 0) return fail(FG_ERR_ARG, "attention sizes");
  if (q_heads % pool->heads)
    return fail(FG_ERR_SHAPE, "q_heads %d is no multiple of the pool's %d heads", q_heads, pool->heads);
  if (ntok > INT32_MAX || ntok * q_heads > INT32_MAX - 1024) return fail(FG_ERR_UNSUPPORTED, "more than 2^31 (row, head) pairs");
  // a worker counts its tiles in an int: units of at least 16 rows, tiles of at least 32 tokens, at least 64 workers
  const double units = static_cast<double>(ntok) * (q_heads / pool->heads) / 16 + t->seqs;
  const double tiles = static_cast<double>(t->stride) * t->page_size / 32 + 2;
  if (units * tiles * pool->heads / 64 > 2e9) return fail(FG_ERR_UNSUPPORTED, "more than 2^31 tiles for a worker");
  return FG_OK;
}

fg_status check_rows(const fg_page_pool* pool, const int32_t* cu, const void* q, int64_t ldq, int32_t q_heads, const void* out, int64_t ldo) {
  if (!cu || !q || !out) return fail(FG_ERR_ARG, "null pointer");
  const int64_t h1 = static_cast<int64_t>(q_heads) * pool->head_dim;
  if (ldq < h1 || ldo < h1) return fail(FG_ERR_SHAPE, "row stride below q_heads * head_dim = %lld", (long long)h1);
  if (!aligned(cu, 4) || !aligned(q, 16) || !aligned(out, 16) || ldq % 8 || ldo % 8)
    return fail(FG_ERR_ALIGN, "q and out need 16-byte alignment and strides that are multiples of 8");
  return FG_OK;
}

}  // namespace
}  // namespace paged
}  // namespace fg

using namespace fg;
using namespace fg::paged;

extern "C" {

size_t fg_paged_attention_workspace_bytes(const fg_page_pool* pool, const fg_page_table* t, int32_t q_heads,
                                          int64_t ntok, int64_t max_q) {
  if (check_attn(pool, t, q_heads, ntok, max_q) != FG_OK) return 0;
  return layout_of(*pool, *t, q_heads, max_q, nullptr, kMaxSms).bytes;
}

fg_status fg_paged_attention(const fg_page_pool* pool, const fg_page_table* t, const int32_t* cu, const void* q,
                             int64_t ldq, int32_t q_heads, int64_t ntok, int64_t max_q, int64_t window, int64_t sinks,
                             void* out, int64_t ldo, void* ws, size_t ws_bytes, cudaStream_t stream) {
  FG_TRY(check_attn(pool, t, q_heads, ntok, max_q));
  if (window < 0 || sinks < 0) return fail(FG_ERR_ARG, "negative window or sinks");
  if (ntok == 0 || max_q == 0 || t->seqs == 0) return FG_OK;
  FG_TRY(check_rows(pool, cu, q, ldq, q_heads, out, ldo));
  const size_t need = fg_paged_attention_workspace_bytes(pool, t, q_heads, ntok, max_q);
  if (!ws || ws_bytes < need) return fail(FG_ERR_WORKSPACE, "paged attention needs %zu workspace bytes", need);
  if (!aligned(ws, 256)) return fail(FG_ERR_ALIGN, "workspace needs 256-byte alignment");
  unsigned int* err = device_error_word();
  if (!err) return fail(FG_ERR_CUDA, "device error word");
  if (pool->dtype == FG_F16)
    return launch_attn<__half>(*pool, *t, cu, q, ldq, q_heads, ntok, max_q, window, sinks, out, ldo, ws, err, stream);
  return launch_attn<float>(*pool, *t, cu, q, ldq, q_heads, ntok, max_q, window, sinks, out, ldo, ws, err, stream);
}

size_t fg_paged_attention_shared_workspace_bytes(const fg_page_pool* pool, const fg_page_table* t, int32_t q_heads, int64_t ntok,
                                                 int64_t max_q) {
  if (check_attn(pool, t, q_heads, ntok, max_q) != FG_OK) return 0;
  return layout_of(*pool, *t, q_heads, max_q, nullptr, kMaxSms, pool->dtype == FG_F16 ? ntok : -1).bytes;
}

fg_status fg_paged_attention_shared(const fg_page_pool* pool, const fg_page_table* t, const int32_t* cu, const fg_page_share* s,
                                    const void* q, int64_t ldq, int32_t q_heads, int64_t ntok, int64_t max_q, int64_t min_saved, void* out,
                                    int64_t ldo, void* ws, size_t ws_bytes, cudaStream_t stream) {
  FG_TRY(check_attn(pool, t, q_heads, ntok, max_q));
  if (!s) return fail(FG_ERR_ARG, "null share");
  if (ntok == 0 || max_q == 0 || t->seqs == 0) return FG_OK;
  FG_TRY(check_share(s, t, ntok));
  if (pool->dtype == FG_F32)   // every sequence by itself: no kernel here takes a group's fp32 rows together
    return fg_paged_attention(pool, t, cu, q, ldq, q_heads, ntok, max_q, 0, 0, out, ldo, ws, ws_bytes, stream);
  FG_TRY(check_rows(pool, cu, q, ldq, q_heads, out, ldo));
  const size_t need = fg_paged_attention_shared_workspace_bytes(pool, t, q_heads, ntok, max_q);
  if (!ws || ws_bytes < need) return fail(FG_ERR_WORKSPACE, "shared paged attention needs %zu workspace bytes", need);
  if (!aligned(ws, 256)) return fail(FG_ERR_ALIGN, "workspace needs 256-byte alignment");
  unsigned int* err = device_error_word();
  if (!err) return fail(FG_ERR_CUDA, "device error word");
  // in tokens; K and V of one are 1.25 bytes an element
  const int64_t token = static_cast<int64_t>(pool->heads) * pool->head_dim * 5 / 4;
  SharePrices price = min_saved < 0 ? kMeasured : kCounted;
  for (int64_t& least : price.least) {
    const int64_t of = min_saved < 0 ? least : min_saved, one = min_saved < 0 ? pool->heads : token, tokens = of / one + (of % one != 0);
    least = std::min(tokens, INT64_MAX / kStepPrice) * kStepPrice;
  }
  // all sequences' reads of all that a table row can name are no less than what groups can save
  const double group = static_cast<double>(q_heads / pool->heads), most = static_cast<double>(std::min<int64_t>(t->seqs, ntok));
  const double reads = max_q * group <= kStepRows ? kStepPrice * most : 4 * kStepPrice * (most + static_cast<double>(ntok) * group / kTileRows);
  const int64_t least = std::min(price.least[0], price.least[1]);
  const bool never = least > 0 && static_cast<double>(t->stride) * t->page_size * reads < static_cast<double>(least);
  return launch_attn<__half>(*pool, *t, cu, q, ldq, q_heads, ntok, max_q, 0, 0, out, ldo, ws, err, stream, never ? nullptr : s, price);
}

}  // extern "C"
