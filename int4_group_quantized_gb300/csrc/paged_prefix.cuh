// Shared prefixes: how a call's work on them is dealt out.
//
// A group's rows (its sequences' rows, query heads of a K/V head side by side:
// list row * group + g) are cut into units of at most kPrefixRows, each against
// the tiles of 128 keys of the shared tokens, once per K/V head.  All units of all
// groups, group by group, head by head, make a line of tiles, and worker w takes an
// equal run of it.  The first part of a unit goes to the rows' home, that of a
// worker that goes on with a unit to the worker's own place: a worker begins
// inside at most one.
#pragma once

#include "paged_attn.cuh"

namespace fg {
namespace paged {

struct PrefixArgs {
  AttnArgs<__half> a;
  const int32_t *tokens, *leader, *begin, *rows;   // fg_page_share
  int32_t* skip;          // [seqs] out: the tokens of a sequence that its group attends to
  int workers;
};

constexpr int kPrefixKeysLog2 = 7;

// Group g as the share has it; list = 0: none, or not one that can be followed.
struct SharedGroup {
  int leader, tokens, first, list;
};
__device__ __forceinline__ SharedGroup shared_group(const PrefixArgs& p, int g) {
  const Table& t = p.a.tab;
  SharedGroup s{p.leader[g], 0, p.begin[g], 0};
  const int end = p.begin[g + 1];
  if (s.leader < 0 || s.leader >= t.seqs) return s;
  s.tokens = p.tokens[s.leader];
  const bool ok = s.tokens > 0 && (s.tokens & ((1 << t.ps_log2) - 1)) == 0 && s.tokens <= (t.stride << t.ps_log2) && s.first >= 0 &&
                  end > s.first && end <= p.a.batch.ntok;
  s.list = ok ? end - s.first : 0;
  return s;
}
__device__ __forceinline__ PrefixGroup prefix_group(const SharedGroup& s, int group, int64_t base) {
  PrefixGroup g;
  const int rows = s.list * group, units = (rows + kPrefixRows - 1) / kPrefixRows;
  g.base = base;
  g.tiles = (s.tokens + (1 << kPrefixKeysLog2) - 1) >> kPrefixKeysLog2;
  g.rows = units > 0 ? ((rows + units - 1) / units + 15) / 16 * 16 : 16;   // a unit's rows are as many columns of an MMA
  g.units = (rows + g.rows - 1) / g.rows;
  g.first_row = s.first;
  return g;
}
// The tokens that sequence i leaves to its group: those of its group if all of its rows stand behind them and are the
// group's, as the share lists them.
__device__ __forceinline__ int shared_tokens(const PrefixArgs& p, int i) {
  const Table& t = p.a.tab;
  const int g = p.a.prefix.group[i];
  if (g < 0 || g >= t.seqs) return 0;
  const SharedGroup s = shared_group(p, g);
  const Seq q = seq_of(t, p.a.batch, i);
  const int x = p.a.prefix.first[i];
  if (s.list == 0 || q.n == 0 || p.tokens[i] != s.tokens || q.len - q.n < s.tokens || x < 0 || x > s.list - q.n) return 0;
  const int32_t* rows = p.rows + s.first + x;
  return rows[0] == q.row0 && rows[q.n - 1] == q.row0 + q.n - 1 ? s.tokens : 0;
}

// What every CTA works out first, by all its threads: the whole line's length and share, what the calls after it read
// (written by the CTAs together), and where its own share begins.
struct PrefixLine {
  int64_t total, per;
  int g;                 // the group that the share begins in
  PrefixGroup at;
};
__device__ __forceinline__ void prefix_line(const PrefixArgs& p, PrefixLine& line) {   // line: in shared memory
  const Table& t = p.a.tab;
  const int group = p.a.shape.group, heads = p.a.pool.heads, lane = threadIdx.x & 31;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < t.seqs; i += gridDim.x * blockDim.x) p.skip[i] = shared_tokens(p, i);
  if (threadIdx.x < 32) {
    for (int pass = 0; pass < 2; ++pass) {
      int64_t at = 0;
      const int64_t o0 = pass ? blockIdx.x * line.per : 0;
      for (int g0 = 0; g0 < t.seqs; g0 += 32) {
        const int g = g0 + lane;
        SharedGroup s{-1, 0, 0, 0};
        if (g < t.seqs) s = shared_group(p, g);
        const PrefixGroup x = prefix_group(s, group, 0);
        const int64_t n = s.list > 0 ? static_cast<int64_t>(heads) * x.units * x.tiles : 0;
        int64_t inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += up;
        }
        if (pass == 1) {
          const PrefixGroup y = prefix_group(s, group, at + inc - n);
          if (blockIdx.x == 0 && g < t.seqs) p.a.prefix.info[g] = y;
          if (n > 0 && o0 >= y.base && o0 < y.base + n) {
            line.g = g;
            line.at = y;
          }
        }
        at += __shfl_sync(0xffffffffu, inc, 31);
        if (__any_sync(0xffffffffu, s.leader < 0)) break;   // past the last group
      }
      if (pass == 0 && lane == 0) {
        line.total = at;
        line.per = at > p.workers ? (at + p.workers - 1) / p.workers : 1;
        if (blockIdx.x == 0) *p.a.prefix.per = line.per;
      }
      __syncwarp();
    }
  }
  __syncthreads();
}

fg_status paged_prefix(const PrefixArgs& p, int head_dim, cudaStream_t st);

}  // namespace paged
}  // namespace fg
