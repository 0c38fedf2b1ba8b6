// Shared prefixes: how a call's work on them is dealt out.
//
// A group's rows (its sequences' rows, query heads of a K/V head side by side:
// list row * group + g) are cut into units, each against the tiles of 128 keys of
// the shared tokens, once per K/V head.  The units of all groups of a class, group
// by group, head by head, make a line of tiles, and worker w takes an equal run of
// it.  The first part of a unit goes to the rows' home, that of a worker that goes
// on with a unit to the worker's own place: a worker begins inside at most one.
//
// Two classes: groups of many rows in calls that allow chunks go to the chunks'
// kernel (units of kTileRows rows), all others to this file's (units of at most
// kPrefixRows).
#pragma once

#include "paged_attn.cuh"

namespace fg {
namespace paged {

struct PrefixArgs {
  AttnArgs<__half> a;
  int32_t* skip;          // [seqs] out: the tokens of a sequence that its group attends to
  ClassPlan tile;         // head and pre by group, out; no workers: one class
  int workers;
  int64_t min_saved;      // tokens, times the rows that do not read them again, from which on groups are made
};

constexpr int kPrefixKeysLog2 = 7;
// Rows of a group up to which it is not the chunks' kernel's.
constexpr int kPrefixFew = 128;

__device__ __forceinline__ PrefixGroup prefix_group(const SharedGroup& s, int group, bool tall) {
  PrefixGroup g;
  const int most = tall ? kTileRows : kPrefixRows;
  const int rows = s.list * group, units = (rows + most - 1) / most;
  g.base = g.per = 0;
  g.tiles = (s.tokens + (1 << kPrefixKeysLog2) - 1) >> kPrefixKeysLog2;
  g.rows = tall ? kTileRows : units > 0 ? ((rows + units - 1) / units + 15) / 16 * 16 : 16;   // a unit's rows are as many columns of an MMA
  g.units = (rows + g.rows - 1) / g.rows;
  g.first_row = s.first;
  g.extra = 0;
  g.stride = most;
  return g;
}
// The tokens that sequence i leaves to its group: those of its group if all of its rows stand behind them and are the
// group's, as the share lists them.
__device__ __forceinline__ int shared_tokens(const AttnArgs<__half>& a, int i) {
  const Prefix& p = a.prefix;
  const int g = p.group[i];
  if (g < 0 || g >= a.tab.seqs) return 0;
  const SharedGroup s = shared_group(p, a.tab, a.batch, g);
  const Seq q = seq_of(a.tab, a.batch, i);
  const int x = p.first[i];
  if (s.list == 0 || q.n == 0 || p.tokens[i] != s.tokens || q.len - q.n < s.tokens || x < 0 || x > s.list - q.n) return 0;
  const int32_t* rows = p.rows + s.first + x;
  return rows[0] == q.row0 && rows[q.n - 1] == q.row0 + q.n - 1 ? s.tokens : 0;
}

// What every CTA works out first, by all its threads: the whole line's length and share, what the launches after it read
// (written by the CTAs together), and where its own share begins.
struct PrefixLine {
  int64_t total, per;
  bool worth;            // the groups save enough
  int g;                 // the group that the share begins in
  PrefixGroup at;
};
__device__ __forceinline__ void prefix_line(const PrefixArgs& p, PrefixLine& line) {   // line: in shared memory
  const AttnArgs<__half>& a = p.a;
  const Table& t = a.tab;
  const int group = a.shape.group, heads = a.pool.heads, lane = threadIdx.x & 31;
  bool worth = true;
  if (threadIdx.x < 32) {
    int64_t per[2] = {1, 1};
    for (int pass = 0; pass < 2; ++pass) {
      int64_t saved = 0;                      // tokens that are not read again
      int64_t at[2] = {0, 0};                 // of the two classes' lines
      const int64_t o0 = blockIdx.x * per[0];
      for (int g0 = 0; g0 < t.seqs; g0 += 32) {
        const int g = g0 + lane;
        SharedGroup s{-1, 0, 0, 0};
        if (g < t.seqs) s = shared_group(a.prefix, t, a.batch, g);
        saved += s.list > 0 ? static_cast<int64_t>(s.tokens) * (s.list - 1) : 0;
        if (!worth) s.list = 0;
        const bool tall = p.tile.workers > 0 && static_cast<int64_t>(s.list) * group > kPrefixFew;
        PrefixGroup x = prefix_group(s, group, tall);
        const int64_t n = s.list > 0 ? static_cast<int64_t>(heads) * x.units * x.tiles : 0;
        int64_t inc[2] = {tall ? 0 : n, tall ? n : 0};
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int64_t up = __shfl_up_sync(0xffffffffu, inc[c], o);
            if (lane >= o) inc[c] += up;
          }
        if (pass == 1) {
          x.base = tall ? at[1] + inc[1] - n : at[0] + inc[0] - n;
          x.per = tall ? per[1] : per[0];
          x.extra = tall ? p.workers * kPrefixRows : 0;
          if (blockIdx.x == 0 && g < t.seqs) {
            a.prefix.info[g] = x;
            if (p.tile.workers > 0) p.tile.pre[g] = at[1] + inc[1] - (tall ? n : 0);
          }
          if (!tall && n > 0 && o0 >= x.base && o0 < x.base + n) {
            line.g = g;
            line.at = x;
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) at[c] += __shfl_sync(0xffffffffu, inc[c], 31);
        const bool last = __any_sync(0xffffffffu, s.leader < 0) || g0 + 32 >= t.seqs;   // past the last group
        if (last && pass == 1 && blockIdx.x == 0 && lane == 0) *a.prefix.planned = g0 + 32 < t.seqs ? g0 + 32 : t.seqs;
        if (last && pass == 1 && blockIdx.x == 0 && p.tile.workers > 0)
          for (int i = g0 + 32 + lane; i <= t.seqs; i += 32) p.tile.pre[i] = at[1];
        if (last) break;
      }
      if (pass == 0) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) saved += __shfl_xor_sync(0xffffffffu, saved, o);
        worth = saved >= p.min_saved;
        if (!worth) at[0] = at[1] = 0;
        per[0] = at[0] > p.workers ? (at[0] + p.workers - 1) / p.workers : 1;
        per[1] = p.tile.workers > 0 && at[1] > p.tile.workers ? (at[1] + p.tile.workers - 1) / p.tile.workers : 1;
        if (lane == 0) {
          line.total = at[0];
          line.per = per[0];
          line.worth = worth;
          if (blockIdx.x == 0 && p.tile.workers > 0) {
            p.tile.head[0] = at[1];
            p.tile.head[1] = per[1];
          }
        }
      }
    }
  }
  __syncthreads();
  // the sequences one a CTA in turn, by warps that are not in a hurry
  if (threadIdx.x >= 128 && threadIdx.x < 256)
    for (int64_t i = blockIdx.x + static_cast<int64_t>(gridDim.x) * (threadIdx.x - 128); i < t.seqs; i += static_cast<int64_t>(gridDim.x) * 128) {
      const int skip = line.worth ? shared_tokens(a, static_cast<int>(i)) : 0;
      p.skip[i] = skip;
      if (skip > 0) a.prefix.home_row[i] = a.prefix.begin[a.prefix.group[i]] + a.prefix.first[i];
    }
}

fg_status paged_prefix(const PrefixArgs& p, int head_dim, cudaStream_t st);
// Behind it, and behind the chunks' kernel where that has groups: the parts of every row joined in its home.
fg_status paged_prefix_join(const PrefixArgs& p, int head_dim, cudaStream_t st);

}  // namespace paged
}  // namespace fg
