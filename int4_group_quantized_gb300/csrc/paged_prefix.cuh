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
  int64_t min_saved;      // tokens' reads that groups have to save; 0: groups whatever they save
};

constexpr int kPrefixKeysLog2 = 7;
// Rows of a group up to which it is not the chunks' kernel's.
constexpr int kPrefixFew = 128;
// What a read of a tile costs a unit of the chunks' kernel, in reads of a step's (some 14.5 ns over all SMs against 3 to 6), and
// what a row's parts, written and read again, cost its query heads, in tokens of their K/V head (6400 rows of 32 heads some 70 us
// where the heads have a K/V head each, as many where four share one: 5 to 20).
constexpr int kChunkRead = 4, kRowParts = 8;

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
// group's, as the share lists them, and the group is one of the line's (the first `groups`).
__device__ __forceinline__ int shared_tokens(const AttnArgs<__half>& a, int groups, int i) {
  const Prefix& p = a.prefix;
  const int g = p.group[i];
  if (g < 0 || g >= groups) return 0;
  const SharedGroup s = shared_group(p, a.tab, a.batch, g);
  const Seq q = seq_of(a.tab, a.batch, i);
  const int x = p.first[i];
  if (s.list == 0 || q.n == 0 || p.tokens[i] != s.tokens || q.len - q.n < s.tokens || x < 0 || x > s.list - q.n) return 0;
  const int32_t* rows = p.rows + s.first + x;
  return rows[0] == q.row0 && rows[q.n - 1] == q.row0 + q.n - 1 ? s.tokens : 0;
}

// What sequence i reads of its group's tokens when it goes by itself; nothing where it does so in any case.
__device__ __forceinline__ int64_t read_alone(const PrefixArgs& p, int groups, int i) {
  const AttnArgs<__half>& a = p.a;
  const int64_t tokens = shared_tokens(a, groups, i);
  if (tokens == 0) return 0;
  const int64_t rows = (static_cast<int64_t>(a.batch.cu[i + 1]) - a.batch.cu[i]) * a.shape.group;
  return tokens * (p.tile.workers == 0 || rows <= kStepRows ? 1 : kChunkRead * ((rows + kTileRows - 1) / kTileRows));
}
// What every CTA works out first, by all its threads: the whole line's length and share, what the launches after it read
// (written by the CTAs together), and where its own share begins.
struct PrefixLine {
  int64_t total, per;
  unsigned long long alone;   // reads of the groups' sequences by themselves; 0 before
  int groups;            // that are looked at, 0 where they do not save enough
  int g;                 // the group that the share begins in
  PrefixGroup at;
};
__device__ __forceinline__ void prefix_line(const PrefixArgs& p, PrefixLine& line) {   // line: in shared memory
  const AttnArgs<__half>& a = p.a;
  const Table& t = a.tab;
  const int group = a.shape.group, heads = a.pool.heads, lane = threadIdx.x & 31;
  if (p.min_saved > 0) {
    if (threadIdx.x < 32) {
      int groups = 0;
      bool last = false;
      for (; !last && groups < t.seqs; groups += 32) last = __any_sync(0xffffffffu, groups + lane < t.seqs && a.prefix.leader[groups + lane] < 0);
      if (lane == 0) line.groups = min(groups, t.seqs);
    }
    __syncthreads();
    int64_t sum = 0;
    for (int i = threadIdx.x; i < t.seqs; i += blockDim.x) sum += read_alone(p, line.groups, i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0 && sum > 0) atomicAdd(&line.alone, static_cast<unsigned long long>(sum));
    __syncthreads();
  }
  if (threadIdx.x < 32) {
    bool worth = true;
    int64_t per[2] = {1, 1};
    for (int pass = 0; pass < 2; ++pass) {
      int64_t spent = 0;                      // reads of the groups, and their parts
      int64_t at[2] = {0, 0};                 // of the two classes' lines
      const int64_t o0 = blockIdx.x * per[0];
      for (int g0 = 0; g0 < t.seqs; g0 += 32) {
        const int g = g0 + lane;
        SharedGroup s{-1, 0, 0, 0};
        if (g < t.seqs) s = shared_group(a.prefix, t, a.batch, g);
        if (!worth) s.list = 0;
        const bool tall = p.tile.workers > 0 && static_cast<int64_t>(s.list) * group > kPrefixFew;
        PrefixGroup x = prefix_group(s, group, tall);
        spent += static_cast<int64_t>(s.tokens) * x.units * (tall ? kChunkRead : 1) + static_cast<int64_t>(s.list) * group * kRowParts;
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
        if (!last) continue;
        const int groups = min(g0 + 32, t.seqs);
        if (pass == 1 && lane == 0) line.groups = worth ? groups : 0;
        if (pass == 1 && blockIdx.x == 0 && lane == 0) *a.prefix.planned = worth ? groups : 0;
        if (pass == 1 && blockIdx.x == 0 && p.tile.workers > 0)
          for (int i = groups + lane; i <= t.seqs; i += 32) p.tile.pre[i] = at[1];
        break;
      }
      if (pass == 0) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) spent += __shfl_xor_sync(0xffffffffu, spent, o);
        worth = p.min_saved == 0 || static_cast<int64_t>(line.alone) - spent >= p.min_saved;
        if (!worth) at[0] = at[1] = 0;
        per[0] = at[0] > p.workers ? (at[0] + p.workers - 1) / p.workers : 1;
        per[1] = p.tile.workers > 0 && at[1] > p.tile.workers ? (at[1] + p.tile.workers - 1) / p.tile.workers : 1;
        if (lane == 0) {
          line.total = at[0];
          line.per = per[0];
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
      const int skip = shared_tokens(a, line.groups, static_cast<int>(i));
      p.skip[i] = skip;
      if (skip > 0) a.prefix.home_row[i] = a.prefix.begin[a.prefix.group[i]] + a.prefix.first[i];
    }
}

fg_status paged_prefix(const PrefixArgs& p, int head_dim, cudaStream_t st);
// Behind it, and behind the chunks' kernel where that has groups: the parts of every row joined in its home.
fg_status paged_prefix_join(const PrefixArgs& p, int head_dim, cudaStream_t st);

}  // namespace paged
}  // namespace fg
