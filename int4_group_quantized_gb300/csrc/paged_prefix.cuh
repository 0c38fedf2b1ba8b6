// Shared prefixes: how a call's work on them is dealt out.
//
// A group's rows (its sequences' rows, query heads of a K/V head side by side:
// list row * group + g) are cut into units, each against the tiles of 128 keys of
// the shared tokens, once per K/V head.  The units of all groups of a class, group
// by group, head by head, make a line of tiles, and worker w takes an equal run of
// it.  The first part of a unit goes to the rows' home, that of a worker that goes
// on with a unit to the worker's own place: a worker begins inside at most one.
//
// Two classes: in calls that allow chunks, the chunks of groups that have many
// rows of them go to the chunks' kernel (units of kTileRows rows), all other rows
// to this file's (units of at most kPrefixRows).
#pragma once

#include "paged_attn.cuh"

namespace fg {
namespace paged {

// What a call counts to find whether it shares, by class (0: paged_prefix.cu's rows, 1: the chunks' kernel's), in 24ths of one
// read of a token's K and V of a K/V head: a step's read of a token by itself is 24.
struct SharePrices {
  int chunk[2];           // a chunk's by itself, for each kTileRows of its rows
  int unit[2];            // a group's unit
  int unit_row;           // and each row of a unit of class 0
  int row;                // a row's parts, written and read again
  int64_t least[2];       // what a class's groups have to save; 0: groups whatever they save
};
struct PrefixArgs {
  AttnArgs<__half> a;
  int32_t* skip;          // [seqs] out: the tokens of a sequence that its group attends to
  ClassPlan tile;         // head and pre by group, out; no workers: one class
  int workers;
  SharePrices price;
};

constexpr int kPrefixKeysLog2 = 7;
// Rows of a group's chunks up to which they are not the chunks' kernel's.
constexpr int kPrefixFew = 128;
constexpr int kStepPrice = 24;

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
// group's, as the share lists them, and the group is one of the line's (the first `groups`).  n: its rows.  (Loads that do not
// need one another come first.)
__device__ __forceinline__ int shared_tokens(const AttnArgs<__half>& a, int groups, int i, int& n) {
  const Prefix& p = a.prefix;
  const int g = p.group[i], x = p.first[i], tokens = p.tokens[i];
  const Seq q = seq_of(a.tab, a.batch, i);
  n = q.n;
  if (g < 0 || g >= groups || q.n == 0 || x < 0 || x > a.batch.ntok) return 0;
  const int64_t at = static_cast<int64_t>(p.begin[g]) + x;
  const bool inside = at >= 0 && at + q.n <= a.batch.ntok;
  const int row0 = inside ? p.rows[at] : -1, row1 = inside ? p.rows[at + q.n - 1] : -1;
  const SharedGroup s = shared_group(p, a.tab, a.batch, g);
  return s.list > 0 && tokens == s.tokens && q.len - q.n >= s.tokens && x <= s.list - q.n && row0 == q.row0 && row1 == q.row0 + q.n - 1 ? s.tokens : 0;
}
// Groups that are looked at: up to the first gap, 32 at a time (by a warp).
__device__ __forceinline__ int groups_of(const Prefix& p, int seqs) {
  const int lane = threadIdx.x & 31;
  int groups = 0;
  for (bool last = false; !last && groups < seqs; groups += 32) last = __any_sync(0xffffffffu, groups + lane < seqs && p.leader[groups + lane] < 0);
  return min(groups, seqs);
}
// The whole line's length and share, what the launches after it read, and where the CTA's own share begins.  Worked out by all
// threads of every CTA of paged_prefix.cu's kernel, which write what the others read together; in calls with chunks
// (PLANNED) by one CTA before them.
struct PrefixLine {
  int64_t total, per;
  unsigned long long alone[2];   // reads of the groups' sequences by themselves, by class; 0 before
  bool worth[2];         // whether a class's groups save enough
  int groups;            // that are looked at
  int g;                 // the group that the share begins in
  PrefixGroup at;
};
// shared(groups, i, n, tall): the tokens that sequence i leaves to its group, its rows and their class.
template <bool PLANNED, class F>
__device__ __forceinline__ void prefix_line(const PrefixArgs& p, PrefixLine& line, F shared) {   // line: in shared memory
  const AttnArgs<__half>& a = p.a;
  const Table& t = a.tab;
  const int group = a.shape.group, heads = a.pool.heads, lane = threadIdx.x & 31;
  bool worth[2] = {true, true};
  int64_t per[2] = {1, 1}, spent[2], all[2];   // (warp 0) reads of the groups and their parts, and the classes' lines
  // Groups up to the first gap, 32 at a time: what the classes' lines hold and cost, and (write) where each lies in them.
  auto walk = [&](bool write) {
    int64_t at[2] = {0, 0};
    spent[0] = spent[1] = 0;
    const int64_t o0 = blockIdx.x * per[0];
    int groups = 0;
    for (bool last = false; !last; groups += 32) {
      const int g = groups + lane;
      ClassRows s[2] = {{{-1, 0, 0, 0}, false}, {{-1, 0, 0, 0}, false}};
      if (g < t.seqs) {
        s[0] = class_rows(a.prefix, t, a.batch, g, false);
        if (PLANNED) s[1] = class_rows(a.prefix, t, a.batch, g, true);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (!worth[c]) s[c].list = 0;
      PrefixGroup x[2] = {prefix_group(s[0], group, false), prefix_group(s[1], group, true)};
      int64_t inc[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        spent[c] += static_cast<int64_t>(s[c].tokens) * x[c].units * (p.price.unit[c] + (c ? 0 : p.price.unit_row * x[c].rows)) +
                    static_cast<int64_t>(s[c].list) * group * p.price.row;
        x[c].base = inc[c] = static_cast<int64_t>(heads) * x[c].units * x[c].tiles;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int64_t up = __shfl_up_sync(0xffffffffu, inc[c], o);
          if (lane >= o) inc[c] += up;
        }
      if (write) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          x[c].base = at[c] + inc[c] - x[c].base;
          x[c].per = per[c];
          x[c].extra = c ? p.workers * kPrefixRows : 0;
        }
        if (blockIdx.x == 0 && g < t.seqs) {
          a.prefix.info[g] = x[0];
          if (PLANNED) {
            a.prefix.info[t.seqs + g] = x[1];
            p.tile.pre[g] = x[1].base;
          }
        }
        if (o0 >= x[0].base && o0 < at[0] + inc[0]) {
          line.g = g;
          line.at = x[0];
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) at[c] += __shfl_sync(0xffffffffu, inc[c], 31);
      last = __any_sync(0xffffffffu, s[0].leader < 0) || groups + 32 >= t.seqs;
    }
    all[0] = at[0];
    all[1] = at[1];
    groups = min(groups, t.seqs);
    if (PLANNED && write)
      for (int i = groups + lane; i <= t.seqs; i += 32) p.tile.pre[i] = at[1];
    return groups;
  };
  if (threadIdx.x < 32) {
    const int groups = walk(false);
    if (lane == 0) line.groups = groups;
  } else if (p.price.least[0] > 0 || p.price.least[1] > 0) {   // meanwhile, by the other warps
    const int groups = PLANNED ? 0 : groups_of(a.prefix, t.seqs);
    int64_t sum[2] = {0, 0};
    for (int i = threadIdx.x - 32; i < t.seqs; i += blockDim.x - 32) {   // what a sequence's reads count when it goes by itself
      int n, tall;
      const int64_t tokens = shared(groups, i, n, tall), rows = static_cast<int64_t>(n) * group;
      const int64_t reads = tokens * (!PLANNED || rows <= kStepRows ? kStepPrice : p.price.chunk[tall] * ((rows + kTileRows - 1) / kTileRows));
      sum[0] += tall ? 0 : reads;
      sum[1] += tall ? reads : 0;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], o);
      if (lane == 0 && sum[c] > 0) atomicAdd(&line.alone[c], static_cast<unsigned long long>(sum[c]));
    }
  }
  __syncthreads();
  if (threadIdx.x < 32) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) spent[c] += __shfl_xor_sync(0xffffffffu, spent[c], o);
      worth[c] = p.price.least[c] == 0 || static_cast<int64_t>(line.alone[c]) - spent[c] >= p.price.least[c];
      if (!worth[c]) all[c] = 0;
    }
    per[0] = all[0] > p.workers ? (all[0] + p.workers - 1) / p.workers : 1;
    if (PLANNED) per[1] = all[1] > p.tile.workers ? (all[1] + p.tile.workers - 1) / p.tile.workers : 1;
    if (lane == 0) {
      line.total = all[0];
      line.per = per[0];
      line.worth[0] = worth[0];
      line.worth[1] = worth[1];
      if (blockIdx.x == 0) {
        *a.prefix.planned = worth[0] || worth[1] ? line.groups : 0;
        if (PLANNED) {
          a.prefix.head[0] = all[0];
          a.prefix.head[1] = per[0];
          p.tile.head[0] = all[1];
          p.tile.head[1] = per[1];
        }
      }
    }
    if (worth[0] || worth[1]) walk(true);
  }
  __syncthreads();
  // the sequences one a CTA in turn, by warps that are not in a hurry
  const int from = PLANNED ? 0 : 128, width = PLANNED ? static_cast<int>(blockDim.x) : 128;
  if (threadIdx.x >= from && threadIdx.x < from + width)
    for (int64_t i = blockIdx.x + static_cast<int64_t>(gridDim.x) * (threadIdx.x - from); i < t.seqs; i += static_cast<int64_t>(gridDim.x) * width) {
      int n, tall, skip = 0;
      if (line.worth[0] || line.worth[1]) {
        skip = shared(line.groups, static_cast<int>(i), n, tall);
        if (!line.worth[tall]) skip = 0;
      }
      p.skip[i] = skip;
      if (skip > 0) a.prefix.home_row[i] = a.prefix.begin[a.prefix.group[i]] + a.prefix.first[i];
    }
}
// Where the CTA's share begins, by every warp, of a line that was worked out before.
__device__ __forceinline__ void planned_line(const PrefixArgs& p, PrefixLine& line) {
  const AttnArgs<__half>& a = p.a;
  const int lane = threadIdx.x & 31, planned = *a.prefix.planned;
  const int64_t total = a.prefix.head[0], per = a.prefix.head[1], o0 = blockIdx.x * per;
  if (threadIdx.x == 0) {
    line.total = total;
    line.per = per;
  }
  if (o0 < total && threadIdx.x < 32)
    for (int g0 = 0; g0 < planned; g0 += 32) {
      if (g0 + lane >= planned) continue;
      const PrefixGroup x = a.prefix.info[g0 + lane];
      const int64_t n = static_cast<int64_t>(a.pool.heads) * x.units * x.tiles;
      if (o0 >= x.base && o0 < x.base + n) {
        line.g = g0 + lane;
        line.at = x;
      }
    }
  __syncthreads();
}

// In calls that allow chunks, first: the line, groups' steps and chunks apart.
fg_status paged_prefix_plan(const PrefixArgs& p, cudaStream_t st);
fg_status paged_prefix(const PrefixArgs& p, int head_dim, cudaStream_t st);
// Behind it, and behind the chunks' kernel where that has groups: the parts of every row joined in its home.
fg_status paged_prefix_join(const PrefixArgs& p, int head_dim, cudaStream_t st);

}  // namespace paged
}  // namespace fg
