// Internal interface of the paged attention kernels.
#pragma once

#include "paged_sched.cuh"

namespace fg {
namespace paged {

// What the rows of a shared prefix's groups left behind (paged_prefix.cu, and paged_tile.cu for groups of many rows): sums,
// maximum (base 2) and normaliser of every row over its group's prefix, in parts.  Part 0 of a row is its home; the parts of
// later shares of the line are in the shares' own places until they are joined there (paged_prefix_join).
struct PrefixGroup {
  int64_t base, per;    // tiles of its line before the group, and of a share of the line
  int tiles, rows, units;   // tiles of a unit, rows of a unit, units of a head
  int first_row;        // of the group in the share's list
  int extra, stride;    // rows of `extra` before its line's places, and of a place
};
struct Prefix {
  const int32_t *group, *tokens, *first, *leader, *begin, *rows;   // fg_page_share
  // calls with chunks (else null): of a group whose chunks are the chunks' kernel's the rows of its steps and of its chunks,
  // [seqs] each, steps -1 where it is not split so; and its places in the list, its steps' first, then its chunks'
  int32_t *steps, *chunks, *order;
  int32_t *member, *before;       // [seqs] the group that a sequence leaves tokens to, -1: none; rows of its kind and group before its own
  int64_t* head;                  // tiles of paged_prefix.cu's line, and of a share of it
  PrefixGroup* info;              // [*planned], groups that are none with no units among them; [seqs + *planned] of their chunks
  int32_t* planned;
  int32_t* home_row;              // [seqs] the home of a sequence's first row
  float* home;                    // [ntok][q_heads][D], rows in the share's order
  float2* home_stat;              // [ntok][q_heads]
  float* extra;                   // [workers][kPrefixRows][D], then [workers][kTileRows][D]: of the unit that a share goes on with
  float2* extra_stat;
};
constexpr int kPrefixRows = 64;   // most rows of a unit of paged_prefix.cu

// The home of row t of a sequence (Table::skip of it > 0), query head hq.
__device__ __forceinline__ int64_t prefix_home(const Prefix& p, int seq, int t, int hq, int q_heads) {
  return static_cast<int64_t>(p.home_row[seq] + t) * q_heads + hq;
}

// Group g as the share has it; list = 0: none, or not one that can be followed.
struct SharedGroup {
  int leader, tokens, first, list;
};
__device__ __forceinline__ SharedGroup shared_group(const Prefix& p, const Table& t, const Batch& b, int g) {
  SharedGroup s{p.leader[g], 0, p.begin[g], 0};
  const int end = p.begin[g + 1];
  if (s.leader < 0 || s.leader >= t.seqs) return s;
  s.tokens = p.tokens[s.leader];
  const bool ok = s.tokens > 0 && (s.tokens & ((1 << t.ps_log2) - 1)) == 0 && s.tokens <= (t.stride << t.ps_log2) && s.first >= 0 &&
                  end > s.first && end <= b.ntok;
  s.list = ok ? end - s.first : 0;
  return s;
}
// The rows of group g that go to the chunks' kernel (tall), or to the other, as a part of the list, by `order` where the group
// is split: a step is not to be rounded as chunks are because a chunk shares its prefix.
struct ClassRows : SharedGroup {
  bool split;
};
__device__ __forceinline__ ClassRows class_rows(const Prefix& p, const Table& t, const Batch& b, int g, bool tall) {
  ClassRows s{shared_group(p, t, b, g), false};
  const int steps = p.steps != nullptr && s.list > 0 ? p.steps[g] : -1;
  s.split = steps >= 0;
  if (!s.split) {
    if (tall) s.list = 0;
  } else {
    s.first += tall ? steps : 0;
    s.list = tall ? p.chunks[g] : steps;
  }
  return s;
}
__device__ __forceinline__ int place_of(const Prefix& p, const ClassRows& s, int x) { return s.split ? p.order[x] : x; }
// Row x of the share's list as a row of the batch (row 0 in place of what is none: nobody reads its parts).
__device__ __forceinline__ int listed_row(const Prefix& p, const Batch& b, int x) {
  const int r = p.rows[x];
  return r >= 0 && r < b.ntok ? r : 0;
}

template <typename T>
struct AttnArgs {
  Pool pool;
  Table tab;
  Batch batch;
  const T* q;
  T* out;
  int64_t ldq, ldo;
  int q_heads;
  AttnShape shape;
  float scale;        // 1 / sqrt(head_dim)
  float scale_log2;   // times log2(e)
  Prefix prefix;      // with Table::skip
};

// own_plan: no plan was made (paged_sched.cuh, make_line).
// Sequences of at most kStepRows rows per K/V head (fp16).
int step_workers(int rows, int sms);
// With a.tab.skip the sequences go on from their shared prefixes' parts (a.prefix), here and in the chunks' kernel.
fg_status paged_attention_step(const AttnArgs<__half>& a, const ClassPlan& pl, int head_dim, bool own_plan, cudaStream_t st);

// Longer chunks (fp16) on tcgen05, units of kTileRows rows and tiles of 128 keys; one worker an SM.
constexpr int kTileRows = 256;
// `every`: the call has no step class.
fg_status paged_attention_tile(const AttnArgs<__half>& a, const ClassPlan& pl, int head_dim, bool own_plan, bool every, cudaStream_t st);
// The prefixes of the groups in pl's line (pl.head, pl.pre by group), by the same kernel.
fg_status paged_prefix_tile(const AttnArgs<__half>& a, const ClassPlan& pl, int head_dim, cudaStream_t st);

// fp32 activations, every sequence: units of kF32Rows rows, tiles of 64 keys.
constexpr int kF32Rows = 16, kF32KeysLog2 = 6;
int f32_workers(int head_dim, int sms);
fg_status paged_attention_f32(const AttnArgs<float>& a, const ClassPlan& pl, int head_dim, bool own_plan, cudaStream_t st);

}  // namespace paged
}  // namespace fg
