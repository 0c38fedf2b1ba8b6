// Internal interface of the paged attention kernels.
#pragma once

#include "paged_sched.cuh"

namespace fg {
namespace paged {

// What the rows of a shared prefix's groups left behind (paged_prefix.cu): sums, maximum (base 2) and normaliser of every
// row over its group's prefix, in parts.  Part 0 of a row is its home; the parts of later shares are theirs.
struct PrefixGroup {
  int64_t base;         // tiles of the line before the group
  int tiles, rows, units;   // tiles of a unit, rows of a unit, units of a head
  int first_row;        // of the group in the share's list
};
struct Prefix {
  const int32_t *group, *first;   // of a sequence (fg_page_share)
  PrefixGroup* info;              // [groups]
  int64_t* per;                   // tiles of a worker's share
  float* home;                    // [ntok][q_heads][D], rows in the share's order
  float2* home_stat;              // [ntok][q_heads]
  float* extra;                   // [workers][kPrefixRows][D], of the unit that a share goes on with
  float2* extra_stat;             // [workers][kPrefixRows]
};
constexpr int kPrefixRows = 128;  // most rows of a unit

// Where one row's parts lie.
struct PrefixParts {
  int64_t home;         // row of home
  int w0, count;        // extra parts are those of the shares w0 .. w0 + count - 1
  int row;              // in them
};
__device__ __forceinline__ PrefixParts prefix_parts(const Prefix& p, int seq, int t, int h, int gh, int group, int q_heads) {
  const PrefixGroup g = p.info[p.group[seq]];
  const int x = p.first[seq] + t, r = x * group + gh, u = r / g.rows;
  const int64_t start = g.base + (static_cast<int64_t>(h) * g.units + u) * g.tiles, per = *p.per;
  PrefixParts o;
  o.home = static_cast<int64_t>(g.first_row + x) * q_heads + h * group + gh;
  o.row = r - u * g.rows;
  const int w = static_cast<int>(start / per);
  o.w0 = w + 1;
  o.count = static_cast<int>((start + g.tiles - 1) / per) - w;
  return o;
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

// fp32 activations, every sequence: units of kF32Rows rows, tiles of 64 keys.
constexpr int kF32Rows = 16, kF32KeysLog2 = 6;
int f32_workers(int head_dim, int sms);
fg_status paged_attention_f32(const AttnArgs<float>& a, const ClassPlan& pl, int head_dim, bool own_plan, cudaStream_t st);

}  // namespace paged
}  // namespace fg
