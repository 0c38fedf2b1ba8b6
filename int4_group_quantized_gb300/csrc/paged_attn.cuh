// Internal interface of the paged attention kernels.
#pragma once

#include "paged_sched.cuh"

namespace fg {
namespace paged {

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
};

// own_plan: no plan was made (paged_sched.cuh, make_line).
// Sequences of at most kStepRows rows per K/V head (fp16).
int step_workers(int rows, int sms);
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
