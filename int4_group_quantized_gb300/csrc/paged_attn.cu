// Attention of a ragged batch of chunks over the paged 4-bit cache (FlexGen
// notes, "背景知识": Softmax(x_Q x_K^T / sqrt(h1)) x_V per head, causal; "5.
// 近似方法": K and V stored in 4-bit groups of 64).
//
// A first form: one warp per (row, query head), its lanes along the head
// dimension, one key at a time with a running maximum and sum.
#include <math.h>

#include "paged.cuh"

namespace fg {
namespace paged {
namespace {

template <typename T>
struct AttnArgs {
  Pool pool;
  Table tab;
  Batch batch;
  const T* q;
  T* out;
  int64_t ldq, ldo;
  int q_heads, group;   // query heads, and query heads per K/V head
  int max_q;
  int64_t window, sinks;
  float scale;
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }

template <typename T, int D>
__global__ void __launch_bounds__(128) attn_rows_kernel(const AttnArgs<T> a) {
  constexpr int E = D / 32;   // dims of a lane
  constexpr int NG = D / 64;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (blockIdx.x == 0)   // what no row would notice: offsets that run backwards
    for (int i = threadIdx.x; i < a.tab.seqs; i += blockDim.x) seq_of(a.tab, a.batch, i);
  const int64_t r64 = w / a.q_heads;
  if (r64 >= a.batch.ntok) return;
  const int r = static_cast<int>(r64), qh = static_cast<int>(w % a.q_heads), h = qh / a.group;
  const int i = seq_of_row(a.batch.cu, a.tab.seqs, r);
  if (i >= a.tab.seqs) return;
  const Seq s = seq_of(a.tab, a.batch, i);
  if (r < s.row0 || r >= s.row0 + s.n) return;
  if (s.n > a.max_q) {
    atomicOr(a.batch.err, DEV_ERR_BATCH);
    return;
  }
  const int64_t pos = static_cast<int64_t>(s.len) - s.n + (r - s.row0);
  const int64_t lo = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = to_f(a.q[r * a.ldq + qh * D + lane * E + e]) * a.scale;
    o[e] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  const int g = lane * E / 64;
  for (int64_t j = 0; j <= pos && j < s.keys; ++j) {
    if (j < lo && j >= a.sinks) {
      j = lo - 1;
      continue;
    }
    const int page = page_of(a.tab, i, static_cast<int>(j));
    if (page < 0) {
      if (lane == 0) atomicOr(a.batch.err, DEV_ERR_PAGE);
      continue;
    }
    const int64_t sl = slot_of(a.pool, page, h, static_cast<int>(j));
    auto value = [&](int which, int e) {
      const int c = lane * E + e;
      const int byte = a.pool.codes[which][sl * (D / 2) + c / 2];
      return fmaf(static_cast<float>((byte >> (4 * (c & 1))) & 15), a.pool.scales[which][sl * NG + g],
                  a.pool.mins[which][sl * NG + g]);
    };
    float x = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) x += q[e] * value(0, e);
#pragma unroll
    for (int f = 16; f > 0; f >>= 1) x += __shfl_xor_sync(0xffffffffu, x, f);
    const float nm = fmaxf(m, x);
    const float base = nm == -INFINITY ? 0.0f : nm;
    const float alpha = expf(m - base), p = expf(x - base);
    l = l * alpha + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * alpha + p * value(1, e);
    m = nm;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) put(a.out + r * a.ldo + qh * D + lane * E + e, l != 0.0f ? o[e] / l : 0.0f);
}

template <typename T>
fg_status launch_attn(const fg_page_pool& pool, const fg_page_table& t, const int32_t* cu, const void* q, int64_t ldq,
                      int32_t q_heads, int64_t ntok, int64_t max_q, int64_t window, int64_t sinks, void* out,
                      int64_t ldo, unsigned int* err, cudaStream_t st) {
  AttnArgs<T> a;
  a.pool = pool_of(pool);
  a.tab = table_of(t);
  a.batch = Batch{cu, static_cast<int>(ntok), err};
  a.q = static_cast<const T*>(q);
  a.out = static_cast<T*>(out);
  a.ldq = ldq;
  a.ldo = ldo;
  a.q_heads = q_heads;
  a.group = q_heads / pool.heads;
  a.max_q = static_cast<int>(max_q);
  a.window = window;
  a.sinks = sinks;
  a.scale = static_cast<float>(1.0 / sqrt(static_cast<double>(pool.head_dim)));
  const int64_t warps = ntok * q_heads;
  const unsigned grid = static_cast<unsigned>((warps + 3) / 4);
  Trace tr(KC_ATTN_PAGED, st);
  if (pool.head_dim == 128) attn_rows_kernel<T, 128><<<grid, 128, 0, st>>>(a);
  else attn_rows_kernel<T, 64><<<grid, 128, 0, st>>>(a);
  return check_launch("attn_rows_kernel");
}

fg_status check_attn(const fg_page_pool* pool, const fg_page_table* t, int32_t q_heads, int64_t ntok, int64_t max_q) {
  FG_TRY(check_pool_table(pool, t));
  if (q_heads <= 0 || ntok < 0 || max_q < 0) return fail(FG_ERR_ARG, "attention sizes");
  if (q_heads % pool->heads)
    return fail(FG_ERR_SHAPE, "q_heads %d is no multiple of the pool's %d heads", q_heads, pool->heads);
  if (ntok * q_heads > INT32_MAX - 1024) return fail(FG_ERR_UNSUPPORTED, "more than 2^31 (row, head) pairs");
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
  return 256;
}

fg_status fg_paged_attention(const fg_page_pool* pool, const fg_page_table* t, const int32_t* cu, const void* q,
                             int64_t ldq, int32_t q_heads, int64_t ntok, int64_t max_q, int64_t window, int64_t sinks,
                             void* out, int64_t ldo, void* ws, size_t ws_bytes, cudaStream_t stream) {
  FG_TRY(check_attn(pool, t, q_heads, ntok, max_q));
  if (window < 0 || sinks < 0) return fail(FG_ERR_ARG, "negative window or sinks");
  if (ntok == 0 || max_q == 0 || t->seqs == 0) return FG_OK;
  if (!cu || !q || !out) return fail(FG_ERR_ARG, "null pointer");
  const int64_t h1 = static_cast<int64_t>(q_heads) * pool->head_dim;
  if (ldq < h1 || ldo < h1) return fail(FG_ERR_SHAPE, "row stride below q_heads * head_dim = %lld", (long long)h1);
  if (!aligned(cu, 4) || !aligned(q, 16) || !aligned(out, 16) || ldq % 8 || ldo % 8)
    return fail(FG_ERR_ALIGN, "q and out need 16-byte alignment and strides that are multiples of 8");
  const size_t need = fg_paged_attention_workspace_bytes(pool, t, q_heads, ntok, max_q);
  if (!ws || ws_bytes < need) return fail(FG_ERR_WORKSPACE, "paged attention needs %zu workspace bytes", need);
  if (!aligned(ws, 256)) return fail(FG_ERR_ALIGN, "workspace needs 256-byte alignment");
  unsigned int* err = device_error_word();
  if (!err) return fail(FG_ERR_CUDA, "device error word");
  if (pool->dtype == FG_F16)
    return launch_attn<__half>(*pool, *t, cu, q, ldq, q_heads, ntok, max_q, window, sinks, out, ldo, err, stream);
  return launch_attn<float>(*pool, *t, cu, q, ldq, q_heads, ntok, max_q, window, sinks, out, ldo, err, stream);
}

}  // extern "C"
