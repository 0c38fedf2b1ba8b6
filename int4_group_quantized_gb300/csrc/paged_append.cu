// Concat into pages (FlexGen notes, "背景知识": x_K <- Concat(x_K, t w_K);
// "5. 近似方法": KV quantized in groups of 64 along the hidden dimension), for a
// ragged batch of chunks: each K/V row goes to its position's slot of its
// sequence's pages, and on request comes back as the cache restores it.
#include "codec_dev.cuh"
#include "paged.cuh"

namespace fg {
namespace paged {
namespace {

__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) {
  const uint4 raw = *reinterpret_cast<const uint4*>(p);
  const __half2* h = reinterpret_cast<const __half2*>(&raw);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  uint4 raw;
  __half2* h = reinterpret_cast<__half2*>(&raw);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = raw;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

template <typename T>
struct AppendArgs {
  Pool pool;
  Table tab;
  Batch batch;
  const T* src[2];
  T* restored[2];
  int64_t ld, ldr;
};

// A warp owns one (K or V, head) and a run of 16 batch rows, 8 lanes to a
// 64-group.
constexpr int kRun = 16;

template <typename T, int NG>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs<T> a) {
  constexpr int D = 64 * NG;
  constexpr int kTpi = 4 / NG;   // rows per warp-wide batch
  const int lane = threadIdx.x & 31;
  const int part = lane & 7, gi = (lane >> 3) % NG, tb = lane / (8 * NG);
  const int64_t runs = (a.batch.ntok + kRun - 1) / kRun;
  const int64_t items = 2 * runs * a.pool.heads;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  if (blockIdx.x == 0)   // what no row would notice: offsets that run backwards
    for (int i = threadIdx.x; i < a.tab.seqs; i += blockDim.x) seq_of(a.tab, a.batch, i);
  for (int64_t it = warp; it < items; it += nwarps) {
    const int64_t run = it % runs;
    const int h = static_cast<int>((it / runs) % a.pool.heads);
    const int which = static_cast<int>(it / (runs * a.pool.heads));
    // lane r < 16 finds the slot of row r of the run
    int64_t slot = -1;
    const int64_t row0 = run * kRun;
    if (lane < kRun && row0 + lane < a.batch.ntok) {
      const int r = static_cast<int>(row0 + lane);
      const int i = seq_of_row(a.batch.cu, a.tab.seqs, r);
      if (i < a.tab.seqs) {
        const Seq s = seq_of(a.tab, a.batch, i);
        if (r >= s.row0 && r < s.row0 + s.n) {
          const int pos = s.len - s.n + (r - s.row0);
          if (pos < 0) {
            atomicOr(a.batch.err, DEV_ERR_BATCH);
          } else {
            const int page = page_of(a.tab, i, pos);
            if (page < 0) atomicOr(a.batch.err, DEV_ERR_PAGE);
            else slot = slot_of(a.pool, page, h, pos);
          }
        }
      }
    }
    const T* src = (which ? a.src[1] : a.src[0]) + h * D + gi * 64 + part * 8;
    T* res = which ? a.restored[1] : a.restored[0];
    uint8_t* codes = which ? a.pool.codes[1] : a.pool.codes[0];
    float* mins = which ? a.pool.mins[1] : a.pool.mins[0];
    float* scales = which ? a.pool.scales[1] : a.pool.scales[0];
#pragma unroll
    for (int t0 = 0; t0 < kRun; t0 += kTpi) {
      const int t = t0 + tb;
      const int64_t sl = __shfl_sync(0xffffffffu, slot, t);
      float v[8];
      if (sl >= 0) {
        load8(src + (row0 + t) * a.ld, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
      }
      float mn, sc;
      const uint32_t packed = codec::quantize_group8(v, mn, sc);
      if (sl >= 0) {
        *reinterpret_cast<uint32_t*>(codes + sl * (D / 2) + gi * 32 + part * 4) = packed;
        if (part == 0) {
          mins[sl * NG + gi] = mn;
          scales[sl * NG + gi] = sc;
        }
        if (res != nullptr) {
          float r[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) r[e] = __fmaf_rn(codec::code_float((packed >> (4 * e)) & 15u), sc, mn);
          store8(res + (row0 + t) * a.ldr + h * D + gi * 64 + part * 8, r);
        }
      }
    }
  }
}

template <typename T>
fg_status launch_append(const fg_page_pool& pool, const fg_page_table& t, const int32_t* cu, const void* k,
                        const void* v, int64_t ld, int64_t ntok, void* kr, void* vr, int64_t ldr, unsigned int* err,
                        cudaStream_t st) {
  AppendArgs<T> a;
  a.pool = pool_of(pool);
  a.tab = table_of(t);
  a.batch = Batch{cu, static_cast<int>(ntok), err};
  a.src[0] = static_cast<const T*>(k);
  a.src[1] = static_cast<const T*>(v);
  a.restored[0] = static_cast<T*>(kr);
  a.restored[1] = static_cast<T*>(vr);
  a.ld = ld;
  a.ldr = ldr;
  const int64_t items = 2 * ((ntok + kRun - 1) / kRun) * pool.heads;
  const int64_t want = (items + 7) / 8, cap = static_cast<int64_t>(num_sms()) * 8;
  const unsigned grid = static_cast<unsigned>(want < cap ? want : cap);
  Trace tr(KC_KV_STORE, st);
  if (pool.head_dim == 128) append_kernel<T, 2><<<grid, 256, 0, st>>>(a);
  else append_kernel<T, 1><<<grid, 256, 0, st>>>(a);
  return check_launch("append_kernel");
}

}  // namespace
}  // namespace paged
}  // namespace fg

using namespace fg;
using namespace fg::paged;

extern "C" fg_status fg_paged_append(const fg_page_pool* pool, const fg_page_table* t, const int32_t* cu,
                                     const void* k, const void* v, int64_t ld, int64_t ntok, void* k_restored,
                                     void* v_restored, int64_t ldr, cudaStream_t stream) {
  FG_TRY(check_pool_table(pool, t));
  if (ntok < 0) return fail(FG_ERR_ARG, "negative row count");
  if (ntok > INT32_MAX - 256) return fail(FG_ERR_UNSUPPORTED, "more than 2^31 rows");
  if (ntok == 0 || t->seqs == 0) return FG_OK;
  if (!cu || !k || !v) return fail(FG_ERR_ARG, "null pointer");
  if ((k_restored == nullptr) != (v_restored == nullptr)) return fail(FG_ERR_ARG, "restored K and V: both or neither");
  const int64_t h1 = static_cast<int64_t>(pool->heads) * pool->head_dim;
  if (ld < h1 || (k_restored && ldr < h1)) return fail(FG_ERR_SHAPE, "row stride below heads * head_dim = %lld", (long long)h1);
  if (!aligned(cu, 4) || !aligned(k, 16) || !aligned(v, 16) || ld % 8 || !aligned(k_restored, 16) ||
      !aligned(v_restored, 16) || (k_restored && ldr % 8))
    return fail(FG_ERR_ALIGN, "rows need 16-byte alignment and strides that are multiples of 8");
  unsigned int* err = device_error_word();
  if (!err) return fail(FG_ERR_CUDA, "device error word");
  if (pool->dtype == FG_F16)
    return launch_append<__half>(*pool, *t, cu, k, v, ld, ntok, k_restored, v_restored, ldr, err, stream);
  return launch_append<float>(*pool, *t, cu, k, v, ld, ntok, k_restored, v_restored, ldr, err, stream);
}
