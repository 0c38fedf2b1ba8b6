// Concat into pages (FlexGen notes, "背景知识": x_K <- Concat(x_K, t w_K);
// "5. 近似方法": KV quantized in groups of 64 along the hidden dimension), for a
// ragged batch of chunks: each K/V row goes to its position's slot of its
// sequence's pages, and on request comes back as the cache restores it.
#include "paged_codec.cuh"

namespace fg {
namespace paged {
namespace {

template <typename T>
struct AppendArgs {
  Pool pool;
  Table tab;
  Batch batch;
  const T* src[2];
  T* restored[2];
  int64_t ld, ldr;
};

// A warp takes a run of rows (8 batches of 4 groups: 16 rows of two groups a
// head, 32 rows of one) and some of the 2 * heads (K or V, head) slices.  The
// run's slots are found once.  The bytes are the floor (fp16: 2 read, 0.625
// written and 2 more where the restored rows are wanted); half the instructions
// that could issue do.  fp16 rows therefore come by asynchronous copies a slice
// ahead, 4 KB a warp and slice: 19 thousand rows of 32 heads of 128 with
// restored rows 162.7 us (4.5 TB/s) where loads into registers took 178; two
// slices ahead 161.6, three blocks an SM (80 registers, spills) 196.
constexpr int kAppendWarps = 8;
template <typename T>
constexpr bool kRing = sizeof(T) == 2;
template <typename T>
constexpr int kRingBytes = kRing<T> ? kAppendWarps * 2 * kBatches * 32 * 16 : 0;

template <typename T, int NG>
__global__ void __launch_bounds__(32 * kAppendWarps, 2) append_kernel(const AppendArgs<T> a, int slices) {
  constexpr int D = 64 * NG;
  constexpr uint32_t kNone = kNoToken;
  const int lane = threadIdx.x & 31;
  const int part = lane & 7, gi = (lane >> 3) % NG, rb = (lane >> 3) / NG;   // row of a batch
  const int heads = a.pool.heads;
  extern __shared__ __align__(16) uint8_t ring_mem[];
  tc::griddep_wait();
  uint4* const ring = reinterpret_cast<uint4*>(ring_mem) + (threadIdx.x >> 5) * (2 * kBatches * 32) + lane;
  using X = typename Vec8<T>::type;
  const int64_t runs = (a.batch.ntok + kRun<NG> - 1) / kRun<NG>;
  const int chunks = (2 * heads + slices - 1) / slices;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  if (blockIdx.x == 0)   // what no row would notice: offsets that run backwards
    for (int i = threadIdx.x; i < a.tab.seqs; i += blockDim.x) seq_of(a.tab, a.batch, i);
  for (int64_t it = warp; it < runs * chunks; it += nwarps) {
    const int64_t row0 = it / chunks * kRun<NG>;
    const int s0 = static_cast<int>(it % chunks) * slices, s1 = min(2 * heads, s0 + slices);
    // lane r finds the token of the pool that row r of the run goes to
    uint32_t token = kNone;
    if (lane < kRun<NG> && row0 + lane < a.batch.ntok) {
      int pos;
      token = token_of_row(a.tab, a.batch, static_cast<int>(row0 + lane), pos);
    }
    uint32_t tok[kBatches];   // of this lane's row in each batch
#pragma unroll
    for (int b = 0; b < kBatches; ++b) tok[b] = __shfl_sync(0xffffffffu, token, b * (4 / NG) + rb);
    const uint32_t mine = __shfl_sync(0xffffffffu, token, part * (4 / NG) + rb);
    auto source = [&](int sl) {   // the lane's values of the run's first row
      return (sl >= heads ? a.src[1] : a.src[0]) + row0 * a.ld + (sl >= heads ? sl - heads : sl) * D + gi * 64 + part * 8;
    };
    auto fetch = [&](int sl) {
      if (sl < s1) {
        const T* src = source(sl);
#pragma unroll
        for (int b = 0; b < kBatches; ++b)
          cp16_zfill(tc::smem_u32(ring + ((sl & 1) * kBatches + b) * 32), tok[b] != kNone ? src + (b * (4 / NG) + rb) * a.ld : src, tok[b] != kNone);
      }
      tc::cp_async_commit();
    };
    if constexpr (kRing<T>) fetch(s0);
    for (int sl = s0; sl < s1; ++sl) {
      const bool value = sl >= heads;
      const int h = value ? sl - heads : sl;
      X held[kRing<T> ? 1 : kBatches];
      if constexpr (kRing<T>) {
        fetch(sl + 1);
        tc::cp_async_wait<1>();   // a lane reads what it copied itself
      } else {
        const T* src = source(sl);
#pragma unroll
        for (int b = 0; b < kBatches; ++b) {
          if (tok[b] != kNone) held[b].load(src + (b * (4 / NG) + rb) * a.ld);
          else held[b].clear();
        }
      }
      auto batch = [&](int b) {
        if constexpr (kRing<T>) return X{ring[((sl & 1) * kBatches + b) * 32]};
        else return held[b];
      };
      store_slice<T, NG>(a.pool, value, h, tok, mine, row0, value ? a.restored[1] : a.restored[0], a.ldr, batch);
    }
  }
}

template <typename T, int NG>
fg_status launch_run(const AppendArgs<T>& a, int slices, unsigned grid, cudaStream_t st) {
  static bool set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (kRingBytes<T> > 48 * 1024 && dev >= 0 && dev < 64 && !set[dev]) {
    if (cudaFuncSetAttribute(append_kernel<T, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes<T>) != cudaSuccess)
      return check_launch("append_kernel smem attribute");
    set[dev] = true;
  }
  return paged::launch("append_kernel", true, append_kernel<T, NG>, grid, 32 * kAppendWarps, kRingBytes<T>, st, a, slices);
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
  // as many slices a warp as leave every SM its 16 warps, so that a run's slots are looked up no oftener than need be; at
  // most 8 (4 to 8: 162 us for the rows above; 10, whose last warps run alone: 177; 16: 208)
  const int run = pool.head_dim == 128 ? kRun<2> : kRun<1>;
  const int64_t runs = (ntok + run - 1) / run, warps = static_cast<int64_t>(num_sms()) * 16;
  const int64_t fit = runs * 2 * pool.heads / warps;
  const int slices = static_cast<int>(fit < 1 ? 1 : fit > 8 ? 8 : fit);
  const int64_t items = runs * ((2 * pool.heads + slices - 1) / slices);
  const int64_t want = (items + 7) / 8, cap = static_cast<int64_t>(num_sms()) * 16;
  const unsigned grid = static_cast<unsigned>(want < cap ? want : cap);
  Trace tr(KC_KV_STORE, st);
  if (pool.head_dim == 128) return launch_run<T, 2>(a, slices, grid, st);
  return launch_run<T, 1>(a, slices, grid, st);
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
  if (pool->pages * pool->page_size >= UINT32_MAX) return fail(FG_ERR_UNSUPPORTED, "a pool of 2^32 tokens or more");
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
