// Reading cached rows back: K and V of a ragged batch of positions, as their
// codes stand for them (FlexGen notes, "5. 近似方法": stored quantized, converted
// back to FP16).
//
// Bound by the bytes (fp16: 0.625 read and 2 written an element).  A warp takes a
// run of 32 rows, whose places the lanes find together, and one or two of the
// 2 * heads (K or V, head) slices; a lane restores one word of eight codes at a
// time, kAhead of them loaded at once, and stores 16 (fp32: 32) bytes.  64
// sequences of 300 to 900 rows, 32 heads of 128: 102 us for 619 MB, 89% of a
// copy's rate (32 warps an SM in blocks of 4; in blocks of 8 103; 24 warps 107;
// four slices a warp 107, eight 115; half the words at once, 40 warps, 128); fp32 208
// us for 1,090 MB, 77%.
#include "paged_codec.cuh"

namespace fg {
namespace paged {
namespace {

constexpr int kWarps = 4;

template <typename T>
struct ReadArgs {
  Pool pool;
  Table tab;
  Batch batch;
  const int32_t* start;
  T* out[2];
  int64_t ld;
  int slices;
};

template <typename T, int NG>
__global__ void __launch_bounds__(32 * kWarps, 8) read_kernel(const ReadArgs<T> a) {
  constexpr int D = 64 * NG, kLanes = 8 * NG, kAtOnce = 32 / kLanes;   // lanes of a row, rows of a step
  constexpr int kAhead = 8;
  const int lane = threadIdx.x & 31, at = lane % kLanes, rb = lane / kLanes;
  const int heads = a.pool.heads, psl = a.pool.ps_log2;
  tc::griddep_launch();
  tc::griddep_wait();
  const int64_t runs = (a.batch.ntok + 31) / 32;
  const int chunks = (2 * heads + a.slices - 1) / a.slices;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  if (blockIdx.x == 0)   // what no row would notice: offsets that run backwards
    for (int i = threadIdx.x; i < a.tab.seqs; i += blockDim.x) seq_of(a.tab, a.batch, i);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < runs * chunks; it += nwarps) {
    const int64_t row0 = it / chunks * 32;
    const int s0 = static_cast<int>(it % chunks) * a.slices, s1 = min(2 * heads, s0 + a.slices);
    uint32_t token = kNoToken;
    if (row0 + lane < a.batch.ntok) {
      const int r = static_cast<int>(row0 + lane);
      if (a.start == nullptr) {
        int pos;
        token = token_of_row(a.tab, a.batch, r, pos);
      } else {
        const int i = seq_of_row(a.batch.cu, a.tab.seqs, r);
        if (i < a.tab.seqs) {
          const Seq s = seq_of(a.tab, a.batch, i);
          if (r >= s.row0 && r < s.row0 + s.n) {
            const int64_t pos = static_cast<int64_t>(a.start[i]) + (r - s.row0);
            const int page = pos >= 0 && pos < s.len ? page_of(a.tab, i, static_cast<int>(pos)) : -1;
            if (pos < 0 || pos >= s.len) atomicOr(a.batch.err, DEV_ERR_BATCH);
            else if (page < 0) atomicOr(a.batch.err, DEV_ERR_PAGE);
            else token = (static_cast<uint32_t>(page) << psl) + (static_cast<uint32_t>(pos) & ((1u << psl) - 1));
          }
        }
      }
    }
    for (int sl = s0; sl < s1; ++sl) {
      const bool value = sl >= heads;
      const int h = value ? sl - heads : sl;
      T* out = value ? a.out[1] : a.out[0];
      if (out == nullptr) continue;
      const uint8_t* codes = value ? a.pool.codes[1] : a.pool.codes[0];
      const float* mins = value ? a.pool.mins[1] : a.pool.mins[0];
      const float* scales = value ? a.pool.scales[1] : a.pool.scales[0];
      for (int r0 = 0; r0 < 32; r0 += kAhead * kAtOnce) {
        uint32_t word[kAhead], tok[kAhead];
        float mn[kAhead], sc[kAhead];
#pragma unroll
        for (int b = 0; b < kAhead; ++b) {
          tok[b] = __shfl_sync(0xffffffffu, token, r0 + b * kAtOnce + rb);
          const uint32_t k = tok[b] == kNoToken ? 0u : tok[b];
          const int64_t slot = ((static_cast<int64_t>(k >> psl) * heads + h) << psl) + (k & ((1u << psl) - 1));
          word[b] = *reinterpret_cast<const uint32_t*>(codes + slot * (D / 2) + 4 * at);
          mn[b] = mins[slot * NG + at / 8];
          sc[b] = scales[slot * NG + at / 8];
        }
#pragma unroll
        for (int b = 0; b < kAhead; ++b) {
          const float2 s2 = make_float2(sc[b], sc[b]), m2 = make_float2(mn[b], mn[b]);
          const uint32_t x = word[b], y = x >> 8;
          float2 q[4] = {q4::nib_pair_f32(q4::lop_mask_or(x, 0x000F000Fu, q4::kMagic)), q4::nib16_pair_f32(q4::lop_mask_or(x, 0x00F000F0u, q4::kMagic)),
                         q4::nib_pair_f32(q4::lop_mask_or(y, 0x000F000Fu, q4::kMagic)), q4::nib16_pair_f32(q4::lop_mask_or(y, 0x00F000F0u, q4::kMagic))};
          float o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = fma_f32x2(q[e], s2, m2);
            o[e] = v.x;
            o[e + 4] = v.y;
          }
          if (tok[b] != kNoToken) store8(out + (row0 + r0 + b * kAtOnce + rb) * a.ld + static_cast<int64_t>(h) * D + 8 * at, o);
        }
      }
    }
  }
}

template <typename T>
fg_status run_read(const fg_page_pool& pool, const fg_page_table& t, const int32_t* cu, const int32_t* start, void* k, void* v, int64_t ld,
                   int64_t ntok, unsigned int* err, cudaStream_t st) {
  ReadArgs<T> a;
  a.pool = pool_of(pool);
  a.tab = table_of(t);
  a.batch = Batch{cu, static_cast<int>(ntok), err};
  a.start = start;
  a.out[0] = static_cast<T*>(k);
  a.out[1] = static_cast<T*>(v);
  a.ld = ld;
  const int64_t runs = (ntok + 31) / 32, sms = num_sms(), warps = sms * 48;
  const int64_t fit = runs * 2 * pool.heads / warps;
  a.slices = static_cast<int>(fit < 1 ? 1 : fit > 2 ? 2 : fit);
  const int64_t items = runs * ((2 * pool.heads + a.slices - 1) / a.slices), want = (items + kWarps - 1) / kWarps, cap = sms * 64;
  Trace tr(KC_PAGED_READ, st);
  return paged::launch("read_kernel", true, pool.head_dim == 128 ? read_kernel<T, 2> : read_kernel<T, 1>,
                       static_cast<unsigned>(want < cap ? want : cap), 32 * kWarps, 0, st, a);
}

}  // namespace
}  // namespace paged
}  // namespace fg

using namespace fg;
using namespace fg::paged;

extern "C" fg_status fg_paged_read(const fg_page_pool* pool, const fg_page_table* t, const int32_t* cu, const int32_t* start, void* k,
                                   void* v, int64_t ld, int64_t ntok, cudaStream_t stream) {
  FG_TRY(check_pool_table(pool, t));
  if (ntok < 0) return fail(FG_ERR_ARG, "negative row count");
  if (pool->pages * pool->page_size >= UINT32_MAX) return fail(FG_ERR_UNSUPPORTED, "a pool of 2^32 tokens or more");
  if (ntok > INT32_MAX - 256) return fail(FG_ERR_UNSUPPORTED, "more than 2^31 rows");
  if (ntok == 0 || t->seqs == 0 || (!k && !v)) return FG_OK;
  if (!cu) return fail(FG_ERR_ARG, "null pointer");
  const int64_t h1 = static_cast<int64_t>(pool->heads) * pool->head_dim;
  if (ld < h1) return fail(FG_ERR_SHAPE, "row stride below heads * head_dim = %lld", (long long)h1);
  if (!aligned(cu, 4) || !aligned(start, 4) || !aligned(k, 16) || !aligned(v, 16) || ld % 8)
    return fail(FG_ERR_ALIGN, "rows need 16-byte alignment and strides that are multiples of 8");
  unsigned int* err = device_error_word();
  if (!err) return fail(FG_ERR_CUDA, "device error word");
  if (pool->dtype == FG_F16) return run_read<__half>(*pool, *t, cu, start, k, v, ld, ntok, err, stream);
  return run_read<float>(*pool, *t, cu, start, k, v, ld, ntok, err, stream);
}
