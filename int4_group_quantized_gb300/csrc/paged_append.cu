// Concat into pages (FlexGen notes, "背景知识": x_K <- Concat(x_K, t w_K);
// "5. 近似方法": KV quantized in groups of 64 along the hidden dimension), for a
// ragged batch of chunks: each K/V row goes to its position's slot of its
// sequence's pages, and on request comes back as the cache restores it.
#include "codec_dev.cuh"
#include "paged.cuh"
#include "q4_dev.cuh"
#include "tc_ptx.cuh"

namespace fg {
namespace paged {
namespace {

using q4::fma_f32x2;

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

// 16 bytes into shared memory, zeros where not `there` (then the address is not read).
__device__ __forceinline__ void cp16_zfill(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16u : 0u) : "memory");
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

// ---- one 64-group over 8 lanes, 8 values a lane --------------------------------
// Smallest and largest of the non-NaN values of a group, in the codec's order
// (-0 < +0; both NaN for a group of NaN), on all of its 8 lanes.
//
// fp16: the type's own minimum skips NaN and puts -0 below +0, and the largest
// is the negated minimum of the negated values, so both travel in one word.
struct Half8 {
  uint4 raw;
  __device__ __forceinline__ float get(int e) const {
    const uint32_t w = (e >> 1) == 0 ? raw.x : (e >> 1) == 1 ? raw.y : (e >> 1) == 2 ? raw.z : raw.w;
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return (e & 1) ? f.y : f.x;
  }
  __device__ __forceinline__ void bounds(float& mn, float& mx) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t lo = min2(min2(w[0], w[1]), min2(w[2], w[3]));
    uint32_t hi = min2(min2(w[0] ^ kSigns, w[1] ^ kSigns), min2(w[2] ^ kSigns, w[3] ^ kSigns));
    uint32_t both = min2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));   // (min, -max)
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) both = min2(both, __shfl_xor_sync(0xffffffffu, both, o));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&both));
    mn = f.x;
    mx = -f.y;
  }
  static constexpr uint32_t kSigns = 0x80008000u;
  static __device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};
// fp32: through the codec's order-preserving keys.
struct Float8 {
  float v[8];
  __device__ __forceinline__ void load(const float* p) { load8(p, v); }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
  }
  __device__ __forceinline__ float get(int e) const { return v[e]; }
  __device__ __forceinline__ void bounds(float& mn, float& mx) const {
    uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (!isnan(v[e])) {
        const uint32_t key = codec::order_key(v[e]);
        lo = min(lo, key);
        hi = max(hi, key);
      }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    codec::group_bounds(lo, hi, mn, mx);
  }
};
template <typename T>
struct Vec8 {
  using type = Float8;
};
template <>
struct Vec8<__half> {
  using type = Half8;
};

__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5};\n"
      "add.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul_f32x2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5};\n"
      "mul.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// The codes of 8 values as floats, by the codec's short form (code_fast in
// codec_dev.cuh: one product by c15 = 15 / r, rounded by adding 1.5 * 2^23), two
// at a time; q[e] holds values e and e + 4.  Returns whether they stand: every
// |u - rint(u)| stays 1e-5 below a rounding boundary.  What the short form is
// not made for gives a NaN there and does not stand either: a NaN value, a
// range of 0 or one too small for a finite c15 (u is infinite or NaN), an
// infinite value (c15 = 0).  No u exceeds 15 (1 + 2^-23), so no code does.
__device__ __forceinline__ bool codes_fast(const float2 (&v)[4], float mn, float c15, float2 (&q)[4]) {
  const float2 nmn = make_float2(-mn, -mn), c2 = make_float2(c15, c15), neg = make_float2(-1.0f, -1.0f);
  const float2 up = make_float2(codec::kRound, codec::kRound), down = make_float2(-codec::kRound, -codec::kRound);
  float far = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 u = mul_f32x2(add_f32x2(v[e], nmn), c2);
    q[e] = add_f32x2(add_f32x2(u, up), down);
    const float2 t = fma_f32x2(q[e], neg, u);
    far = max_nan(far, max_nan(fabsf(t.x), fabsf(t.y)));
  }
  return far <= 0.5f - 1e-5f;
}
// 8 codes (q[e] = codes e, e + 4) as a word, low nibble first: sums of multiples
// of 16^e below 2^16, exact in fp32.
__device__ __forceinline__ uint32_t pack_codes(const float2 (&q)[4]) {
  const float2 k16 = make_float2(16.0f, 16.0f);
  float2 s = q[3];
#pragma unroll
  for (int e = 2; e >= 0; --e) s = fma_f32x2(s, k16, q[e]);
  s = add_f32x2(s, make_float2(8388608.0f, 8388608.0f));   // 2^23: the sum in the low mantissa bits
  return __byte_perm(__float_as_uint(s.x), __float_as_uint(s.y), 0x5410);
}

// The literal codes of 8 values, packed: out of the way of the common path.
template <class X>
__device__ __noinline__ uint32_t exact_word(X x, float mn, float r) {
  uint32_t word = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) word |= static_cast<uint32_t>(codec::code_exact(x.get(e), mn, r)) << (4 * e);
  return word;
}

// A warp takes a run of rows (8 batches of 4 groups: 16 rows of two groups a
// head, 32 rows of one) and some of the 2 * heads (K or V, head) slices.  The
// run's slots are found once; after the batches' minima and maxima every lane
// holds one of the 32 groups and takes its two divisions (the literal form
// spent two per lane and batch); then the batches are coded with their group's
// numbers from that lane.  The bytes are the floor (fp16: 2 read, 0.625 written
// and 2 more where the restored rows are wanted); half the instructions that
// could issue do.  fp16 rows therefore come by asynchronous copies a slice
// ahead, 4 KB a warp and slice: 19 thousand rows of 32 heads of 128 with
// restored rows 162.7 us (4.5 TB/s) where loads into registers took 178; two
// slices ahead 161.6, three blocks an SM (80 registers, spills) 196.
template <int NG>
constexpr int kRun = 32 / NG;
constexpr int kBatches = 8;

constexpr int kAppendWarps = 8;
template <typename T>
constexpr bool kRing = sizeof(T) == 2;
template <typename T>
constexpr int kRingBytes = kRing<T> ? kAppendWarps * 2 * kBatches * 32 * 16 : 0;

template <typename T, int NG>
__global__ void __launch_bounds__(32 * kAppendWarps, 2) append_kernel(const AppendArgs<T> a, int slices) {
  constexpr int D = 64 * NG;
  constexpr uint32_t kNone = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int part = lane & 7, gi = (lane >> 3) % NG, rb = (lane >> 3) / NG;   // row of a batch
  const int heads = a.pool.heads, psl = a.pool.ps_log2;
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
            else token = (static_cast<uint32_t>(page) << psl) + (pos & ((1 << psl) - 1));
          }
        }
      }
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
      const int col = h * D + gi * 64 + part * 8;
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
      // lane 8 g + b keeps group g of batch b
      float mn = 0.0f, mx = 0.0f;
#pragma unroll
      for (int b = 0; b < kBatches; ++b) {
        float lo, hi;
        batch(b).bounds(lo, hi);
        if (part == b) {
          mn = lo;
          mx = hi;
        }
      }
      if (isnan(mn)) mn = mx = __uint_as_float(0x7fffffffu);   // the codec's NaN
      const float r = __fsub_rn(mx, mn), c15 = __fdiv_rn(15.0f, r), scale = __fdiv_rn(r, 15.0f);
      uint8_t* codes = value ? a.pool.codes[1] : a.pool.codes[0];
      // row of the pool's arrays that a token's slice of head h is
      auto slot = [&](uint32_t k) { return ((static_cast<int64_t>(k >> psl) * heads + h) << psl) + (k & ((1u << psl) - 1)); };
      if (mine != kNone) {
        const int64_t at = slot(mine) * NG + gi;
        (value ? a.pool.mins[1] : a.pool.mins[0])[at] = mn;
        (value ? a.pool.scales[1] : a.pool.scales[0])[at] = scale;
      }
      T* res = value ? a.restored[1] : a.restored[0];
#pragma unroll
      for (int b = 0; b < kBatches; ++b) {
        const int from = (lane & 24) + b, t = b * (4 / NG) + rb;
        const float bmn = __shfl_sync(0xffffffffu, mn, from), bc = __shfl_sync(0xffffffffu, c15, from);
        const X x = batch(b);
        float2 v[4], q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = make_float2(x.get(e), x.get(e + 4));
        const bool stands = codes_fast(v, bmn, bc, q);
        if (__any_sync(0xffffffffu, !stands)) {   // rare
          const float br = __shfl_sync(0xffffffffu, r, from);
          const uint32_t word = exact_word(x, bmn, br);
          if (!stands)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              q[e] = make_float2(codec::code_float((word >> (4 * e)) & 15u), codec::code_float((word >> (4 * e + 16)) & 15u));
        }
        if (tok[b] != kNone) *reinterpret_cast<uint32_t*>(codes + slot(tok[b]) * (D / 2) + gi * 32 + part * 4) = pack_codes(q);
        if (res != nullptr) {
          const float bs = __shfl_sync(0xffffffffu, scale, from);
          const float2 s2 = make_float2(bs, bs), m2 = make_float2(bmn, bmn);
          float o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y = fma_f32x2(q[e], s2, m2);
            o[e] = y.x;
            o[e + 4] = y.y;
          }
          if (tok[b] != kNone) store8(res + (row0 + t) * a.ldr + col, o);
        }
      }
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
