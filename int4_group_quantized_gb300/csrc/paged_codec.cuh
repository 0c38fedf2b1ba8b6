// The group quantizer of the paged appends: 64-groups over 8 lanes, and a slice
// (one head's K or V of a run of rows) into the pages.
#pragma once

#include "codec_dev.cuh"
#include "paged.cuh"
#include "q4_dev.cuh"
#include "tc_ptx.cuh"

namespace fg {
namespace paged {

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

template <int NG>
constexpr int kRun = 32 / NG;   // rows of a run
constexpr int kBatches = 8;     // of 4 groups
constexpr uint32_t kNoToken = 0xffffffffu;

// The token of the pool that row r of the batch goes to (kNoToken: none) and its
// position (-1: the row belongs to no sequence, or stands before its first token).
__device__ __forceinline__ uint32_t token_of_row(const Table& t, const Batch& batch, int r, int& pos) {
  pos = -1;
  const int i = seq_of_row(batch.cu, t.seqs, r);
  if (i >= t.seqs) return kNoToken;
  const Seq s = seq_of(t, batch, i);
  if (r < s.row0 || r >= s.row0 + s.n) return kNoToken;
  pos = s.len - s.n + (r - s.row0);
  if (pos < 0) {
    atomicOr(batch.err, DEV_ERR_BATCH);
    pos = -1;
    return kNoToken;
  }
  const int page = page_of(t, i, pos);
  if (page < 0) {
    atomicOr(batch.err, DEV_ERR_PAGE);
    return kNoToken;
  }
  return (static_cast<uint32_t>(page) << t.ps_log2) + (pos & ((1 << t.ps_log2) - 1));
}

// K (value: V) of head h of a run's rows: a lane holds 8 values (group gi, part
// `part`) of row b * (4 / NG) + rb in batch(b); tok[b] is that row's token, `mine`
// the token of the row whose group the lane keeps.  After the batches' minima and
// maxima every lane holds one of the 32 groups and takes its two divisions (the
// literal form spent two per lane and batch); then the batches are coded with
// their group's numbers from that lane.  res: where the restored rows go, or null.
template <typename T, int NG, class F>
__device__ __forceinline__ void store_slice(const Pool& pool, bool value, int h, const uint32_t (&tok)[kBatches], uint32_t mine, int64_t row0,
                                            T* res, int64_t ldr, F batch) {
  using X = typename Vec8<T>::type;
  constexpr int D = 64 * NG;
  constexpr uint32_t kNone = kNoToken;
  const int lane = threadIdx.x & 31;
  const int part = lane & 7, gi = (lane >> 3) % NG, rb = (lane >> 3) / NG;
  const int heads = pool.heads, psl = pool.ps_log2;
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
  uint8_t* codes = value ? pool.codes[1] : pool.codes[0];
  // row of the pool's arrays that a token's slice of head h is
  auto slot = [&](uint32_t k) { return ((static_cast<int64_t>(k >> psl) * heads + h) << psl) + (k & ((1u << psl) - 1)); };
  if (mine != kNone) {
    const int64_t at = slot(mine) * NG + gi;
    (value ? pool.mins[1] : pool.mins[0])[at] = mn;
    (value ? pool.scales[1] : pool.scales[0])[at] = scale;
  }
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
      if (tok[b] != kNone) store8(res + (row0 + t) * ldr + h * D + gi * 64 + part * 8, o);
    }
  }
}

}  // namespace paged
}  // namespace fg
