// Concat into pages with rotary positions: queries and keys of a ragged batch
// are rotated to their positions, keys and values quantized into their slots
// (FlexGen notes, "背景知识": x_K <- Concat(x_K, t w_K); "5. 近似方法": KV in
// groups of 64 along the hidden dimension), in one pass over the rows.
//
// A block takes a run of rows (16 of head_dim 128, 32 of 64) and some of the
// 2 * heads + q_heads slices (K, V, then Q; a head's columns of the run each),
// dealt round its eight warps.  The run's cosines and sines are worked out once,
// by all threads, into shared memory; a lane holds eight neighbouring dims of a
// row, and the dims that they turn with lie in a lane beside it (halves) or in
// the same one (pairs).  Rotated keys are rounded to the activations' type, as a
// rotation of its own would leave them, and take the append's quantizer from
// registers.
//
// Bound by the bytes on paper (48 prompts of 300 to 700 rows, 32 query heads on 8,
// d 128: 533 MB, 78 us); takes 141: the append's quantizer and two blocks of 128
// registers an SM, 15 warps of which every second instruction waits for the one
// before or for its load.  Eight slices a warp for many rows (four 155, two 168: a
// run's angles are worked out again for each); blocks that stay, two an SM, 149;
// three blocks an SM 190; four of four warps 155; half the queries' loads at once 149;
// the next head's loads under the one before 169 (spills), pieces found without divisions 140.
// The same as two calls, fg_rotate of the queries and this without them: 156 (69 and 85).
// fp32: 225 us for 1,039 MB, 68% of a copy's rate.
#include <initializer_list>

#include "paged_codec.cuh"
#include "rotary.cuh"

namespace fg {
namespace paged {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
template <typename T>
constexpr bool kRing = sizeof(T) == 2;
template <typename T>
constexpr int kRingBytes = kRing<T> ? kWarps * 2 * kBatches * 32 * 16 : 0;

template <typename T>
struct RotatedArgs {
  Pool pool;
  Table tab;
  Batch batch;
  const uint64_t* turns;
  const T* src[3];      // K, V, Q
  T* restored[2];
  T* q_out;
  int64_t ld[3], ldr, ldqo;
  int q_heads, rot;
  float scale;
  int slices;           // of a warp
};

// Cosine (kind 0) or sine (1) of pair p in a row's 2 P floats: a lane reads its
// chunk's 4 (pairs) or twice 4 (halves) side by side with its neighbours.
template <bool HALF>
__device__ __forceinline__ int cs_at(int kind, int p, int P) {
  return HALF ? kind * P + ((p >> 2) & 1) * (P / 2) + (p >> 3) * 4 + (p & 3) : kind * P + p;
}

__device__ __forceinline__ void unpack(const Half8& x, float2 (&v)[4]) {
  const uint32_t w[4] = {x.raw.x, x.raw.y, x.raw.z, x.raw.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
}
__device__ __forceinline__ void unpack(const Float8& x, float2 (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = make_float2(x.v[2 * e], x.v[2 * e + 1]);
}
__device__ __forceinline__ void pack(Half8& x, const float2 (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 h = __float22half2_rn(v[e]);
    w[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  x.raw = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(Float8& x, const float2 (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x.v[2 * e] = v[e].x;
    x.v[2 * e + 1] = v[e].y;
  }
}
__device__ __forceinline__ Half8 from_lane(const Half8& x, int lane) {
  Half8 y;
  y.raw = make_uint4(__shfl_sync(0xffffffffu, x.raw.x, lane), __shfl_sync(0xffffffffu, x.raw.y, lane),
                     __shfl_sync(0xffffffffu, x.raw.z, lane), __shfl_sync(0xffffffffu, x.raw.w, lane));
  return y;
}
__device__ __forceinline__ Float8 from_lane(const Float8& x, int lane) {
  Float8 y;
#pragma unroll
  for (int e = 0; e < 8; ++e) y.v[e] = __shfl_sync(0xffffffffu, x.v[e], lane);
  return y;
}
__device__ __forceinline__ void put8(__half* p, const Half8& x) { *reinterpret_cast<uint4*>(p) = x.raw; }
__device__ __forceinline__ void put8(float* p, const Float8& x) { store8(p, x.v); }
__device__ __forceinline__ void get8(const __half* p, Half8& x) { x.raw = *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void get8(const float* p, Float8& x) { x.load(p); }

// Cosines and sines of eight pairs from p on (HALF), or of four (PAIRS).
template <bool HALF>
__device__ __forceinline__ void read_cs(const float* cs, int p, int P, float4 (&c)[2], float4 (&s)[2]) {
#pragma unroll
  for (int e = 0; e < (HALF ? 2 : 1); ++e) {
    c[e] = *reinterpret_cast<const float4*>(cs + cs_at<HALF>(0, p + 4 * e, P));
    s[e] = *reinterpret_cast<const float4*>(cs + cs_at<HALF>(1, p + 4 * e, P));
  }
}
__device__ __forceinline__ void turn_half(float2 (&u)[4], float2 (&v)[4], const float4 (&c)[2], const float4 (&s)[2]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    rotary::turn2(u[2 * e], v[2 * e], make_float2(c[e].x, c[e].y), make_float2(s[e].x, s[e].y));
    rotary::turn2(u[2 * e + 1], v[2 * e + 1], make_float2(c[e].z, c[e].w), make_float2(s[e].z, s[e].w));
  }
}
__device__ __forceinline__ void turn_pairs(float2 (&u)[4], const float4& c, const float4& s) {
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    float2 p = make_float2(u[e].x, u[e + 1].x), q = make_float2(u[e].y, u[e + 1].y);
    rotary::turn2(p, q, e ? make_float2(c.z, c.w) : make_float2(c.x, c.y), e ? make_float2(s.z, s.w) : make_float2(s.x, s.y));
    u[e] = make_float2(p.x, q.x);
    u[e + 1] = make_float2(p.y, q.y);
  }
}

// A head's queries of a run, by a warp: a lane has a piece of a row (HALF: eight dims of each half), four (fp32: two) of them at a time.
template <typename T, int NG, bool HALF>
__device__ __forceinline__ void rotate_slice(const T* x, int64_t ldx, T* out, int64_t ldo, const float* cs, const int* pos, int rot, bool copy) {
  using X = typename Vec8<T>::type;
  constexpr int D = 64 * NG, R = kRun<NG>, kAhead = sizeof(T) == 2 ? 4 : 2;
  const int lane = threadIdx.x & 31, P = rot / 2;
  const int turn = HALF ? rot / 16 : rot / 8, per = turn + (copy ? (D - rot) / 8 : 0);
  for (int i0 = lane; i0 < R * per; i0 += 32 * kAhead) {
    X a[kAhead], b[kAhead];
    int row[kAhead], j[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int i = i0 + 32 * e;
      row[e] = i / per;
      j[e] = i - row[e] * per;
      if (i >= R * per || pos[row[e]] < 0) row[e] = -1;
      if (row[e] >= 0) {
        const T* from = x + row[e] * ldx + (j[e] < turn ? 8 * j[e] : rot + 8 * (j[e] - turn));
        get8(from, a[e]);
        if (HALF && j[e] < turn) get8(from + P, b[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      if (row[e] < 0) continue;
      T* to = out + row[e] * ldo + (j[e] < turn ? 8 * j[e] : rot + 8 * (j[e] - turn));
      if (j[e] < turn) {
        float2 u[4], v[4];
        float4 c[2], s[2];
        read_cs<HALF>(cs + row[e] * rot, HALF ? 8 * j[e] : 4 * j[e], P, c, s);
        unpack(a[e], u);
        if (HALF) {
          unpack(b[e], v);
          turn_half(u, v, c, s);
          pack(b[e], v);
          put8(to + P, b[e]);
        } else {
          turn_pairs(u, c[0], s[0]);
        }
        pack(a[e], u);
      }
      put8(to, a[e]);
    }
  }
}

// The lane's eight dims (chunk ck of the row's head) rotated; cs: the row's cosines and sines.
template <bool HALF, class X>
__device__ __forceinline__ void rotate8(X& x, const float* cs, int ck, int rot, int lane) {
  const int P = rot / 2;
  float2 u[4], v[4];
  if (HALF) {
    const int far = rot / 16;   // chunks of a half
    const bool second = ck >= far, on = ck < 2 * far;
    const X y = from_lane(x, on ? lane - ck + (second ? ck - far : ck + far) : lane);   // all lanes take part
    if (!on) return;
    unpack(second ? y : x, u);
    unpack(second ? x : y, v);
    float4 c[2], s[2];
    read_cs<true>(cs, 8 * (second ? ck - far : ck), P, c, s);
    turn_half(u, v, c, s);
    if (second) pack(x, v);
    else pack(x, u);
  } else {
    if (8 * ck >= rot) return;
    unpack(x, u);
    float4 c[2], s[2];
    read_cs<false>(cs, 4 * ck, P, c, s);
    turn_pairs(u, c[0], s[0]);
    pack(x, u);
  }
}

template <typename T, int NG, bool HALF>
__global__ void __launch_bounds__(kThreads, 2) rotated_kernel(const RotatedArgs<T> a) {
  constexpr int D = 64 * NG, R = kRun<NG>;
  using X = typename Vec8<T>::type;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t run_token[R];
  __shared__ int run_pos[R];
  float* const cs = reinterpret_cast<float*>(smem + kRingBytes<T>);   // [R][2][rot / 2]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = lane & 7, gi = (lane >> 3) % NG, rb = (lane >> 3) / NG, ck = 8 * gi + part;
  const int heads = a.pool.heads, all = 2 * heads + a.q_heads;
  uint4* const ring = reinterpret_cast<uint4*>(smem) + warp * (2 * kBatches * 32) + lane;
  tc::griddep_launch();
  tc::griddep_wait();
  const int64_t runs = (a.batch.ntok + R - 1) / R;
  const int of_block = kWarps * a.slices, chunks = (all + of_block - 1) / of_block;
  if (blockIdx.x == 0)   // what no row would notice: offsets that run backwards
    for (int i = threadIdx.x; i < a.tab.seqs; i += kThreads) seq_of(a.tab, a.batch, i);
  for (int64_t it = blockIdx.x; it < runs * chunks; it += gridDim.x) {
    const int64_t row0 = it / chunks * R;
    const int s0 = static_cast<int>(it % chunks) * of_block, s1 = min(all, s0 + of_block);
    __syncthreads();   // the run before is done with
    if (threadIdx.x < R) {
      int pos = -1;
      uint32_t token = kNoToken;
      if (row0 + lane < a.batch.ntok) token = token_of_row(a.tab, a.batch, static_cast<int>(row0 + lane), pos);
      run_token[lane] = token;
      run_pos[lane] = pos;
    }
    __syncthreads();
    uint32_t tok[kBatches];   // of this lane's row in each batch
    uint32_t there = 0;       // bit b: the row stands at a position
#pragma unroll
    for (int b = 0; b < kBatches; ++b) {
      tok[b] = run_token[b * (4 / NG) + rb];
      there |= (run_pos[b * (4 / NG) + rb] >= 0 ? 1u : 0u) << b;
    }
    const uint32_t mine = run_token[part * (4 / NG) + rb];
    auto kind_of = [&](int sl) { return sl < heads ? 0 : sl < 2 * heads ? 1 : 2; };
    auto source = [&](int sl) {   // the lane's values of the run's first row
      const int kind = kind_of(sl);
      return (kind == 0 ? a.src[0] : kind == 1 ? a.src[1] : a.src[2]) + row0 * (kind == 0 ? a.ld[0] : kind == 1 ? a.ld[1] : a.ld[2]) +
             static_cast<int64_t>(sl - kind * heads) * D + 8 * ck;
    };
    auto stride = [&](int sl) { return sl < heads ? a.ld[0] : sl < 2 * heads ? a.ld[1] : a.ld[2]; };
    auto fetch = [&](int sl, int slot) {
      if (sl < s1 && kind_of(sl) != 2) {
        const T* src = source(sl);
        const int64_t ld = stride(sl);
#pragma unroll
        for (int b = 0; b < kBatches; ++b)
          cp16_zfill(tc::smem_u32(ring + (slot * kBatches + b) * 32), (there >> b) & 1u ? src + (b * (4 / NG) + rb) * ld : src, (there >> b) & 1u);
      }
      tc::cp_async_commit();
    };
    int slot = 0;
    if constexpr (kRing<T>) fetch(s0 + warp, 0);
    if (s0 < heads || s1 > 2 * heads) {   // cosines and sines, under the first copies
      const int P = a.rot / 2;
      for (int i = threadIdx.x; i < R * P; i += kThreads) {
        const int r = i / P, p = i - r * P;
        const float2 v = rotary::cos_sin(rotary::phase_of(run_pos[r], a.turns[p]), a.scale);
        float* row = cs + 2 * r * P;
        row[cs_at<HALF>(0, p, P)] = v.x;
        row[cs_at<HALF>(1, p, P)] = v.y;
      }
    }
    __syncthreads();
    for (int sl = s0 + warp; sl < s1; sl += kWarps, slot ^= 1) {
      const int kind = kind_of(sl), h = sl - kind * heads;
      if (kind == 2) {
        rotate_slice<T, NG, HALF>(a.src[2] + row0 * a.ld[2] + static_cast<int64_t>(h) * D, a.ld[2], a.q_out + row0 * a.ldqo + static_cast<int64_t>(h) * D, a.ldqo,
                                  cs, run_pos, a.rot, a.src[2] != a.q_out);
        if constexpr (kRing<T>) fetch(sl + kWarps, slot ^ 1);   // a group of copies each round
        continue;
      }
      X held[kBatches];
      if constexpr (kRing<T>) {
        fetch(sl + kWarps, slot ^ 1);
        tc::cp_async_wait<1>();   // a lane reads what it copied itself
        if (kind == 0)
#pragma unroll
          for (int b = 0; b < kBatches; ++b) held[b].raw = ring[(slot * kBatches + b) * 32];
      } else {
        const T* src = source(sl);
        const int64_t ld = stride(sl);
#pragma unroll
        for (int b = 0; b < kBatches; ++b) {
          if ((there >> b) & 1u) held[b].load(src + (b * (4 / NG) + rb) * ld);
          else held[b].clear();
        }
      }
      if (kind == 0) {
#pragma unroll
        for (int b = 0; b < kBatches; ++b) rotate8<HALF>(held[b], cs + (b * (4 / NG) + rb) * a.rot, ck, a.rot, lane);
        store_slice<T, NG>(a.pool, false, h, tok, mine, row0, a.restored[0], a.ldr, [&](int b) { return held[b]; });
      } else {
        auto batch = [&](int b) {
          if constexpr (kRing<T>) return X{ring[(slot * kBatches + b) * 32]};
          else return held[b];
        };
        store_slice<T, NG>(a.pool, true, h, tok, mine, row0, a.restored[1], a.ldr, batch);
      }
    }
    if constexpr (kRing<T>) tc::cp_async_wait<0>();
  }
}

template <typename T, int NG, bool HALF>
fg_status launch_kernel(const RotatedArgs<T>& a, unsigned grid, cudaStream_t st) {
  constexpr int kMost = kRingBytes<T> + kRun<NG> * 64 * NG * 4;
  const size_t smem = kRingBytes<T> + static_cast<size_t>(kRun<NG>) * a.rot * sizeof(float);
  static bool set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (kMost > 48 * 1024 && dev >= 0 && dev < 64 && !set[dev]) {
    if (cudaFuncSetAttribute(rotated_kernel<T, NG, HALF>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess)
      return check_launch("rotated_kernel smem attribute");
    set[dev] = true;
  }
  Trace tr(KC_KV_STORE, st);
  return paged::launch("rotated_kernel", true, rotated_kernel<T, NG, HALF>, grid, kThreads, smem, st, a);
}

template <typename T>
fg_status launch_rotated(RotatedArgs<T>& a, int head_dim, int layout, cudaStream_t st) {
  const int run = head_dim == 128 ? kRun<2> : kRun<1>;
  const int64_t runs = (a.batch.ntok + run - 1) / run, all = 2 * a.pool.heads + a.q_heads, sms = num_sms();
  // as many slices a warp as leave every SM two blocks, so that a run's angles are worked out no oftener than need be
  const int64_t fit = runs * all / (sms * 2 * kWarps);
  a.slices = static_cast<int>(fit < 1 ? 1 : fit > 8 ? 8 : fit);
  const int64_t items = runs * ((all + kWarps * a.slices - 1) / (kWarps * a.slices)), cap = sms * 16;
  const unsigned grid = static_cast<unsigned>(items < cap ? items : cap);
  const bool half = layout == FG_ROTARY_HALF;
  if (head_dim == 128) return half ? launch_kernel<T, 2, true>(a, grid, st) : launch_kernel<T, 2, false>(a, grid, st);
  return half ? launch_kernel<T, 1, true>(a, grid, st) : launch_kernel<T, 1, false>(a, grid, st);
}

template <typename T>
fg_status run_rotated(const fg_page_pool& pool, const fg_page_table& t, const int32_t* cu, const fg_rotary& r, const void* q,
                      int64_t ldq, int32_t q_heads, void* q_out, int64_t ldqo, const void* k, const void* v, int64_t ld, int64_t ntok,
                      void* kr, void* vr, int64_t ldr, unsigned int* err, cudaStream_t st) {
  RotatedArgs<T> a;
  a.pool = pool_of(pool);
  a.tab = table_of(t);
  a.batch = Batch{cu, static_cast<int>(ntok), err};
  a.turns = r.turns;
  a.src[0] = static_cast<const T*>(k);
  a.src[1] = static_cast<const T*>(v);
  a.src[2] = static_cast<const T*>(q);
  a.restored[0] = static_cast<T*>(kr);
  a.restored[1] = static_cast<T*>(vr);
  a.q_out = static_cast<T*>(q_out);
  a.ld[0] = a.ld[1] = ld;
  a.ld[2] = ldq;
  a.ldr = ldr;
  a.ldqo = ldqo;
  a.q_heads = q ? q_heads : 0;
  a.rot = r.rot;
  a.scale = r.scale;
  return launch_rotated(a, pool.head_dim, r.layout, st);
}

}  // namespace
}  // namespace paged
}  // namespace fg

using namespace fg;
using namespace fg::paged;

extern "C" fg_status fg_paged_append_rotated(const fg_page_pool* pool, const fg_page_table* t, const int32_t* cu, const fg_rotary* r,
                                             const void* q, int64_t ldq, int32_t q_heads, void* q_out, int64_t ldqo, const void* k,
                                             const void* v, int64_t ld, int64_t ntok, void* k_restored, void* v_restored,
                                             int64_t ldr, cudaStream_t stream) {
  FG_TRY(check_pool_table(pool, t));
  FG_TRY(check_rotary(r, pool->head_dim));
  if (r->rot % 16) return fail(FG_ERR_SHAPE, "rotation of %d dims: a multiple of 16 here", r->rot);
  if (ntok < 0 || q_heads < 0) return fail(FG_ERR_ARG, "negative sizes");
  if (q_heads > 65535) return fail(FG_ERR_UNSUPPORTED, "more than 65535 query heads");
  if (pool->pages * pool->page_size >= UINT32_MAX) return fail(FG_ERR_UNSUPPORTED, "a pool of 2^32 tokens or more");
  if (ntok > INT32_MAX - 256) return fail(FG_ERR_UNSUPPORTED, "more than 2^31 rows");
  if (ntok == 0 || t->seqs == 0) return FG_OK;
  if (!cu || !k || !v || (q && q_heads > 0 && !q_out)) return fail(FG_ERR_ARG, "null pointer");
  if ((k_restored == nullptr) != (v_restored == nullptr)) return fail(FG_ERR_ARG, "restored K and V: both or neither");
  const int64_t h1 = static_cast<int64_t>(pool->heads) * pool->head_dim, hq = q ? static_cast<int64_t>(q_heads) * pool->head_dim : 0;
  if (ld < h1 || (k_restored && ldr < h1)) return fail(FG_ERR_SHAPE, "row stride below heads * head_dim = %lld", (long long)h1);
  if (hq > 0 && (ldq < hq || ldqo < hq)) return fail(FG_ERR_SHAPE, "row stride below q_heads * head_dim = %lld", (long long)hq);
  if (!aligned(cu, 4) || !aligned(k, 16) || !aligned(v, 16) || ld % 8 || !aligned(k_restored, 16) || !aligned(v_restored, 16) ||
      (k_restored && ldr % 8) || (hq > 0 && (!aligned(q, 16) || !aligned(q_out, 16) || ldq % 8 || ldqo % 8)))
    return fail(FG_ERR_ALIGN, "rows need 16-byte alignment and strides that are multiples of 8");
  if (hq > 0) {
    const fg_dtype dt = static_cast<fg_dtype>(pool->dtype);
    FG_TRY(check_apart(q, ldq, q_out, ldqo, ntok, hq, dt));
    // blocks read k and v, and write restored rows, while others move queries
    for (const void* x : {k, v})
      if (rows_meet(x, ld, h1, q_out, ldqo, hq, ntok, dt)) return fail(FG_ERR_ARG, "rotated queries over keys or values");
    for (const void* x : {k_restored, v_restored})
      if (x && (rows_meet(x, ldr, h1, q_out, ldqo, hq, ntok, dt) || rows_meet(x, ldr, h1, q, ldq, hq, ntok, dt)))
        return fail(FG_ERR_ARG, "restored rows over queries");
  }
  unsigned int* err = device_error_word();
  if (!err) return fail(FG_ERR_CUDA, "device error word");
  if (pool->dtype == FG_F16)
    return run_rotated<__half>(*pool, *t, cu, *r, q, ldq, q_heads, q_out, ldqo, k, v, ld, ntok, k_restored, v_restored, ldr, err, stream);
  return run_rotated<float>(*pool, *t, cu, *r, q, ldq, q_heads, q_out, ldqo, k, v, ld, ntok, k_restored, v_restored, ldr, err, stream);
}
