// Paged attention of sequences with at most 16 rows per K/V head (decode
// steps; FlexGen notes, "背景知识" decode equations, "5. 近似方法" 4-bit K/V),
// fp16 activations.
//
// The path is bound by the cache's bytes, so every byte is read once for all
// rows of a K/V head (8 rows are one N = 8 block of the warp-level MMA) and
// codes are multiplied as they are:
//   scores   s = sum_g scale_g (q . c)_g + min_g (sum q)_g: a masked nibble
//            is the subnormal fp16 c * 2^-24 (or 16 c * 2^-24, against q /
//            16), which the MMA multiplies exactly: no bias to take out;
//   values   o = sum_t (p_t scale_t) (c_t - 8) + sum_t p_t (min_t + 8
//            scale_t), tile by tile: a tile's MMAs begin from -8 sum w, which
//            centres the code, because the MMA truncates and a positive sum
//            over thousands of tokens would lose its low bits.  The weight w =
//            p * scale is rounded to fp16 for the MMA after scaling by a power
//            of two that fits the largest weight of the query, so that small
//            activations keep their bits; sum w is an MMA against ones, of the
//            rounded weights.  Where rows leave half the MMA's columns free (1
//            to 4; up to 8 when max_q allows more than 8), those carry the rounding's
//            remainders: the result is then as exact as fp32 sums of unrounded
//            weights (2.1e-4 of its size off, the fp16 result's own rounding;
//            otherwise 3.1 to 3.6e-4: for 5 to 8 rows a second MMA beside
//            each, with the remainders, gave 2.5e-4 and took 125 us for the
//            107 of the long step below).
// A warp is a worker (see paged_sched.cuh) and walks tiles of 32 tokens of its
// share: its own ring of stages in shared memory, filled by asynchronous
// copies kStages - 1 tiles ahead across items; no CTA barrier.  Where the next
// 32 tiles lie (item, pages, edges) the lanes look up together, a tile each:
// one tile after another that took a third of the instructions.  (A warp that
// filled all rings by bulk copies, six a tile, measured slower: 178 us against
// 124 for a step over 8 sequences of 30 to 65 thousand tokens.)  Rows of a
// stage lie so that both the score reads (8 bytes of token s(g)) and the value
// reads (4 bytes of 4 tokens side by side) fall on 32 different banks: token
// row m of an MMA is token s(m) = m/2 + 4 (m%2), which makes the transposed
// weights' token pairs (tig, tig + 4), and 16-byte pieces are swizzled by the
// row.
//
// Measured, a call replayed from a graph (plan in the kernel, join after it):
// 64 sequences of 300 to 900 tokens, 32 heads of 128, one row each 54 us (3.6
// TB/s); 8 sequences of 30 to 65 thousand tokens, 8 K/V heads of 128 with 8
// query heads each 107 us (4.7 TB/s; the copies alone, without the sums, 95);
// 4 sequences of 100 to 300 tokens, 12 heads of 64 10.7 us, of which the two
// launches are most.  What bounds a long step are fixed latencies at three warps
// a scheduler (issue slots 56% used; a warp waits 16 of a tile's 3,200 cycles
// for copies; DRAM at 64% of its rate), then the integer pipe that masks the
// nibbles (45%); four warps of three CTAs and three stages were the best of the
// shapes tried (8 warps x 5 stages 120 us, 11 x 4 122).
#include <math.h>

#include <algorithm>

#include "attn_dev.cuh"
#include "paged_attn.cuh"
#include "tc_ptx.cuh"

namespace fg {
namespace paged {
namespace {

using attn::mma16816;
using attn::pack_h2;
using attn::unpack_h2;
using attn::kHiNib;
using attn::kLoNib;

constexpr int kTileLog2 = kStepTileLog2;
constexpr int kTile = 1 << kTileLog2;   // tokens of a tile
constexpr int kWarps = 4;               // warps of a CTA
// CTAs an SM.  Two blocks of columns take 255 registers at head_dim 128; in the 168 of three CTAs they spilled 668 bytes:
// 16 rows of 32 sequences of 4000 tokens 67 us for 108 (head_dim 64: 44 for 59), 63 single tokens beside a chunk of 512
// rows 355 for 549.
template <int NB>
constexpr int kCtasPerSm = NB == 2 ? 2 : 3;
template <int D, int NB>
constexpr int kStepStages = D == 128 ? 3 : 4;
constexpr float kGrow = 12.0f;          // how far (in powers of two) a score may lie above the maximum
// The weights w = p * scale travel as fp16 times a power of two, one per query and group: found when the sum of a lane's
// four would pass kMostW, so that the largest lies in [2^5, 2^6), and raised with the maximum of the scores.  What is small
// beside the largest weight of its row alone may lose bits (below 2^-19 of it), whatever the scales of tokens that the
// row does not see or gives no weight.
constexpr float kMostW = 32768.0f;
constexpr int kTargetW = 5;
constexpr float kMostInv = 1.329227995784916e36f;   // 2^120: of a row without weights

template <int D>
struct Stage {
  static constexpr int C = D / 2;                  // code bytes of a row
  static constexpr int NG = D / 64;
  static constexpr int kMeta = kTile * NG * 4;     // one (min or scale) array
  static constexpr int kV = kTile * C, kKs = 2 * kTile * C, kKm = kKs + kMeta, kVs = kKm + kMeta, kVm = kVs + kMeta;
  static constexpr int kInfo = kVm + kMeta;        // (first token, flags, head, sequence)
  static constexpr int kBytes = kInfo + 16;
};
// Flags of a tile: the halves that are there, every row sees all of it, the
// item's first and last tile, the share's last.
enum : int { kHalf0 = 1, kHalf1 = 2, kWhole = 4, kFirst = 8, kLast = 16, kEnd = 32 };
// Where the 16-byte piece pc of row t lies: pieces swizzled so that rows 0, 4,
// 1, 5 (and 2, 6, 3, 7), and rows 0 .. 3 (and 4 .. 7), use all banks.
template <int D>
__device__ __forceinline__ int piece_at(int t, int pc) {
  if (D == 128) return t * 64 + ((pc ^ ((((t >> 1) ^ (t >> 2)) & 1) << 1)) << 4);
  return (t ^ (((t >> 2) & 1) << 1)) * 32 + (pc << 4);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t add_h2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two fp32 at once (the queries 2 tig and 2 tig + 1 of a lane).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7};\n"
      "fma.rn.f32x2 x, x, y, z; mov.b64 {%0, %1}, x; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5};\n"
      "mul.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5};\n"
      "add.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float reciprocal2(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }   // of 2^k
// Whether one of two fp16 is above kMostW, or NaN.
__device__ __forceinline__ bool past(uint32_t h) {
  return !__hble2(*reinterpret_cast<const __half2*>(&h), __floats2half2_rn(kMostW, kMostW));
}
// The factor that takes the weight `most` > 0 into [2^kTargetW, 2 * 2^kTargetW).
__device__ __forceinline__ float factor_for(float most) {
  const int e = min(static_cast<int>(__float_as_uint(most) >> 23), 253);
  return __uint_as_float(static_cast<uint32_t>(min(254 + kTargetW - e, 247)) << 23);
}
constexpr uint32_t kOnes = 0x3C003C00u;   // fp16 (1, 1)
constexpr float k2p24 = 16777216.0f;      // a code's bits as a subnormal fp16 are c * 2^-24
// D = A B + C with C = (c0, c1, c2, c3)
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, float c0, float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// One query row as this lane's B fragments of each 64-group (dims 16 tig ..
// 16 tig + 15 of the group, in the order the code words give them: (0, 4),
// (1, 5) / 16 | (2, 6), (3, 7) / 16), and the sum of the query over this lane's
// dims.  The row is multiplied by the power of two that takes its largest
// element into [2^10, 2^11): a sixteenth of an element then loses bits only
// below 2^-20 of the largest, however small the row is.  undo takes that back.
template <int NG>
struct QFrag {
  uint32_t b[NG][4][2];
  float qsum[NG];
  float undo;
};
template <int NG>
__device__ __forceinline__ void load_q(QFrag<NG>& f, const __half* qrow, int tig, bool there) {
  uint4 raw[NG][2];
  uint32_t most = 0;                // of |q| as fp16 bits, two at once
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      raw[g][w] = there ? reinterpret_cast<const uint4*>(qrow + 64 * g + 16 * tig)[w] : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t x[4] = {raw[g][w].x, raw[g][w].y, raw[g][w].z, raw[g][w].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) most = __vmaxu2(most, x[e] & 0x7fff7fffu);
    }
  most = max(most >> 16, most & 0xffffu);
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
  // the exponent of the largest (zeros, infinities and NaN stay as they are)
  const uint32_t e = most == 0 || most >= 0x7c00u ? 127u + 10u : __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(most)))) >> 23;
  const float up = __uint_as_float((264u - e) << 23);
  f.undo = __uint_as_float((e - 10u) << 23);
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    f.qsum[g] = 0.0f;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const float2 up2 = both(up), up16 = both(up * 0.0625f);
      const float2 d01 = unpack_h2(raw[g][w].x), d23 = unpack_h2(raw[g][w].y), d45 = unpack_h2(raw[g][w].z), d67 = unpack_h2(raw[g][w].w);
      auto pair = [](float a, float b, float2 by) { const float2 p = mul2(make_float2(a, b), by); return pack_h2(p.x, p.y); };
      f.b[g][2 * w][0] = pair(d01.x, d45.x, up2);
      f.b[g][2 * w][1] = pair(d01.y, d45.y, up16);
      f.b[g][2 * w + 1][0] = pair(d23.x, d67.x, up2);
      f.b[g][2 * w + 1][1] = pair(d23.y, d67.y, up16);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 x = unpack_h2(f.b[g][2 * w + h][0]), y = unpack_h2(f.b[g][2 * w + h][1]);
        f.qsum[g] += (x.x + x.y) + 16.0f * (y.x + y.y);
      }
    }
  }
}

// (scale or min) of a row's groups from a stage's array.
template <int NG>
__device__ __forceinline__ void read_meta(const uint8_t* arr, int t, float (&v)[NG]) {
  if (NG == 2) {
    const float2 x = *reinterpret_cast<const float2*>(arr + 8 * t);
    v[0] = x.x;
    v[NG - 1] = x.y;
  } else {
    v[0] = *reinterpret_cast<const float*>(arr + 4 * t);
  }
}

template <int D, int NB>
__global__ void __launch_bounds__(32 * kWarps, kCtasPerSm<NB>) step_kernel(const AttnArgs<__half> a, const ClassPlan pl, const bool own_plan) {
  constexpr int NG = D / 64, NT = D / 16;
  using St = Stage<D>;
  constexpr int kStages = kStepStages<D, NB>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gq = lane >> 2, tig = lane & 3;
  uint8_t* ring = smem + warp * (kStages * St::kBytes);
  const int w = blockIdx.x * kWarps + warp;

  tc::griddep_launch();
  tc::griddep_wait();
  __shared__ OwnPlan own;
  const Line line = own_plan ? make_line<true, kStepRows, kTileLog2>(own, a.tab, a.batch, a.shape, a.pool.heads, pl.workers, false)
                             : Line{pl.pre, pl.head[0], pl.head[1]};
  const int64_t* const pre = line.pre;
  const int64_t total = line.total, per = line.per;
  const int64_t o0 = w * per;
  if (o0 >= total) {
    if (lane == 0) pl.rec[w] = make_int4(-1, 0, 0, 0);
    return;
  }
  const int heads = a.pool.heads;

  const int mine = static_cast<int>(total - o0 < per ? total - o0 : per);   // tiles of the share

  // ---- looking up: a lane finds one of the next 32 tiles ----------------------------
  const int psl = a.pool.ps_log2, psm = (1 << psl) - 1;
  int t_i = 0, t_h = 0, t_key = 0, t_flags = 0, t_pg0 = -1, t_pg1 = -1;
  {
    int lo = 0, hi = a.tab.seqs;     // pre[lo] <= o0 < pre[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= o0) lo = mid;
      else hi = mid;
    }
    t_i = lo;
  }
  auto look_up = [&](int k) {        // tile k + lane of the share
    k += lane;
    t_pg0 = t_pg1 = -1;
    if (k >= mine) return;
    const int64_t o = o0 + k;
    while (pre[t_i + 1] <= o) ++t_i;
    const Seq s = seq_of(a.tab, a.batch, t_i);
    const Span sp = span_of<kTileLog2>(s.len - s.n, s.len - 1, s.keys, a.shape.window, a.shape.sinks);
    const int64_t in = o - pre[t_i];
    t_h = in <= INT32_MAX ? static_cast<int>(in) / sp.n : static_cast<int>(in / sp.n);
    const int x = static_cast<int>(in - static_cast<int64_t>(t_h) * sp.n);
    t_key = sp.tile(x) << kTileLog2;
    const int last = min(s.len, s.keys) - 1, lo_key = a.shape.window > 0 ? s.len - s.n - a.shape.window + 1 : 0;
    // page of the 16 tokens from t on (-1: none, or nothing of them is seen)
    auto page_at = [&](int t) {
      if (t > last || (t + 15 < lo_key && t >= a.shape.sinks)) return -1;
      const int page = a.tab.table[t_i * a.tab.stride + (t >> psl)];   // t <= last < keys: the row reaches that far
      if (static_cast<uint32_t>(page) < static_cast<uint32_t>(a.tab.pages)) return page;
      atomicOr(a.batch.err, DEV_ERR_PAGE);
      return -1;
    };
    t_pg0 = page_at(t_key);
    t_pg1 = psl >= kTileLog2 && t_key + 16 <= last && t_pg0 >= 0 ? t_pg0 : page_at(t_key + 16);
    // a row sees all of the tile: inside all rows' positions, stored, and inside the window or the sinks
    const bool whole = t_pg0 >= 0 && t_pg1 >= 0 && t_key + kTile - 1 <= min(s.len - s.n, s.keys - 1) &&
                       (a.shape.window == 0 || t_key >= s.len - a.shape.window || t_key + kTile <= a.shape.sinks);
    t_flags = (t_pg0 >= 0 ? kHalf0 : 0) | (t_pg1 >= 0 ? kHalf1 : 0) | (whole ? kWhole : 0) | (x == 0 ? kFirst : 0) |
              (x + 1 == sp.n ? kLast : 0) | (k + 1 == mine ? kEnd : 0);
  };
  // ---- copying ------------------------------------------------------------------
  // A lane's pieces lie at the same places of every half tile: 16-byte pieces
  // lane and lane + 32 of the 16 rows' codes, and piece lane % (4 NG) of the
  // (scale or min) array lane / (4 NG).
  const uint32_t page_codes = static_cast<uint32_t>(heads) * static_cast<uint32_t>(St::C) << psl;   // bytes of a page
  const uint32_t page_meta = static_cast<uint32_t>(heads) * static_cast<uint32_t>(4 * NG) << psl;
  const bool meta_lane = lane < 16 * NG;
  const int arr = lane / (4 * NG), mpc = lane % (4 * NG);
  const char* const meta0 = reinterpret_cast<const char*>(arr == 0   ? a.pool.scales[0]
                                                          : arr == 1 ? a.pool.mins[0]
                                                          : arr == 2 ? a.pool.scales[1]
                                                                     : a.pool.mins[1]) +
                            16 * mpc;
  const int meta_at = St::kKs + arr * St::kMeta + 16 * mpc;
  const uint32_t ring_u32 = tc::smem_u32(ring);
  const int to0 = piece_at<D>(lane / (St::C / 16), lane % (St::C / 16)), to1 = D == 128 ? piece_at<D>(8 + lane / 4, lane % 4) : 0;
  // one half's codes and (min, scale) into stage s
  auto copy_half = [&](uint32_t s, int hf, int page, uint32_t row) {   // row: of the page's arrays
    const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(page)) * page_codes + (row * St::C + 16 * lane);
    const uint8_t* kc = a.pool.codes[0] + at;
    const uint8_t* vc = a.pool.codes[1] + at;
    const uint32_t to = s + 16 * hf * St::C;
    cp16(to + to0, kc);
    cp16(to + St::kV + to0, vc);
    if (D == 128) {
      cp16(to + to1, kc + 512);
      cp16(to + St::kV + to1, vc + 512);
    }
    if (meta_lane)
      cp16(s + meta_at + hf * (64 * NG), meta0 + (static_cast<uint64_t>(static_cast<uint32_t>(page)) * page_meta + row * (4 * NG)));
  };
  // copies the share's next tile into the stage at offset st
  int next = 0;
  auto issue = [&](uint32_t st) {
    if (next < mine) {
      const int from = next & 31;
      if (from == 0) look_up(next);
      const int key = __shfl_sync(0xffffffffu, t_key, from), h = __shfl_sync(0xffffffffu, t_h, from);
      const int pg0 = __shfl_sync(0xffffffffu, t_pg0, from), pg1 = __shfl_sync(0xffffffffu, t_pg1, from);
      const uint32_t row = (static_cast<uint32_t>(h) << psl);
      if (pg0 >= 0) copy_half(ring_u32 + st, 0, pg0, row + (key & psm));
      if (pg1 >= 0) copy_half(ring_u32 + st, 1, pg1, row + ((key + 16) & psm));
      if (lane == from) *reinterpret_cast<int4*>(ring + st + St::kInfo) = make_int4(t_key, t_flags, t_h, t_i);
      ++next;
    }
    tc::cp_async_commit();
  };

  // ---- the item's state --------------------------------------------------------
  uint32_t qb[NB][NG][4][2];                     // q as B fragments (query gq of each block of 8)
  float2 qsum[NB][NG];                           // of queries 2 tig, 2 tig + 1
  float m[NB][2];
  float2 l[NB], cmn[NB][NG];
  float acc[NB][NT][4];
  float2 inv[NB][NG];                            // the weights' factor
  uint32_t nans = 0;                             // bit 4 nb + 2 e + g: the query sees a NaN value group
  int rows = 0, row0 = 0, keys = 0;
  // Up to four rows (eight with two blocks of columns) leave half of the MMAs' columns free: columns 4 .. 7 (the second
  // block) take the same queries again and carry what the rounding of the weights to fp16 left over, so that the two add
  // up to the weights in full.
  bool split = false;
  float2 kc2[NB];                                // takes scores of queries 2 tig, 2 tig + 1 to base 2

  int pn[NB][2];                                 // positions of queries 2 tig, 2 tig + 1 (none: below every key)

  auto begin_item = [&](const uint8_t* s) {
    const int4 info = *reinterpret_cast<const int4*>(s + St::kInfo);
    const int h = info.z;
    const Seq sq = seq_of(a.tab, a.batch, info.w);
    rows = sq.n * a.shape.group;
    split = rows <= 4 * NB;
    row0 = sq.row0;
    keys = sq.keys;
    const int pos0 = sq.len - sq.n;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int n = !split ? 8 * nb + gq : NB == 1 ? gq & 3 : gq;
      QFrag<NG> f;
      const int t = n / a.shape.group;
      load_q<NG>(f, a.q + static_cast<int64_t>(row0 + t) * a.ldq + static_cast<int64_t>(h * a.shape.group + n - t * a.shape.group) * D,
                 tig, n < rows);
      kc2[nb] = make_float2(a.scale_log2 * __shfl_sync(0xffffffffu, f.undo, 8 * tig), a.scale_log2 * __shfl_sync(0xffffffffu, f.undo, 8 * tig + 4));
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float sum = f.qsum[g];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        qsum[nb][g] = make_float2(__shfl_sync(0xffffffffu, sum, 8 * tig), __shfl_sync(0xffffffffu, sum, 8 * tig + 4));
        cmn[nb][g] = both(0.0f);
        inv[nb][g] = both(kMostInv);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          qb[nb][g][e][0] = f.b[g][e][0];
          qb[nb][g][e][1] = f.b[g][e][1];
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = !split ? 8 * nb + 2 * tig + e : NB == 1 ? (2 * tig + e) & 3 : 2 * tig + e;
        pn[nb][e] = k < rows ? pos0 + k / a.shape.group : -(1 << 30);
        m[nb][e] = -INFINITY;
      }
      l[nb] = both(0.0f);
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[nb][i][0] = acc[nb][i][1] = acc[nb][i][2] = acc[nb][i][3] = 0.0f;
    }
    nans = 0;
  };

  auto compute = [&](uint8_t* s, int t0, int flags) {
    float2 sc[NB][2][2];                // [block][half][row]: scores, then weights, of this lane's two queries
    const int tok = (gq >> 1) + 4 * (gq & 1);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint2 kw[2][NG];
      float ks[2][NG], km[2][NG];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int t = 16 * hf + 8 * r + tok;
#pragma unroll
        for (int g = 0; g < NG; ++g)
          kw[r][g] = *reinterpret_cast<const uint2*>(s + piece_at<D>(t, 2 * g + (tig >> 1)) + 8 * (tig & 1));
        read_meta<NG>(s + St::kKs, t, ks[r]);
        read_meta<NG>(s + St::kKm, t, km[r]);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float d[NB][4];
#pragma unroll
        for (int ww = 0; ww < 2; ++ww) {
          const uint32_t x0 = ww ? kw[0][g].y : kw[0][g].x, x1 = ww ? kw[1][g].y : kw[1][g].x;
          const uint32_t y0 = x0 >> 8, y1 = x1 >> 8;
          const uint32_t a0 = (x0 & kLoNib), a1 = (x1 & kLoNib);
          const uint32_t a2 = (x0 & kHiNib), a3 = (x1 & kHiNib);
          const uint32_t b0 = (y0 & kLoNib), b1 = (y1 & kLoNib);
          const uint32_t b2 = (y0 & kHiNib), b3 = (y1 & kHiNib);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            if (ww == 0)
              mma_from(d[nb], a0, a1, a2, a3, qb[nb][g][0][0], qb[nb][g][0][1], 0.0f, 0.0f, 0.0f, 0.0f);
            else
              mma16816(d[nb], a0, a1, a2, a3, qb[nb][g][2][0], qb[nb][g][2][1]);
            mma16816(d[nb], b0, b1, b2, b3, qb[nb][g][2 * ww + 1][0], qb[nb][g][2 * ww + 1][1]);
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float2 base = g == 0 ? mul2(both(km[r][0]), qsum[nb][0]) : fma2(both(km[r][g]), qsum[nb][g], sc[nb][hf][r]);
            sc[nb][hf][r] = fma2(both(ks[r][g] * k2p24), make_float2(d[nb][2 * r], d[nb][2 * r + 1]), base);
          }
      }
    }
    // scale or minimum of this lane's value token of half hf, row r
    auto value_meta = [&](uint8_t* arr, int hf, int r, int g) {
      return reinterpret_cast<float*>(arr) + (16 * hf + 8 * r + tok) * NG + g;
    };
    uint32_t seen = 0xffffffffu;   // bit 8 nb + 4 hf + 2 r + e: the query sees the token
    if (!(flags & kWhole)) {       // a row or a token at the edge
      seen = 0;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int j = t0 + 16 * hf + 8 * r + tok;
          const bool here = ((flags >> hf) & 1) && j < keys;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int p = pn[nb][e];
              const bool see = here && j <= p && (a.shape.window == 0 || j > p - a.shape.window || j < a.shape.sinks);
              if (!see) (e ? sc[nb][hf][r].y : sc[nb][hf][r].x) = -INFINITY;
              seen |= (see ? 1u : 0u) << (8 * nb + 4 * hf + 2 * r + e);
            }
          // what was not copied may be anything: its values count as zeros
          if (!here && tig == 0)
#pragma unroll
            for (int g = 0; g < NG; ++g) *value_meta(s + St::kVs, hf, r, g) = *value_meta(s + St::kVm, hf, r, g) = 0.0f;
        }
      __syncwarp();
    }
    // The maximum known so far serves while no score of a query lies more than 2^12 above it (a larger one would only change
    // the scale of sums that are divided in the end).  Otherwise, and before a key was seen, the tile's maximum is found
    // over the lanes of a query and the sums are rescaled.
    bool asks[NB][2];
    bool ask = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const float x = fmaxf(fmaxf(sc[nb][0][0].x, sc[nb][0][1].x), fmaxf(sc[nb][1][0].x, sc[nb][1][1].x));
      const float y = fmaxf(fmaxf(sc[nb][0][0].y, sc[nb][0][1].y), fmaxf(sc[nb][1][0].y, sc[nb][1][1].y));
      asks[nb][0] = (x - m[nb][0]) * kc2[nb].x > kGrow;   // -inf - -inf: no
      asks[nb][1] = (y - m[nb][1]) * kc2[nb].y > kGrow;
      ask = ask || asks[nb][0] || asks[nb][1];
    }
    if (__any_sync(0xffffffffu, ask)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float x = fmaxf(fmaxf(sc[nb][0][0].x, sc[nb][0][1].x), fmaxf(sc[nb][1][0].x, sc[nb][1][1].x));
        float y = fmaxf(fmaxf(sc[nb][0][0].y, sc[nb][0][1].y), fmaxf(sc[nb][1][0].y, sc[nb][1][1].y));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
        }
        // only the queries whose sums ask for it: a row's bits do not depend on its neighbours
        const uint32_t mine = 0x11111111u << tig;
        const bool ask0 = __ballot_sync(0xffffffffu, asks[nb][0]) & mine, ask1 = __ballot_sync(0xffffffffu, asks[nb][1]) & mine;
        const float nm[2] = {ask0 ? fmaxf(m[nb][0], x) : m[nb][0], ask1 ? fmaxf(m[nb][1], y) : m[nb][1]};
        float al[2], grown[2];            // the power of two by which the weights' factor grows with the maximum
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float up = (nm[e] - m[nb][e]) * (e ? kc2[nb].y : kc2[nb].x);
          al[e] = nm[e] == -INFINITY ? 1.0f : ex2(-up);
          grown[e] = nm[e] == -INFINITY ? 1.0f : __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(fminf(up, 126.0f))) << 23);
        }
        const float2 f = make_float2(al[0], al[1]);
        l[nb] = mul2(l[nb], f);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          cmn[nb][g] = mul2(cmn[nb][g], f);
          const float ni[2] = {fminf(inv[nb][g].x * grown[0], kMostInv), fminf(inv[nb][g].y * grown[1], kMostInv)};
          const float fx = al[0] * (ni[0] * reciprocal2(inv[nb][g].x)), fy = al[1] * (ni[1] * reciprocal2(inv[nb][g].y));
          inv[nb][g] = make_float2(ni[0], ni[1]);
#pragma unroll
          for (int i = 4 * g; i < 4 * g + 4; ++i) {
            acc[nb][i][0] *= fx;
            acc[nb][i][1] *= fy;
            acc[nb][i][2] *= fx;
            acc[nb][i][3] *= fy;
          }
        }
        m[nb][0] = nm[0];
        m[nb][1] = nm[1];
      }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const float2 neg = make_float2(m[nb][0] == -INFINITY ? 0.0f : -m[nb][0] * kc2[nb].x, m[nb][1] == -INFINITY ? 0.0f : -m[nb][1] * kc2[nb].y);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 x = fma2(sc[nb][hf][r], kc2[nb], neg);
          sc[nb][hf][r] = make_float2(ex2(x.x), ex2(x.y));   // scores become weights
          l[nb] = add2(l[nb], sc[nb][hf][r]);
        }
    }
    float vs[2][2][NG], mid[2][2][NG];   // scales, and values of the centre code
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        read_meta<NG>(s + St::kVs, 16 * hf + 8 * r + tok, vs[hf][r]);
        read_meta<NG>(s + St::kVm, 16 * hf + 8 * r + tok, mid[hf][r]);
#pragma unroll
        for (int g = 0; g < NG; ++g) mid[hf][r][g] = fmaf(8.0f, vs[hf][r][g], mid[hf][r][g]);
      }
    // the values' products, group by group: the two halves' weights as B
    // fragments, their sums, then the codes
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      constexpr float lo = -8.0f / k2p24, hi = -128.0f / k2p24;
      uint32_t vb[NB][2][2];
      float ps[NB][4];
      auto weight = [&](int nb, int hf, int r) { return mul2(mul2(sc[nb][hf][r], both(vs[hf][r][g])), inv[nb][g]); };
      auto weigh = [&]() {              // whether a lane's weights pass the bound (or are NaN)
        bool over = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float2 wt = weight(nb, hf, r);
              vb[nb][hf][r] = pack_h2(wt.x, wt.y);
            }
          over = over || past(add_h2(add_h2(vb[nb][0][0], vb[nb][0][1]), add_h2(vb[nb][1][0], vb[nb][1][1])));
        }
        return over;
      };
      if (__any_sync(0xffffffffu, weigh())) {
        // A group whose scale is not finite stands for NaN: it is noted for the queries that see it and leaves the sums.
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (!(fabsf(vs[hf][r][g]) < INFINITY)) {
              vs[hf][r][g] = mid[hf][r][g] = 0.0f;
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if ((seen >> (8 * nb + 4 * hf + 2 * r + e)) & 1u) nans |= 1u << (4 * nb + 2 * e + g);
            }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float2 most = both(0.0f), sum = both(0.0f);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float2 t = mul2(sc[nb][hf][r], both(vs[hf][r][g]));
              most = make_float2(fmaxf(most.x, t.x), fmaxf(most.y, t.y));
              sum = add2(sum, t);
            }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            most.x = fmaxf(most.x, __shfl_xor_sync(0xffffffffu, most.x, o));
            most.y = fmaxf(most.y, __shfl_xor_sync(0xffffffffu, most.y, o));
          }
          // only the queries whose own weights ask for it; a little below the bound, since fp16 sums are rounded
          const uint32_t mine = 0x11111111u << tig;
          const bool ask0 = __ballot_sync(0xffffffffu, sum.x * inv[nb][g].x > 0.9f * kMostW) & mine;
          const bool ask1 = __ballot_sync(0xffffffffu, sum.y * inv[nb][g].y > 0.9f * kMostW) & mine;
          const float2 ni = make_float2(ask0 ? factor_for(most.x) : inv[nb][g].x, ask1 ? factor_for(most.y) : inv[nb][g].y);
          const float fx = ni.x * reciprocal2(inv[nb][g].x), fy = ni.y * reciprocal2(inv[nb][g].y);
          inv[nb][g] = ni;
#pragma unroll
          for (int i = 4 * g; i < 4 * g + 4; ++i) {
            acc[nb][i][0] *= fx;
            acc[nb][i][1] *= fy;
            acc[nb][i][2] *= fx;
            acc[nb][i][3] *= fy;
          }
        }
        weigh();
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            if (split && (NB == 1 ? tig >= 2 : nb == 1)) {
              const float2 wt = weight(nb, hf, r), hi = unpack_h2(vb[nb][hf][r]);
              vb[nb][hf][r] = pack_h2(wt.x - hi.x, wt.y - hi.y);
            }
            cmn[nb][g] = fma2(sc[nb][hf][r], both(mid[hf][r][g]), cmn[nb][g]);
            vb[nb][hf][r] = movmatrix_trans(vb[nb][hf][r]);
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (hf == 0) mma_from(ps[nb], kOnes, kOnes, kOnes, kOnes, vb[nb][0][0], vb[nb][0][1], 0.0f, 0.0f, 0.0f, 0.0f);
          else mma16816(ps[nb], kOnes, kOnes, kOnes, kOnes, vb[nb][1][0], vb[nb][1][1]);
        }
      }
      uint32_t vw[2][4];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          vw[hf][k] = *reinterpret_cast<const uint32_t*>(s + St::kV + piece_at<D>(16 * hf + 4 * k + tig, 2 * g + (gq >> 2)) + 4 * (gq & 3));
#pragma unroll
      for (int ii = 0; ii < 4; ++ii) {
        const uint32_t sel = static_cast<uint32_t>(ii) | (static_cast<uint32_t>(ii + 4) << 8);
        float d[NB][4];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t x01 = __byte_perm(vw[hf][0], vw[hf][1], sel), x89 = __byte_perm(vw[hf][2], vw[hf][3], sel);
          const uint32_t a0 = x01 & kLoNib, a1 = x01 & kHiNib;
          const uint32_t a2 = x89 & kLoNib, a3 = x89 & kHiNib;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            if (hf == 0)
              mma_from(d[nb], a0, a1, a2, a3, vb[nb][0][0], vb[nb][0][1], lo * ps[nb][0], lo * ps[nb][1], hi * ps[nb][0],
                       hi * ps[nb][1]);
            else
              mma16816(d[nb], a0, a1, a2, a3, vb[nb][1][0], vb[nb][1][1]);
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float (&o)[4] = acc[nb][4 * g + ii];
          const float2 u = add2(make_float2(o[0], o[1]), make_float2(d[nb][0], d[nb][1]));
          const float2 v = add2(make_float2(o[2], o[3]), make_float2(d[nb][2], d[nb][3]));
          o[0] = u.x;
          o[1] = u.y;
          o[2] = v.x;
          o[3] = v.y;
        }
      }
    }
  };
  // the item's rows, finished (one share) or as this share's partial
  auto end_item = [&](const uint8_t* s, bool from_start, bool to_end) {
    const int h = reinterpret_cast<const int4*>(s + St::kInfo)->z;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) nans |= __shfl_xor_sync(0xffffffffu, nans, o);
    if (split) {   // the weights' remainders
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][i][e] += NB == 1 ? __shfl_xor_sync(0xffffffffu, acc[0][i][e], 2) : acc[NB - 1][i][e];
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float lsum = e ? l[nb].y : l[nb].x, cm[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) cm[g] = e ? cmn[nb][g].y : cmn[nb][g].x;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          lsum += __shfl_xor_sync(0xffffffffu, lsum, o);
#pragma unroll
          for (int g = 0; g < NG; ++g) cm[g] += __shfl_xor_sync(0xffffffffu, cm[g], o);
        }
        const int n = 8 * nb + 2 * tig + e;
        if (n >= rows) continue;
        const bool whole = from_start && to_end;
        const float f = !whole ? 1.0f : lsum == 0.0f ? 0.0f : 1.0f / lsum;
        float v[NG][8];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          // 2^24 / inv
          const float un = __uint_as_float(min(278u - (__float_as_uint(e ? inv[nb][g].y : inv[nb][g].x) >> 23), 254u) << 23);
          if ((nans >> (4 * nb + 2 * e + g)) & 1u) cm[g] = __uint_as_float(0x7fffffffu);
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) {
            v[g][2 * ii] = fmaf(acc[nb][4 * g + ii][e], un, cm[g]) * f;
            v[g][2 * ii + 1] = fmaf(acc[nb][4 * g + ii][2 + e], 0.0625f * un, cm[g]) * f;
          }
        }
        if (whole) {
          const int t = n / a.shape.group;
          __half* dst = a.out + static_cast<int64_t>(row0 + t) * a.ldo +
                        static_cast<int64_t>(h * a.shape.group + n - t * a.shape.group) * D + 8 * gq;
#pragma unroll
          for (int g = 0; g < NG; ++g)
            *reinterpret_cast<uint4*>(dst + 64 * g) = make_uint4(pack_h2(v[g][0], v[g][1]), pack_h2(v[g][2], v[g][3]),
                                                                pack_h2(v[g][4], v[g][5]), pack_h2(v[g][6], v[g][7]));
        } else {
          const int64_t slot = (static_cast<int64_t>(w) * 2 + (from_start ? 1 : 0)) * pl.rows + n;
          float* dst = pl.part + slot * D + 8 * gq;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            *reinterpret_cast<float4*>(dst + 64 * g) = make_float4(v[g][0], v[g][1], v[g][2], v[g][3]);
            *reinterpret_cast<float4*>(dst + 64 * g + 4) = make_float4(v[g][4], v[g][5], v[g][6], v[g][7]);
          }
          if (gq == 0) pl.stat[slot] = make_float2(m[nb][e] * (e ? kc2[nb].y : kc2[nb].x), lsum);
        }
      }
  };

  // ---- the share ------------------------------------------------------------------
#pragma unroll
  for (int st = 0; st < kStages - 1; ++st) issue(st * St::kBytes);
  int4 rec = make_int4(-1, 0, 0, 0);
  bool fresh = true, from_start = false;
  uint32_t st_rd = (kStages - 1) * St::kBytes, st_cs = 0;
  while (true) {
    issue(st_rd);                         // that stage was read in the round before, which ended in a warp barrier
    st_rd = st_rd == (kStages - 1) * St::kBytes ? 0 : st_rd + St::kBytes;
    tc::cp_async_wait<kStages - 1>();     // this lane's copies of the tile have landed
    __syncwarp();                         // and every lane's
    uint8_t* s = ring + st_cs;
    st_cs = st_cs == (kStages - 1) * St::kBytes ? 0 : st_cs + St::kBytes;
    const int4 info = *reinterpret_cast<const int4*>(s + St::kInfo);
    if (fresh) {
      from_start = info.y & kFirst;
      begin_item(s);
    }
    compute(s, info.x, info.y);
    fresh = info.y & (kLast | kEnd);
    if (fresh) {
      const bool to_end = info.y & kLast;
      end_item(s, from_start, to_end);
      if (from_start && !to_end) {
        const int64_t cost = (pre[info.w + 1] - pre[info.w]) / heads;   // of the item
        rec = make_int4(info.w, info.z, 0, static_cast<int>((pre[info.w] + (info.z + 1) * cost - 1) / per));
      }
    }
    __syncwarp();
    if (info.y & kEnd) break;
  }
  if (lane == 0) pl.rec[w] = rec;
}

template <int D, int NB>
constexpr int step_smem() {
  return kWarps * kStepStages<D, NB> * Stage<D>::kBytes;
}

template <int D, int NB>
fg_status launch(const AttnArgs<__half>& a, const ClassPlan& pl, bool own_plan, cudaStream_t st) {
  constexpr int bytes = step_smem<D, NB>();
  static bool set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (bytes > 48 * 1024 && dev >= 0 && dev < 64 && !set[dev]) {
    if (cudaFuncSetAttribute(step_kernel<D, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
      return check_launch("step_kernel smem attribute");
    set[dev] = true;
  }
  Trace tr(KC_ATTN_PAGED, st);
  return paged::launch("step_kernel", true, step_kernel<D, NB>, static_cast<unsigned>(pl.workers / kWarps), 32 * kWarps, bytes, st, a, pl, own_plan);
}

}  // namespace

int step_workers(int rows, int sms) { return sms * (rows <= 8 ? kCtasPerSm<1> : kCtasPerSm<2>) * kWarps; }

fg_status paged_attention_step(const AttnArgs<__half>& a, const ClassPlan& pl, int head_dim, bool own_plan, cudaStream_t st) {
  if (head_dim == 128) return pl.rows <= 8 ? launch<128, 1>(a, pl, own_plan, st) : launch<128, 2>(a, pl, own_plan, st);
  return pl.rows <= 8 ? launch<64, 1>(a, pl, own_plan, st) : launch<64, 2>(a, pl, own_plan, st);
}

}  // namespace paged
}  // namespace fg
