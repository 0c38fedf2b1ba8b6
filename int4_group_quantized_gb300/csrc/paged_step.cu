// Paged attention of sequences with at most 16 rows per K/V head (decode
// steps; FlexGen notes, "背景知识" decode equations, "5. 近似方法" 4-bit K/V),
// fp16 activations.
//
// The path is bound by the cache's bytes, so every byte is read once for all
// rows of a K/V head (8 rows are one N = 8 block of the warp-level MMA) and
// codes are multiplied as they are:
//   scores   s = sum_g scale_g (q . c)_g + min_g (sum q)_g: lop3 makes a
//            nibble the exact fp16 1024 + c (or 1024 + 16c, against q / 16),
//            and the bias 1024 sum q leaves in fp32;
//   values   o = sum_t (p_t scale_t) (c_t - 8) + sum_t p_t (min_t + 8
//            scale_t): centred, because a bias of 1024 in a sum over thousands
//            of tokens would cost its low bits (the MMA truncates).  The
//            weight p * scale is rounded to fp16 for the MMA after scaling by
//            a power of two near 1 / max scale, so that small activations
//            keep their bits.
// A warp is a worker (see paged_sched.cuh) and walks tiles of 32 tokens of its
// share: its own ring of stages in shared memory, filled by asynchronous
// copies kStages - 1 tiles ahead across items, page numbers another tile
// ahead; no CTA barrier.  Rows of a stage lie so that both the score reads
// (8 bytes of token s(g)) and the value reads (4 bytes of 4 tokens side by
// side) fall on 32 different banks: token row m of an MMA is token s(m) =
// m/2 + 4 (m%2), which makes the transposed weights' token pairs (tig, tig +
// 4), and 16-byte pieces are swizzled by the row.
#include <math.h>

#include <algorithm>

#include "attn_dev.cuh"
#include "paged_attn.cuh"
#include "tc_ptx.cuh"

namespace fg {
namespace paged {
namespace {

using attn::lop_mask_or;
using attn::mma16816;
using attn::pack_h2;
using attn::unpack_h2;
using attn::kHiNib;
using attn::kLoNib;
using attn::kMagic;

constexpr int kTileLog2 = 5;
constexpr int kTile = 1 << kTileLog2;   // tokens of a tile
constexpr int kWarps = 4;               // warps of a CTA
template <int NB>
constexpr int kCtasPerSm = NB == 1 ? 4 : 3;
template <int D, int NB>
constexpr int kStepStages = D == 128 ? (NB == 1 ? 2 : 3) : 4;
constexpr float kGrow = 8.0f;           // log2 growth of a maximum that forces a rescale

template <int D>
struct Stage {
  static constexpr int C = D / 2;                  // code bytes of a row
  static constexpr int NG = D / 64;
  static constexpr int kMeta = kTile * NG * 4;     // one (min or scale) array
  static constexpr int kV = kTile * C, kKs = 2 * kTile * C, kKm = kKs + kMeta, kVs = kKm + kMeta, kVm = kVs + kMeta;
  static constexpr int kInfo = kVm + kMeta;        // which halves are present
  static constexpr int kBytes = kInfo + 16;
};
// Where the 16-byte piece pc of row t lies: pieces swizzled so that rows 0, 4,
// 1, 5 (and 2, 6, 3, 7), and rows 0 .. 3 (and 4 .. 7), use all banks.
template <int D>
__device__ __forceinline__ int piece_at(int t, int pc) {
  if (D == 128) return t * 64 + ((pc ^ ((((t >> 1) ^ (t >> 2)) & 1) << 1)) << 4);
  return (t ^ (((t >> 2) & 1) << 1)) * 32 + (pc << 4);
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
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
constexpr uint32_t kOne2 = 0x3C003C00u, kNeg1032 = 0xE408E408u, kSixteenth2 = 0x2C002C00u, kNeg72 = 0xD480D480u;

// One query row as this lane's B fragments of each 64-group (dims 16 tig ..
// 16 tig + 15 of the group, in the order the code words give them: (0, 4),
// (1, 5) / 16 | (2, 6), (3, 7) / 16), the sum of the fragments' entries (the
// bias's factor) and of the query itself, over this lane's dims.
template <int NG>
struct QFrag {
  uint32_t b[NG][4][2];
  float esum[NG], qsum[NG];
};
template <int NG>
__device__ __forceinline__ void load_q(QFrag<NG>& f, const __half* qrow, int tig) {
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const uint4* src = reinterpret_cast<const uint4*>(qrow + 64 * g + 16 * tig);
    f.esum[g] = f.qsum[g] = 0.0f;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint4 raw = src[w];
      const float2 d01 = unpack_h2(raw.x), d23 = unpack_h2(raw.y), d45 = unpack_h2(raw.z), d67 = unpack_h2(raw.w);
      f.b[g][2 * w][0] = pack_h2(d01.x, d45.x);
      f.b[g][2 * w][1] = pack_h2(d01.y * 0.0625f, d45.y * 0.0625f);
      f.b[g][2 * w + 1][0] = pack_h2(d23.x, d67.x);
      f.b[g][2 * w + 1][1] = pack_h2(d23.y * 0.0625f, d67.y * 0.0625f);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 x = unpack_h2(f.b[g][2 * w + e][0]), y = unpack_h2(f.b[g][2 * w + e][1]);
        f.esum[g] += (x.x + x.y) + (y.x + y.y);
        f.qsum[g] += (x.x + x.y) + 16.0f * (y.x + y.y);
      }
    }
  }
}

// A place in the line of tiles: the item and the tile in it.
struct Cursor {
  int64_t left;          // tiles of the share still to come
  int64_t seq_left;      // tiles of the sequence still to come
  int i, h, x;           // sequence, head, tile of the item
  Seq s;
  Span span;
};

template <int D, int NB>
__global__ void __launch_bounds__(32 * kWarps, kCtasPerSm<NB>) step_kernel(const AttnArgs<__half> a, const ClassPlan pl) {
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
  const int64_t total = pl.head[0], per = pl.head[1];
  const int64_t o0 = w * per;
  if (o0 >= total) {
    if (lane == 0) pl.rec[w] = make_int4(-1, 0, 0, 0);
    return;
  }
  const int heads = a.pool.heads;

  auto enter = [&](Cursor& c) {   // c.i, c.seq_left set: the sequence's shape
    c.s = seq_of(a.tab, a.batch, c.i);
    const int base = c.s.len - c.s.n;
    c.span = span_of<kTileLog2>(base, c.s.len - 1, c.s.keys, a.shape.window, a.shape.sinks);
  };
  Cursor rd;                      // the tile to be copied next
  {
    int lo = 0, hi = a.tab.seqs;     // pre[lo] <= o0 < pre[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pl.pre[mid] <= o0) lo = mid;
      else hi = mid;
    }
    rd.i = lo;
    rd.seq_left = pl.pre[lo + 1] - o0;
    rd.left = total - o0 < per ? total - o0 : per;
    enter(rd);
    const int64_t in = o0 - pl.pre[lo];
    rd.h = static_cast<int>(in / rd.span.n);
    rd.x = static_cast<int>(in - static_cast<int64_t>(rd.h) * rd.span.n);
  }
  auto advance = [&](Cursor& c) {
    --c.left;
    --c.seq_left;
    if (++c.x == c.span.n) {
      c.x = 0;
      ++c.h;
      if (c.seq_left == 0 && c.left > 0) {
        do {
          ++c.i;
          c.seq_left = pl.pre[c.i + 1] - pl.pre[c.i];
        } while (c.seq_left == 0);
        c.h = 0;
        enter(c);
      }
    }
  };
  Cursor cs = rd;                 // the tile to be computed next

  // pages of the two halves of the tile at rd (-1: none, or nothing of it is seen)
  int pg0 = -1, pg1 = -1;
  auto look_up = [&]() {
    if (rd.left <= 0) return;
    const int t0 = rd.span.tile(rd.x) << kTileLog2;
    const int last = rd.s.len - 1 < rd.s.keys - 1 ? rd.s.len - 1 : rd.s.keys - 1;
    const int lo = a.shape.window > 0 ? rd.s.len - rd.s.n - a.shape.window + 1 : 0;
    auto half = [&](int t) {
      if (t > last || (t + 15 < lo && t >= a.shape.sinks)) return -1;
      const int page = page_of(a.tab, rd.i, t);
      if (page < 0 && lane == 0) atomicOr(a.batch.err, DEV_ERR_PAGE);
      return page;
    };
    pg0 = half(t0);
    pg1 = half(t0 + 16);
  };
  // copies the tile at rd into stage st, and moves rd on
  auto issue = [&](int st) {
    if (rd.left > 0) {
      uint8_t* s = ring + st * St::kBytes;
      const int t0 = rd.span.tile(rd.x) << kTileLog2;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int page = hf ? pg1 : pg0;
        if (page >= 0) {
          const int64_t slot = slot_of(a.pool, page, rd.h, t0 + 16 * hf);
          const uint8_t* kc = a.pool.codes[0] + slot * St::C + 16 * lane;
          const uint8_t* vc = a.pool.codes[1] + slot * St::C + 16 * lane;
#pragma unroll
          for (int u = 0; u < D / 64; ++u) {   // 16 rows of C bytes: D / 64 pieces a lane
            const int pc = lane + 32 * u, row = 16 * hf + pc / (St::C / 16), at = piece_at<D>(row, pc % (St::C / 16));
            tc::cp_async16(s + at, kc + 512 * u);
            tc::cp_async16(s + St::kV + at, vc + 512 * u);
          }
          // (min, scale): 16 * NG floats of each array, 4 * NG pieces
          if (lane < 16 * NG) {
            const int arr = lane / (4 * NG), pc = lane % (4 * NG);
            const float* from = arr == 0 ? a.pool.scales[0] : arr == 1 ? a.pool.mins[0] : arr == 2 ? a.pool.scales[1] : a.pool.mins[1];
            tc::cp_async16(s + St::kKs + arr * St::kMeta + hf * (64 * NG) + 16 * pc, from + slot * NG + 4 * pc);
          }
        }
      }
      if (lane == 0) *reinterpret_cast<int*>(s + St::kInfo) = (pg0 >= 0 ? 1 : 0) | (pg1 >= 0 ? 2 : 0);
      advance(rd);
    }
    tc::cp_async_commit();
    look_up();
  };

  // ---- the item's state --------------------------------------------------------
  uint32_t qb[NB][NG][4][2];                     // q as B fragments (query gq of each block of 8)
  float bias[NB][NG][2], qsum[NB][NG][2];        // of queries 2 tig, 2 tig + 1
  float m[NB][2], l[NB][2], cmn[NB][NG][2];
  float acc[NB][NT][4];
  float cap[NG], inv[NG];                        // weights carry the factor inv = 2 / cap
  int rows = 0, pos0 = 0;
  const float kc2 = a.scale_log2;

  int pn[NB][2];                                 // positions of queries 2 tig, 2 tig + 1 (none: below every key)

  auto begin_item = [&]() {
    rows = cs.s.n * a.shape.group;
    pos0 = cs.s.len - cs.s.n;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int n = 8 * nb + gq;
      QFrag<NG> f;
      if (n < rows) {
        const int t = n / a.shape.group;
        load_q<NG>(f, a.q + static_cast<int64_t>(cs.s.row0 + t) * a.ldq +
                          static_cast<int64_t>(cs.h * a.shape.group + n - t * a.shape.group) * D, tig);
      } else {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          f.esum[g] = f.qsum[g] = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) f.b[g][e][0] = f.b[g][e][1] = 0u;
        }
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float b = f.esum[g], s = f.qsum[g];
        b += __shfl_xor_sync(0xffffffffu, b, 1);
        b += __shfl_xor_sync(0xffffffffu, b, 2);
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          bias[nb][g][e] = 1024.0f * __shfl_sync(0xffffffffu, b, 8 * tig + 4 * e);
          qsum[nb][g][e] = __shfl_sync(0xffffffffu, s, 8 * tig + 4 * e);
          cmn[nb][g][e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          qb[nb][g][e][0] = f.b[g][e][0];
          qb[nb][g][e][1] = f.b[g][e][1];
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = 8 * nb + 2 * tig + e;
        pn[nb][e] = k < rows ? pos0 + k / a.shape.group : -(1 << 30);
        m[nb][e] = -INFINITY;
        l[nb][e] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[nb][i][0] = acc[nb][i][1] = acc[nb][i][2] = acc[nb][i][3] = 0.0f;
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) cap[g] = inv[g] = 0.0f;
  };

  auto compute = [&](const uint8_t* s, int tile) {
    const int t0 = tile << kTileLog2;
    const int present = *reinterpret_cast<const int*>(s + St::kInfo);
    const int pl1 = cs.s.len - 1;   // the last row's position
    // every row sees the whole tile: inside all positions, stored, and inside the window or the sinks
    const bool whole = present == 3 && t0 + kTile - 1 <= pos0 && t0 + kTile <= cs.s.keys &&
                       (a.shape.window == 0 || t0 > pl1 - a.shape.window || t0 + kTile <= a.shape.sinks);
    float ks[2][2][NG], vs[2][2][NG], vm[2][2][NG];   // [16-token half][row gq, gq + 8][group]
    float sc[NB][2][2][2];                            // [block][half][row][query]
    const int tok = (gq >> 1) + 4 * (gq & 1);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint2 kw[2][NG];
      float km[2][NG];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 16 * hf + 8 * r + tok;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          kw[r][g] = *reinterpret_cast<const uint2*>(s + piece_at<D>(row, 2 * g + (tig >> 1)) + 8 * (tig & 1));
          ks[hf][r][g] = *reinterpret_cast<const float*>(s + St::kKs + 4 * (row * NG + g));
          km[r][g] = *reinterpret_cast<const float*>(s + St::kKm + 4 * (row * NG + g));
          vs[hf][r][g] = *reinterpret_cast<const float*>(s + St::kVs + 4 * (row * NG + g));
          vm[hf][r][g] = *reinterpret_cast<const float*>(s + St::kVm + 4 * (row * NG + g));
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 2; ++r) sc[nb][hf][r][0] = sc[nb][hf][r][1] = 0.0f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float d[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) d[nb][0] = d[nb][1] = d[nb][2] = d[nb][3] = 0.0f;
#pragma unroll
        for (int ww = 0; ww < 2; ++ww) {
          const uint32_t x0 = ww ? kw[0][g].y : kw[0][g].x, x1 = ww ? kw[1][g].y : kw[1][g].x;
          const uint32_t y0 = x0 >> 8, y1 = x1 >> 8;
          const uint32_t a0 = lop_mask_or(x0, kLoNib, kMagic), a1 = lop_mask_or(x1, kLoNib, kMagic);
          const uint32_t a2 = lop_mask_or(x0, kHiNib, kMagic), a3 = lop_mask_or(x1, kHiNib, kMagic);
          const uint32_t b0 = lop_mask_or(y0, kLoNib, kMagic), b1 = lop_mask_or(y1, kLoNib, kMagic);
          const uint32_t b2 = lop_mask_or(y0, kHiNib, kMagic), b3 = lop_mask_or(y1, kHiNib, kMagic);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma16816(d[nb], a0, a1, a2, a3, qb[nb][g][2 * ww][0], qb[nb][g][2 * ww][1]);
            mma16816(d[nb], b0, b1, b2, b3, qb[nb][g][2 * ww + 1][0], qb[nb][g][2 * ww + 1][1]);
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              sc[nb][hf][r][e] = fmaf(ks[hf][r][g], d[nb][2 * r + e] - bias[nb][g][e],
                                      fmaf(km[r][g], qsum[nb][g][e], sc[nb][hf][r][e]));
      }
    }
    uint32_t seen = 0xffffffffu;   // bit 8 nb + 4 hf + 2 r + e: the query sees the token
    if (!whole) {                  // a row or a token at the edge
      seen = 0;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int j = t0 + 16 * hf + 8 * r + tok;
          const bool here = ((present >> hf) & 1) && j < cs.s.keys;
          bool any = false;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int p = pn[nb][e];
              const bool see = here && j <= p && (a.shape.window == 0 || j > p - a.shape.window || j < a.shape.sinks);
              if (!see) sc[nb][hf][r][e] = -INFINITY;
              seen |= (see ? 1u : 0u) << (8 * nb + 4 * hf + 2 * r + e);
              any |= see;
            }
          // scale and minimum of a token that no query of this lane sees may be anything
          if (!any)
#pragma unroll
            for (int g = 0; g < NG; ++g) vs[hf][r][g] = vm[hf][r][g] = 0.0f;
        }
    }
    // the weights' factor: a power of two that keeps max scale * factor in [1, 2)
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float mx = 0.0f;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (!(vs[hf][r][g] < INFINITY)) vs[hf][r][g] = __uint_as_float(0x7fffffffu);   // such a group is NaN
          mx = fmaxf(mx, vs[hf][r][g]);
        }
      if (__any_sync(0xffffffffu, mx >= cap[g])) {
        const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
        const int e = static_cast<int>(bits >> 23) > 1 ? static_cast<int>(bits >> 23) : 1;   // biased exponent
        const float ncap = e >= 253 ? 1.7e38f : __uint_as_float(static_cast<uint32_t>(e + 1) << 23);
        const float ninv = __uint_as_float(static_cast<uint32_t>(254 - (e >= 253 ? 253 : e)) << 23);
        if (inv[g] != 0.0f) {
          const float f = ninv / inv[g];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 4 * g; i < 4 * g + 4; ++i)
#pragma unroll
              for (int e4 = 0; e4 < 4; ++e4) acc[nb][i][e4] *= f;
        }
        cap[g] = ncap;
        inv[g] = ninv;
      }
    }
    // maxima: of this lane's tokens, then over the lanes of a query
    bool grow = false;
    float nm[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(fmaxf(sc[nb][0][0][e], sc[nb][0][1][e]), fmaxf(sc[nb][1][0][e], sc[nb][1][1][e]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        nm[nb][e] = x;
        grow |= (x - m[nb][e]) * kc2 > kGrow;   // -inf - -inf: no
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float al[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = fmaxf(m[nb][e], nm[nb][e]);
          al[e] = x == -INFINITY ? 1.0f : ex2((m[nb][e] - x) * kc2);
          m[nb][e] = x;
          l[nb][e] *= al[e];
#pragma unroll
          for (int g = 0; g < NG; ++g) cmn[nb][g][e] *= al[e];
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          acc[nb][i][0] *= al[0];
          acc[nb][i][1] *= al[1];
          acc[nb][i][2] *= al[0];
          acc[nb][i][3] *= al[1];
        }
      }
    }
    // weights, and the values' products
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const float mc0 = m[nb][0] == -INFINITY ? 0.0f : m[nb][0] * kc2, mc1 = m[nb][1] == -INFINITY ? 0.0f : m[nb][1] * kc2;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          sc[nb][hf][r][0] = ex2(fmaf(sc[nb][hf][r][0], kc2, -mc0));
          sc[nb][hf][r][1] = ex2(fmaf(sc[nb][hf][r][1], kc2, -mc1));
          l[nb][0] += sc[nb][hf][r][0];
          l[nb][1] += sc[nb][hf][r][1];
        }
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        uint32_t vb[NB][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float f = vs[hf][r][g] * inv[g], mid = fmaf(8.0f, vs[hf][r][g], vm[hf][r][g]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float w0 = sc[nb][hf][r][0] * f, w1 = sc[nb][hf][r][1] * f;
            float c0 = sc[nb][hf][r][0] * mid, c1 = sc[nb][hf][r][1] * mid;
            if (!whole) {   // a NaN group reaches only the queries that see it
              const int bit = 8 * nb + 4 * hf + 2 * r;
              w0 = (seen >> bit) & 1u ? w0 : 0.0f;
              c0 = (seen >> bit) & 1u ? c0 : 0.0f;
              w1 = (seen >> (bit + 1)) & 1u ? w1 : 0.0f;
              c1 = (seen >> (bit + 1)) & 1u ? c1 : 0.0f;
            }
            cmn[nb][g][0] += c0;
            cmn[nb][g][1] += c1;
            vb[nb][r] = movmatrix_trans(pack_h2(w0, w1));
          }
        }
        uint32_t vw[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = 16 * hf + 4 * k + tig;
          vw[k] = *reinterpret_cast<const uint32_t*>(s + St::kV + piece_at<D>(row, 2 * g + (gq >> 2)) + 4 * (gq & 3));
        }
#pragma unroll
        for (int ii = 0; ii < 4; ++ii) {
          const uint32_t sel = static_cast<uint32_t>(ii) | (static_cast<uint32_t>(ii + 4) << 8);
          const uint32_t x01 = __byte_perm(vw[0], vw[1], sel), x89 = __byte_perm(vw[2], vw[3], sel);
          const uint32_t a0 = hfma2(lop_mask_or(x01, kLoNib, kMagic), kOne2, kNeg1032);
          const uint32_t a1 = hfma2(lop_mask_or(x01, kHiNib, kMagic), kSixteenth2, kNeg72);
          const uint32_t a2 = hfma2(lop_mask_or(x89, kLoNib, kMagic), kOne2, kNeg1032);
          const uint32_t a3 = hfma2(lop_mask_or(x89, kHiNib, kMagic), kSixteenth2, kNeg72);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma16816(acc[nb][4 * g + ii], a0, a1, a2, a3, vb[nb][0], vb[nb][1]);
        }
      }
  };
  // the item's rows, finished (one share) or as this share's partial
  auto end_item = [&](bool from_start, bool to_end) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], o);
#pragma unroll
          for (int g = 0; g < NG; ++g) cmn[nb][g][e] += __shfl_xor_sync(0xffffffffu, cmn[nb][g][e], o);
        }
        const int n = 8 * nb + 2 * tig + e;
        if (n >= rows) continue;
        const float lsum = l[nb][e];
        const bool whole = from_start && to_end;
        const float f = !whole ? 1.0f : lsum == 0.0f ? 0.0f : 1.0f / lsum;
        float v[NG][8];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float un = inv[g] != 0.0f ? 1.0f / inv[g] : 0.0f;
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) {
            v[g][2 * ii] = fmaf(acc[nb][4 * g + ii][e], un, cmn[nb][g][e]) * f;
            v[g][2 * ii + 1] = fmaf(acc[nb][4 * g + ii][2 + e], un, cmn[nb][g][e]) * f;
          }
        }
        if (whole) {
          const int t = n / a.shape.group;
          __half* dst = a.out + static_cast<int64_t>(cs.s.row0 + t) * a.ldo +
                        static_cast<int64_t>(cs.h * a.shape.group + n - t * a.shape.group) * D + 8 * gq;
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
          if (gq == 0) pl.stat[slot] = make_float2(m[nb][e] * kc2, lsum);
        }
      }
  };

  // ---- the share ------------------------------------------------------------------
  look_up();
#pragma unroll
  for (int st = 0; st < kStages - 1; ++st) issue(st);
  int4 rec = make_int4(-1, 0, 0, 0);
  bool from_start = cs.x == 0;
  begin_item();
  for (int j = 0; cs.left > 0; ++j) {
    issue((j + kStages - 1) % kStages);   // that stage was read in the round before, which ended in a warp barrier
    tc::cp_async_wait<kStages - 1>();     // this lane's copies of the tile have landed
    __syncwarp();                         // and every lane's
    compute(ring + (j % kStages) * St::kBytes, cs.span.tile(cs.x));
    __syncwarp();
    const bool to_end = cs.x + 1 == cs.span.n;
    if (to_end || cs.left == 1) {
      end_item(from_start, to_end);
      if (from_start && !to_end) {
        const int64_t start = pl.pre[cs.i] + static_cast<int64_t>(cs.h) * cs.span.n;
        rec = make_int4(cs.i, cs.h, 0, static_cast<int>((start + cs.span.n - 1) / per));
      }
      advance(cs);
      if (cs.left > 0) {
        from_start = true;
        begin_item();
      }
    } else {
      advance(cs);
    }
  }
  if (lane == 0) pl.rec[w] = rec;
}

template <int D, int NB>
constexpr int step_smem() {
  return kWarps * kStepStages<D, NB> * Stage<D>::kBytes;
}

template <int D, int NB>
fg_status launch(const AttnArgs<__half>& a, const ClassPlan& pl, cudaStream_t st) {
  constexpr int bytes = step_smem<D, NB>();
  static bool set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (bytes > 48 * 1024 && dev >= 0 && dev < 64 && !set[dev]) {
    if (cudaFuncSetAttribute(step_kernel<D, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
      return check_launch("step_kernel smem attribute");
    set[dev] = true;
  }
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  Trace tr(KC_ATTN_PAGED, st);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pl.workers / kWarps));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, step_kernel<D, NB>, a, pl) != cudaSuccess) return check_launch("step_kernel (launch)");
  return check_launch("step_kernel");
}

}  // namespace

int step_workers(int rows, int sms) { return sms * (rows <= 8 ? kCtasPerSm<1> : kCtasPerSm<2>) * kWarps; }

fg_status paged_attention_step(const AttnArgs<__half>& a, const ClassPlan& pl, int head_dim, cudaStream_t st) {
  if (head_dim == 128) return pl.rows <= 8 ? launch<128, 1>(a, pl, st) : launch<128, 2>(a, pl, st);
  return pl.rows <= 8 ? launch<64, 1>(a, pl, st) : launch<64, 2>(a, pl, st);
}

}  // namespace paged
}  // namespace fg
