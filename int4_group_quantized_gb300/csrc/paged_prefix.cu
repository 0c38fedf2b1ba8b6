// Attention of a group's rows over the prefix that its sequences share, on
// tcgen05 (FlexGen notes, "背景知识" attention; "4. 卸载策略": one read serves every
// sequence of the block; "5. 近似方法" 4-bit K/V), fp16 activations.
//
// A few rows against many keys, so the keys take the MMA's 128 rows and the rows
// its columns, 16 to 64 of them, and the cost falls with them:
//   S^T[key][row] = C q per 64-group, C the codes themselves (a masked nibble is
//     the subnormal fp16 c * 2^-24, exact in the MMA) as the A operand in tensor
//     memory; score = sum_g scale_g (C q)_g + min_g (sum q)_g, by the thread that
//     owns the key, which holds its scales and minima: no rounding of K;
//   O^T[dim][row] += V^T P^T, V and P as two fp16 each, value and remainder. V's
//     128-byte-swizzled rows are the A operand, MN-major; P's remainders lie beside
//     the values as columns N .. 2 N - 1, added when the sums leave. V's remainders
//     at 64 dims are the operand's rows 64 .. 127; at 128 they are operands of their
//     own against P's values. The remainders' product is left out: it is 2^-22 of
//     the whole, as what a remainder rounds away is.
// What is left is the result's rounding (2.1e-4 of its size, as a step by itself; with
// V rounded to fp16, as the chunks' kernel does, 2.7e-4 to 2.9e-4).
//
// One CTA an SM walks its share of the line of tiles (paged_prefix.cuh), 128 keys a
// tile.  Warps 0..7: softmax, a key a thread, half of the rows each group of four
// warps; 8..11: K's codes into tensor memory, a key a thread, a segment's Q, and in
// turn a group of V's last 32 keys; 12..14: V's others; 15: the MMAs.  Two stages of
// everything but Q.  A row's maximum is known to all threads of its half: the segment's
// first tile finds it, a later tile takes it as it is and looks only whether a weight
// has left fp16 (a vote of the half); then the tile finds its maximum, the sums are
// rescaled and the weights formed again.  The normaliser stays with the threads (a
// key's share of every row's) until the segment ends.
//
// Not bound by the bytes (5 to 10% of the memory's rate) nor by the MMAs but by a
// tile's latencies: some 3,700 cycles, of which the 24 MMAs of d 128 take the issuing
// thread most (some 110 each), its waits the rest; the weights of 64 rows take 1,700,
// the vote 300, restoring V longer than that.  A launch has some 15 to 20 us besides
// that no tile accounts for (first fetches and loads, a segment's beginning and end).
// 64 rows over 4,096 tokens, 32 heads of 128: 39 us; ten sequences' 80 rows a head each
// over 12,928 to 31,104, 8 heads of 128: 131 (38 and 114 without V's remainders).
// Measured and not kept without these, for the latter's call, 161 us then: 17 warps at 96 registers 170, 16 softmax warps at 72 193, S two
// tiles ahead 180, three copies of the restoring code 241 (instruction fetches).
//
// Every wait is bounded.  A half of the softmax warps decides everything by a
// reduction over all its warps, so that none is left waiting in a barrier for one
// that gave up.
#include <math.h>

#include "paged_prefix.cuh"
#include "q4_dev.cuh"
#include "tc_ptx.cuh"

namespace fg {
namespace paged {
namespace {

using namespace tc;

constexpr int kKeys = 1 << kPrefixKeysLog2;
constexpr int kSoftWarps = 8, kKeyWarps = 4, kValueWarps = 3;
constexpr int kFirstKey = kSoftWarps, kFirstValue = kFirstKey + kKeyWarps, kMmaWarp = kFirstValue + kValueWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);
static_assert(kPrefixRows == 64 && kThreads == 512 && kFirstKey % 4 == 0 && kFirstValue % 4 == 0, "the layout below");
constexpr float kLift = 4.0f;          // a row's largest weight is 2^4 or more when its maximum is found (paged_tile.cu)
constexpr uint32_t kMostHalf = 0x7800u;   // 2^15 as fp16: weights up to it stand

template <int D>
struct Smem {
  static constexpr int kPanel = kKeys * 128;            // 128 rows of 128 bytes
  static constexpr int kV = (D == 128 ? 4 : 2) * kPanel;   // values, then remainders
  static constexpr int kLow = D / 64 * kPanel;          // where the remainders begin
  static constexpr int kP = 2 * kPanel;                 // 2 N <= 128 columns
  static constexpr int kQPanel = kPrefixRows * 128;
  static constexpr int kQ = D / 64 * kQPanel;
  static constexpr int kSums = kPrefixRows * 8;         // (sum q of group 0, 1) of two rows side by side
  static constexpr int kMeta = kKeys * 16;              // K's scales and minima in units of the exponent
  static constexpr int kTurn = D == 128 ? 0 : kPrefixRows * 64 * 4;   // D = 64: a segment's sums of V's remainders, [row][64]
  // one Q (a second would leave no room for V's remainders)
  static constexpr int kBytes = 1024 + 2 * (kV + kP + kMeta) + kQ + kTurn + 2 * kSums + 4 * kPrefixRows * 2 + 4 * kPrefixRows * 4 + 256;
};

// A share's walk over its segments: parts of one unit's key tiles.
struct Walk {
  int64_t left;
  int g, h, u, x, x1;
  ClassRows s;
  PrefixGroup at;
};
__device__ __forceinline__ void walk_begin(Walk& k, const PrefixArgs& p, const PrefixLine& line) {
  const int64_t o0 = blockIdx.x * line.per;
  k.left = 0;
  if (o0 >= line.total) return;
  k.left = line.per < line.total - o0 ? line.per : line.total - o0;
  k.g = line.g;
  k.at = line.at;
  k.s = class_rows(p.a.prefix, p.a.tab, p.a.batch, k.g, false);
  const int64_t in = o0 - k.at.base, unit = in / k.at.tiles;
  k.h = static_cast<int>(unit / k.at.units);
  k.u = static_cast<int>(unit - static_cast<int64_t>(k.h) * k.at.units);
  k.x = static_cast<int>(in - unit * k.at.tiles);
  k.x1 = static_cast<int>(k.left < k.at.tiles - k.x ? k.x + k.left : k.at.tiles);
}
__device__ __forceinline__ void walk_next(Walk& k, const PrefixArgs& p) {
  k.left -= k.x1 - k.x;
  if (k.left == 0) return;
  if (++k.u == k.at.units) {
    k.u = 0;
    if (++k.h == p.a.pool.heads) {
      k.h = 0;
      do k.s = class_rows(p.a.prefix, p.a.tab, p.a.batch, ++k.g, false);
      while (k.s.list == 0);
      k.at = prefix_group(k.s, p.a.shape.group, false);
    }
  }
  k.x = 0;
  k.x1 = static_cast<int>(k.left < k.at.tiles ? k.left : k.at.tiles);
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5};\n"
      "add.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 halves(uint32_t h) {   // fp16x2 in fp32
  float2 r;
  asm("{ .reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b; }" : "=f"(r.x), "=f"(r.y) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t mbar_test(uint64_t* bar, uint32_t parity) {   // without waiting
  uint32_t over;
  asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(over)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return over;
}
__device__ __forceinline__ uint32_t max_h2(uint32_t a, uint32_t b) {   // NaN if either is
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// 8 consecutive columns of a warp's 32 lanes (arrived() before they are read), and back.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void arrived(uint32_t (&a)[8], uint32_t (&b)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]), "+r"(b[0]), "+r"(b[1]),
                 "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7])
               :
               : "memory");
}
// Of eight values of every lane: lane i's (i < 8) is the sum or the maximum of value i over the lanes, in one order.
template <bool MAX>
__device__ __forceinline__ float fold8(float (&v)[8]) {
  const int lane = threadIdx.x & 31;
  auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int o = 4; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      v[i] = join(up ? v[i + o] : v[i], __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + o], o));
    }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) v[0] = join(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  return v[0];
}
// Named barrier over a half's 128 threads; true where any of them says so.
__device__ __forceinline__ bool bar_any(int id, bool pred) {
  uint32_t r;
  asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %2, 0; barrier.cta.red.or.pred q, %1, 128, p; selp.u32 %0, 1, 0, q; }"
               : "=r"(r)
               : "r"(id), "r"(pred ? 1u : 0u)
               : "memory");
  return r != 0;
}
// MMAs with A in tensor memory, and with both operands in shared memory; descriptors as a low word and a high one.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, bool acc) {
  asm volatile(
      "{ .reg .pred p; .reg .b64 y; setp.ne.b32 p, %5, 0; mov.b64 y, {%2, %3};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p; }" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, bool acc) {
  asm volatile(
      "{ .reg .pred p; .reg .b64 x, y; setp.ne.b32 p, %6, 0; mov.b64 x, {%1, %2}; mov.b64 y, {%3, %4};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p; }" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
// 32 codes of a group through fmaf(q, scale, min) into row r of two swizzled panels, `low` bytes apart, from the row's 16-byte
// piece c0 on: the value cut to fp16's 11 bits, and what that leaves (below fp16's normal numbers, in steps of 2^-24).  Every 8
// dims in the order (0, 4), (1, 5), (2, 6), (3, 7).  Two pieces a round, and a round for each half of a group, as instruction
// fetches are what it costs (ten sequences each over 12,928 to 31,104 tokens, the call: 167 us; four pieces 172; rounding
// and converting back in place of cutting 177 and 182, and 220 with no loop at all).
__device__ __forceinline__ void restore_half(const uint4& code, float scale, float mn, uint8_t* prow, int low, int r, int c0) {
  const float2 lo2 = both(scale * 16777216.0f), hi2 = both(scale * 1048576.0f), m2 = both(mn);
  uint32_t w0 = code.x, w1 = code.y;
#pragma unroll 1
  for (int c = 0; c < 4; c += 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t x = i ? w1 : w0, y = x >> 8;
      const float2 v[4] = {q4::fma_f32x2(halves(x & 0x000F000Fu), lo2, m2), q4::fma_f32x2(halves(x & 0x00F000F0u), hi2, m2),
                           q4::fma_f32x2(halves(y & 0x000F000Fu), lo2, m2), q4::fma_f32x2(halves(y & 0x00F000F0u), hi2, m2)};
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 cut = make_float2(__uint_as_float(__float_as_uint(v[e].x) & 0xffffe000u), __uint_as_float(__float_as_uint(v[e].y) & 0xffffe000u));
        hi[e] = q4::cvt_f16x2(cut);
        lo[e] = q4::cvt_f16x2(q4::fma_f32x2(cut, both(-1.0f), v[e]));
      }
      uint8_t* const to = prow + (((c0 + c + i) ^ (r & 7)) << 4);
      *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(to + low) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    w0 = code.z;
    w1 = code.w;
  }
}
template <int NG>
__device__ __forceinline__ void load_meta(float (&v)[NG], const float* base, uint64_t at) {
  const char* p = reinterpret_cast<const char*>(base) + at;
  if (NG == 2) {
    const float2 x = *reinterpret_cast<const float2*>(p);
    v[0] = x.x;
    v[NG - 1] = x.y;
  } else {
    v[0] = *reinterpret_cast<const float*>(p);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const PrefixArgs p, uint32_t wait_limit) {
  using S = Smem<D>;
  constexpr int NG = D / 64;
  constexpr uint32_t kScore = 0, kOut = 256, kCodes = 384, kTmemCols = 512;   // two stages of two groups' 64, 128, two of 64
  constexpr uint32_t kDescHi = static_cast<uint32_t>((uint64_t(1) << 14) | (uint64_t(2) << 29) | (1024 >> 4));   // of smem_desc_sw128
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const sV = sm;
  uint8_t* const sP = sV + 2 * S::kV;
  uint8_t* const sQ = sP + 2 * S::kP;
  float* const sTurn = reinterpret_cast<float*>(sQ + S::kQ);
  float4* const sMeta = reinterpret_cast<float4*>(sQ + S::kQ + S::kTurn);         // [stage][key] (scale, scale of group 1, minimum, minimum)
  float* const sSum = reinterpret_cast<float*>(sMeta + 2 * kKeys);         // [segment % 2][row / 2][group][row % 2]
  float* const sNeg = sSum + 2 * S::kSums / 4;                             // [row] minus the maximum
  float* const sShrink = sNeg + kPrefixRows;                               // [row] what a new maximum makes of sums
  float* const sNorm = sShrink + kPrefixRows;                              // [quarter][row] maxima, and normalisers in the end
  uint64_t* const bars = reinterpret_cast<uint64_t*>(sNorm + 4 * kPrefixRows);
  uint64_t* const kfull = bars;        // [stage] K's codes of the tile are in tensor memory
  uint64_t* const sfull = bars + 2;    // [stage] S^T of the tile is, K's place is free, and P V of the tile two before has completed
  uint64_t* const vfull = bars + 6;    // [stage] V of the tile is in shared memory
  uint64_t* const pfull = bars + 8;    // [stage] P is, and S^T and the rows' sums have been read
  uint64_t* const pvdone = bars + 10;  // [stage] P V of the tile has completed
  uint64_t* const qfull = bars + 12;   // [segment % 2] Q of the segment is in shared memory, and its sums
  uint64_t* const drained = bars + 14; // O of the segment has been read
  uint64_t* const done = bars + 15;    // every MMA has completed
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(bars + 16);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* const sHere = tmem_slot + 2;                                   // [stage][quarter] keys of the tile that are there
  __shared__ PrefixLine line;

  const AttnArgs<__half>& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kfull[i], kKeyWarps);
      mbar_init(&sfull[i], 2);   // the commit, and the issuer itself: it has seen K's barrier and Q's, and so the scales and sums
      mbar_init(&vfull[i], kValueWarps + NG);
      mbar_init(&pfull[i], kSoftWarps);
      mbar_init(&pvdone[i], 1);
      mbar_init(&qfull[i], kKeyWarps);
    }
    mbar_init(drained, kSoftWarps);
    mbar_init(done, 1);
    *abort_flag = 0;
    line.alone[0] = line.alone[1] = 0;
    mbar_fence_init();
  }
  griddep_launch();
  griddep_wait();
  __syncthreads();
  if (p.tile.workers > 0) planned_line(p, line);
  else prefix_line<false>(p, line, [&](int groups, int i, int& n, int& tall) { return tall = 0, shared_tokens(a, groups, i, n); });
  if (line.total == 0) return;   // a call that does not share: no tensor memory is taken
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk k = {};
  walk_begin(k, p, line);

  if (warp >= kFirstKey && warp < kMmaWarp) {
    // ---- K's codes and V, a key a lane: warps 8 .. 11 a quarter of every tile's K each, 12 .. 14 quarters 0 .. 2 of V; V's last
    // quarter, group by group, is the K warps' in turn, which have time for it.
    const bool value = warp >= kFirstValue;
    const int quarter = warp & 3, r = 32 * quarter + lane;   // (of 12 .. 14 the same)
    const int tiles = static_cast<int>(k.left);
    const int psl = a.pool.ps_log2, psm = (1 << psl) - 1;
    const uint32_t page_codes = static_cast<uint32_t>(a.pool.heads) * (D / 2) << psl;   // bytes of a page in a codes array
    const uint32_t page_meta = static_cast<uint32_t>(a.pool.heads) * (4 * NG) << psl;   // and in a (min or scale) array
    const uint8_t* const codes = value ? a.pool.codes[1] : a.pool.codes[0];
    const float* const scales = value ? a.pool.scales[1] : a.pool.scales[0];
    const float* const mins = value ? a.pool.mins[1] : a.pool.mins[0];
    // a key as it is stored; its row in a page (-1: no key of the prefix), and the table's entry: looked up a tile before it
    // is loaded, loaded a tile before it is used.  x...: the same of a K warp's group of V
    uint4 code[2 * NG], xcode[2];
    float scale[NG], mn[NG], xscale = 0.0f, xmn = 0.0f;
    bool there = false;
    Walk w = k;              // of the tile that is looked up next
    const int32_t* row = a.tab.table + w.s.leader * a.tab.stride;
    int wx = k.x, seen = 0, loaded = 0, page = -1, off = -1, xpage = -1, xoff = -1;
    auto extra = [&](int tile) { return !value && (NG == 2 ? (tile & 1) == (quarter >> 1) : (tile & 3) == quarter); };
    const int xg = NG == 2 ? quarter & 1 : 0;
    auto look_up = [&]() {
      off = xoff = -1;
      if (seen == tiles) return;
      const int t0 = wx << kPrefixKeysLog2, j = t0 + r, xj = t0 + 96 + lane;
      if (j < w.s.tokens) {
        page = row[j >> psl];
        off = (w.h << psl) + (j & psm);
      }
      if (extra(seen) && xj < w.s.tokens) {
        xpage = row[xj >> psl];
        xoff = (w.h << psl) + (xj & psm);
      }
      ++seen;
      if (++wx == w.x1) {
        walk_next(w, p);
        wx = w.x;
        row = a.tab.table + w.s.leader * a.tab.stride;
      }
    };
    auto is_page = [&](int e) { return static_cast<uint32_t>(e) < static_cast<uint32_t>(a.tab.pages); };
    auto load = [&]() {
      asm volatile("" : "+r"(page), "+r"(xpage));   // the entries are waited for here and not where they were asked for
      there = off >= 0 && is_page(page);
#pragma unroll
      for (int e = 0; e < 2 * NG; ++e) code[e] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int g = 0; g < NG; ++g) scale[g] = mn[g] = 0.0f;
      if (there) {
        const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(page)) * page_codes + static_cast<uint32_t>(off) * (D / 2);
        const uint64_t am = static_cast<uint64_t>(static_cast<uint32_t>(page)) * page_meta + static_cast<uint32_t>(off) * (4 * NG);
        const uint4* c = reinterpret_cast<const uint4*>(codes + at);
#pragma unroll
        for (int e = 0; e < 2 * NG; ++e) code[e] = c[e];
        load_meta(scale, scales, am);
        load_meta(mn, mins, am);
      } else if (off >= 0 && !value) {
        atomicOr(a.batch.err, DEV_ERR_PAGE);
      }
      if (extra(loaded)) {
        xcode[0] = xcode[1] = make_uint4(0u, 0u, 0u, 0u);
        xscale = xmn = 0.0f;
        if (xoff >= 0 && is_page(xpage)) {
          const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(xpage)) * page_codes + static_cast<uint32_t>(xoff) * (D / 2);
          const uint64_t am = static_cast<uint64_t>(static_cast<uint32_t>(xpage)) * page_meta + static_cast<uint32_t>(xoff) * (4 * NG);
          const uint4* c = reinterpret_cast<const uint4*>(a.pool.codes[1] + at) + 2 * xg;
          xcode[0] = c[0];
          xcode[1] = c[1];
          xscale = reinterpret_cast<const float*>(reinterpret_cast<const char*>(a.pool.scales[1]) + am)[xg];
          xmn = reinterpret_cast<const float*>(reinterpret_cast<const char*>(a.pool.mins[1]) + am)[xg];
        }
      }
      ++loaded;
    };
    // a group whose scale is not finite is NaN for all rows: they all see the key
    auto finite = [](float f) { return fabsf(f) < INFINITY ? f : __uint_as_float(0x7fffffffu); };
    look_up();
    load();
    look_up();
    bool ok = true;
    int seg = 0, x = k.x;
    for (int n = 0; n < tiles; ++n) {
      if (value) {
        ok = n < 2 || mbar_wait(&pvdone[n & 1], ((n >> 1) - 1) & 1, wait_limit, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t* const to = sV + (n & 1) * S::kV + r * 128;
#pragma unroll 1
        for (int e = 0; e < 2 * NG; ++e) {
          const int g = e >> 1;
          restore_half(code[0], finite(g ? scale[NG - 1] : scale[0]), g ? mn[NG - 1] : mn[0], to + g * S::kPanel, S::kLow, r, 4 * (e & 1));
#pragma unroll
          for (int i = 0; i + 1 < 2 * NG; ++i) code[i] = code[i + 1];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&vfull[n & 1]);
        load();      // behind the fence, which would wait for it
        look_up();
        continue;
      }
      // P of the tile two before is there: S has read its codes, the softmax its scales (and the sums of the segment two
      // before, whose place a new segment's take: its last tile is no later).  A new segment's Q waits for S of the tile before.
      ok = n < 2 || mbar_wait(&pfull[n & 1], ((n >> 1) - 1) & 1, wait_limit, abort_flag);
      if (ok && x == k.x && n > 0) ok = mbar_wait(&sfull[(n - 1) & 1], ((n - 1) >> 1) & 1, wait_limit, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (x == k.x) {
        uint8_t* const q = sQ;
        float* const sum = sSum + (seg & 1) * (S::kSums / 4);
        constexpr int kPieces = D / 8;                    // 16 bytes each, a lane a piece
        const int pc = lane % kPieces, all = k.s.list * a.shape.group, r0 = k.u * k.at.rows;
        for (int m = quarter * (32 / kPieces) + lane / kPieces; m < k.at.rows; m += kKeyWarps * (32 / kPieces)) {
          const int row = r0 + m, lx = row / a.shape.group;
          const bool on = row < all;
          const __half* from = a.q + static_cast<int64_t>(on ? listed_row(a.prefix, a.batch, place_of(a.prefix, k.s, k.s.first + lx)) : 0) * a.ldq +
                               static_cast<int64_t>(k.h * a.shape.group + (on ? row - lx * a.shape.group : 0)) * D + 8 * pc;
          const uint4 u = on ? *reinterpret_cast<const uint4*>(from) : make_uint4(0u, 0u, 0u, 0u);
          // every 8 dims in the codes' order
          *reinterpret_cast<uint4*>(q + (pc >> 3) * S::kQPanel + m * 128 + (((pc & 7) ^ (m & 7)) << 4)) =
              make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410), __byte_perm(u.y, u.w, 0x7632));
          const float2 f0 = halves(u.x), f1 = halves(u.y), f2 = halves(u.z), f3 = halves(u.w);
          float s = ((f0.x + f0.y) + (f1.x + f1.y)) + ((f2.x + f2.y) + (f3.x + f3.y));
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);   // rows are a multiple of 16: every lane comes as often
          if ((pc & 7) == 0) sum[(m >> 1) * 4 + (pc >> 3) * 2 + (m & 1)] = s;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&qfull[seg & 1]);
      }
      tc_fence_after();
      const uint32_t to = tmem + kCodes + 64 * (n & 1) + (static_cast<uint32_t>(32 * quarter) << 16);
#pragma unroll
      for (int e = 0; e < 2 * NG; ++e) {
        uint32_t o[16];
        const uint32_t c4[4] = {code[e].x, code[e].y, code[e].z, code[e].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          o[4 * c] = c4[c] & 0x000F000Fu;
          o[4 * c + 1] = (c4[c] >> 4) & 0x000F000Fu;
          o[4 * c + 2] = (c4[c] >> 8) & 0x000F000Fu;
          o[4 * c + 3] = (c4[c] >> 12) & 0x000F000Fu;
        }
        tmem_st_32x32b_x16(to + 16 * e, o);
      }
      // a code in the MMA is c * 2^-24; a scale that is not finite makes the key's scores NaN
      const float unit = a.scale_log2 * 16777216.0f;
      sMeta[(n & 1) * kKeys + r] = make_float4(finite(scale[0]) * unit, finite(scale[NG - 1]) * unit, mn[0] * a.scale_log2, mn[NG - 1] * a.scale_log2);
      const uint32_t here = __ballot_sync(0xffffffffu, there);
      if (lane == 0) sHere[4 * (n & 1) + quarter] = here;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&kfull[n & 1]);
      if (extra(n)) {
        ok = n < 2 || mbar_wait(&pvdone[n & 1], ((n >> 1) - 1) & 1, wait_limit, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t* const vto = sV + (n & 1) * S::kV + xg * S::kPanel + (96 + lane) * 128;
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
          restore_half(xcode[0], finite(xscale), xmn, vto, S::kLow, lane, 4 * e);   // (row 96 + lane: the same swizzle)
          xcode[0] = xcode[1];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&vfull[n & 1]);
      }
      load();      // behind the arrivals, which would wait for it
      look_up();
      if (++x == k.x1) {
        ++seg;
        walk_next(k, p);
        x = k.x;
      }
    }
  } else if (warp == kMmaWarp) {
    // ---- MMA issuer --------------------------------------------------------------------
    if (lane == 0) {
      const uint32_t q_lo = static_cast<uint32_t>(smem_desc_sw128(smem_u32(sQ), 16, 1024));
      const uint32_t v_lo = static_cast<uint32_t>(smem_desc_sw128(smem_u32(sV), S::kPanel, 1024));
      const uint32_t p_lo = static_cast<uint32_t>(smem_desc_sw128(smem_u32(sP), S::kPanel, 1024));
      int n = 0, seg = 0;
      bool ok = true, pending = false;
      auto wait = [&](uint64_t* bar, int phase) {
        if (ok) ok = mbar_wait(bar, phase & 1, wait_limit, abort_flag);
        return ok;
      };
      // A wait takes some 250 cycles even where it is over, and a batch of MMAs 600 to issue: so barriers are looked at before
      // a batch is issued, and waited for after it only where they were not over yet.
      auto look = [&](uint64_t* bar, int phase) { return mbar_test(bar, phase & 1); };
      uint32_t k_in = 0;
      // P V of tile g; first: of its segment, whose number is `of` and whose unit has `rows` rows
      auto issue_o = [&](int g, bool first, int of, int rows, uint32_t v_in, uint32_t p_in) {
        if (first && of > 0 && !wait(drained, of - 1)) return;
        if (!v_in && !wait(&vfull[g & 1], g >> 1)) return;
        if (!p_in && !wait(&pfull[g & 1], g >> 1)) return;
        tc_fence_after();
        const uint32_t idesc = idesc_f16(128, 0, 1, 1) + (static_cast<uint32_t>(rows >> 2) << 17);   // 2 rows columns
        const uint32_t idesc_low = idesc_f16(128, 0, 1, 1) + (static_cast<uint32_t>(rows >> 3) << 17);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk) {
          if (kk == kKeys / 16 - 2) k_in = look(&kfull[g & 1], (g + 2) >> 1);   // of tile g + 2, late in the batch
          const uint32_t weights = p_lo + (g & 1) * (S::kP >> 4) + kk * (2048 >> 4);
          const uint32_t values = v_lo + (g & 1) * (S::kV >> 4) + kk * (2048 >> 4);
          mma_ss(tmem + kOut, values, kDescHi, weights, kDescHi, idesc, !first || kk > 0);
          if (D == 128) mma_ss(tmem + kOut, values + (S::kLow >> 4), kDescHi, weights, kDescHi, idesc_low, true);
        }
        mma_commit(&pvdone[g & 1]);
      };
      bool first = false;   // of the tile before this one
      int of = 0, rows = 16;
      while (k.left > 0 && ok) {
        const uint32_t idesc = idesc_f16(128, 0, 0, 0) + (static_cast<uint32_t>(k.at.rows >> 3) << 17);
        if (!wait(&qfull[seg & 1], seg >> 1)) break;
        for (int x = k.x; x < k.x1; ++x, ++n) {
          // S's place is free: P of the tile two before was waited for
          if (!k_in && !wait(&kfull[n & 1], n >> 1)) break;
          tc_fence_after();
          const uint32_t v_in = pending ? look(&vfull[(n - 1) & 1], (n - 1) >> 1) : 0u, p_in = pending ? look(&pfull[(n - 1) & 1], (n - 1) >> 1) : 0u;
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts(tmem + kScore + 128 * (n & 1) + 64 * g, tmem + kCodes + 64 * (n & 1) + 32 * g + 8 * kk,
                     q_lo + ((g * S::kQPanel + 32 * kk) >> 4), kDescHi, idesc, kk > 0);
          mbar_arrive(&sfull[n & 1]);
          mma_commit(&sfull[n & 1]);
          k_in = 0;
          if (pending) issue_o(n - 1, first, of, rows, v_in, p_in);
          if (!ok) break;
          pending = true;
          first = x == k.x;
          of = seg;
          rows = k.at.rows;
        }
        ++seg;
        walk_next(k, p);
      }
      if (ok && pending) issue_o(n - 1, first, of, rows, 0u, 0u);
      mma_commit(done);
    }
    __syncwarp();
  } else {
    // ---- softmax: key r of the tile, rows 8 c of the half ---------------------------------------
    const int half = warp >> 2, quarter = warp & 3, r = 32 * quarter + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    const int bar = 1 + half;
    int n = 0, seg = 0;
    bool ok = true;
    while (k.left > 0) {
      const int rows = k.at.rows / 2, chunks = rows / 8, first = half * rows;   // of this half
      const float* const sum = sSum + (seg & 1) * (S::kSums / 4) + first * 2;
      float2 l[16];        // the normaliser's part of this key and those 128 after it, of two rows each
#pragma unroll
      for (int i = 0; i < 16; ++i) l[i] = both(0.0f);
      bool gave_up = false;
      for (int x = k.x; x < k.x1; ++x, ++n) {
        const int st = n & 1;
        const uint32_t ts = tmem + kScore + 128 * st + lanes + first;
        ok = mbar_wait(&sfull[st], (n >> 1) & 1, wait_limit, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        const float4 meta = sMeta[st * kKeys + r];
        const float2 s2[2] = {both(meta.x), both(meta.y)}, m2[2] = {both(meta.z), both(meta.w)};
        const bool on = (sHere[4 * st + quarter] >> lane) & 1u;
        // scores of rows 8 c .. 8 c + 7 of the half, on top of from(row)
        auto fetch = [&](int c, uint32_t (&u)[8], uint32_t (&v)[8]) {
          tmem_ld8(ts + 8 * c, u);
          if (NG == 2) tmem_ld8(ts + 64 + 8 * c, v);
        };
        auto scores_of = [&](int c, const uint32_t (&u)[8], const uint32_t (&v)[8], float2 (&z)[4], auto from) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 q = *reinterpret_cast<const float4*>(sum + 4 * (4 * c + e));
            float2 t = q4::fma_f32x2(m2[0], make_float2(q.x, q.y), from(8 * c + 2 * e));
            if (NG == 2) t = q4::fma_f32x2(m2[1], make_float2(q.z, q.w), t);
            t = q4::fma_f32x2(s2[0], make_float2(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1])), t);
            if (NG == 2) t = q4::fma_f32x2(s2[1], make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), t);
            z[e] = t;
          }
        };
        auto scores = [&](int c, float2 (&z)[4], auto from) {
          uint32_t u[8], v[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
          fetch(c, u, v);
          arrived(u, v);
          scores_of(c, u, v, z, from);
        };
        auto below = [&](int i) {   // minus the maximum of rows i, i + 1 of the half; a key that is not there weighs nothing
          const float2 m = *reinterpret_cast<const float2*>(sNeg + first + i);
          return on ? m : both(-INFINITY);
        };
        // the tile's largest score of every row of the half: a row's 32 keys of the warp to one lane, the four warps through
        // sNorm (a barrier after it)
        auto find = [&]() {
          if (ok)
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
              float2 z[4];
              scores(c, z, [](int) { return both(0.0f); });
              float v[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[2 * e] = on ? fmaxf(z[e].x, -INFINITY) : -INFINITY;    // a NaN is no maximum
                v[2 * e + 1] = on ? fmaxf(z[e].y, -INFINITY) : -INFINITY;
              }
              const float top = fold8<true>(v);
              if (lane < 8) sNorm[quarter * kPrefixRows + first + 8 * c + lane] = top;
            }
          bar_any(bar, false);
        };
        auto top_of = [&](int i) {
          const float* const c = sNorm + first + i;
          return fmaxf(fmaxf(c[0], c[kPrefixRows]), fmaxf(c[2 * kPrefixRows], c[3 * kPrefixRows]));
        };
        // A row without a maximum has minus infinity's: +infinity, which takes the weights of any key that is there out of
        // fp16, so that a tile that has one finds it.
        if (x == k.x) {
          find();
          if (quarter == 0 && lane < rows) {
            const float top = top_of(lane);
            sNeg[first + lane] = top == -INFINITY ? INFINITY : kLift - top;
          }
          bar_any(bar, false);
        }
        uint8_t* const sp = sP + st * S::kP + r * 128;
        const int lo_chunk = k.at.rows / 8;
        uint32_t most = 0u;   // of the weights, as fp16 pairs
        auto weigh = [&]() {
          most = 0u;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c < chunks) {
              float2 z[4];
              scores(c, z, below);
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 w = make_float2(ex2_approx(z[e].x), ex2_approx(z[e].y));
                l[4 * c + e] = add_f32x2(l[4 * c + e], w);
                hi[e] = q4::cvt_f16x2(w);
                lo[e] = q4::cvt_f16x2(q4::fma_f32x2(halves(hi[e]), both(-1.0f), w));
                most = max_h2(most, hi[e]);
              }
              const int ch = half * chunks + c, cl = lo_chunk + ch;
              *reinterpret_cast<uint4*>(sp + (ch >> 3) * S::kPanel + (((ch & 7) ^ (r & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              *reinterpret_cast<uint4*>(sp + (cl >> 3) * S::kPanel + (((cl & 7) ^ (r & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
          }
        };
        if (ok) weigh();
        const bool past = (most & 0xffffu) > kMostHalf || (most >> 16) > kMostHalf;   // NaN too
        if (bar_any(bar, past || !ok)) {
          // The weights leave the normaliser again (of one that was huge nothing else is left: its row's sums are about to
          // shrink by as much), the tile's maxima are found, sums and normaliser follow those of the rows that ask.
          if (ok)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (c < chunks) {
                float2 z[4];
                scores(c, z, below);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float w0 = ex2_approx(z[e].x), w1 = ex2_approx(z[e].y);
                  float2& n2 = l[4 * c + e];
                  n2 = make_float2(w0 < 0x1p60f ? n2.x - w0 : w0 == w0 ? 0.0f : n2.x, w1 < 0x1p60f ? n2.y - w1 : w1 == w1 ? 0.0f : n2.y);
                }
              }
          find();
          if (quarter == 0 && lane < rows) {
            const float top = top_of(lane), old = sNeg[first + lane];
            const bool ask = top + old > 15.0f;
            const float neg = ask ? kLift - top : old;
            sNeg[first + lane] = neg;
            sShrink[first + lane] = !ask ? 1.0f : old == INFINITY ? 0.0f : ex2_approx(neg - old);
          }
          bar_any(bar, false);
          const float* const shrink = sShrink + first;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (2 * i < rows) l[i] = make_float2(l[i].x * shrink[2 * i], l[i].y * shrink[2 * i + 1]);
          if (ok && x > k.x) {   // the segment's sums so far
            ok = mbar_wait(&pvdone[st ^ 1], ((n - 1) >> 1) & 1, wait_limit, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            if (ok)
#pragma unroll 1
              for (int c = 0; c < 2 * chunks; ++c) {   // values, then remainders
                const int row = 8 * (c % chunks);
                const uint32_t to = tmem + kOut + lanes + (c < chunks ? 0 : k.at.rows) + first + row;
                uint32_t u[8], none[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
                tmem_ld8(to, u);
                arrived(u, none);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * shrink[row + e]);
                tmem_st8(to, u);
              }
            tmem_st_wait();
          }
          if (ok) weigh();
          if (bar_any(bar, !ok)) {
            gave_up = true;
            break;
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&pfull[st]);
        }
      }
      if (gave_up) break;
      // ---- the segment's rows: their parts ------------------------------------------------
      ok = mbar_wait(&pvdone[(n - 1) & 1], ((n - 1) >> 1) & 1, wait_limit, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 4; ++c)   // the normaliser: a row's 32 keys of the warp to one lane, the four warps in order
        if (c < chunks) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[2 * e] = l[4 * c + e].x;
            v[2 * e + 1] = l[4 * c + e].y;
          }
          const float all = fold8<false>(v);
          if (lane < 8) sNorm[quarter * kPrefixRows + first + 8 * c + lane] = all;
        }
      if (bar_any(bar, !ok)) break;
      // where row `first` + lane of the unit goes
      const int row = k.u * k.at.rows + first + lane;
      const bool real = lane < rows && row < k.s.list * a.shape.group, home = k.x == 0;
      const int lx = real ? row / a.shape.group : 0;
      const int64_t place = home ? static_cast<int64_t>(place_of(a.prefix, k.s, k.s.first + lx)) * a.q_heads + k.h * a.shape.group + (real ? row - lx * a.shape.group : 0)
                                 : static_cast<int64_t>(blockIdx.x) * kPrefixRows + first + lane;
      if (quarter == 0 && real) {
        const float* const c = sNorm + first + lane;
        (home ? a.prefix.home_stat : a.prefix.extra_stat)[place] =
            make_float2(-sNeg[first + lane], (c[0] + c[kPrefixRows]) + (c[2 * kPrefixRows] + c[3 * kPrefixRows]));
      }
      const uint32_t reals = __ballot_sync(0xffffffffu, real);
      // D = 64: the sums of V's remainders, tensor memory's lanes 64 .. 127, to the threads of its values
      float* const turn = sTurn + first * 64 + 32 * (quarter & 1) + lane;
      if (D == 64 && quarter >= 2)
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          uint32_t u[8], v[8];
          tmem_ld8(tmem + kOut + lanes + first + 8 * c, u);
          tmem_ld8(tmem + kOut + lanes + k.at.rows + first + 8 * c, v);
          arrived(u, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) turn[(8 * c + e) * 64] = __uint_as_float(u[e]) + __uint_as_float(v[e]);
        }
      if (D == 64) bar_any(bar, false);
      if (D == 128 || quarter < 2) {
        float* const parts = (home ? a.prefix.home : a.prefix.extra) + 32 * quarter + (lane & 24) + ((lane & 1) << 2) + ((lane & 7) >> 1);   // the lane's dim
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          uint32_t u[8], v[8];
          tmem_ld8(tmem + kOut + lanes + first + 8 * c, u);
          tmem_ld8(tmem + kOut + lanes + k.at.rows + first + 8 * c, v);
          arrived(u, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int64_t to = __shfl_sync(0xffffffffu, place, 8 * c + e);
            const float low = D == 64 ? turn[(8 * c + e) * 64] : 0.0f;
            if ((reals >> (8 * c + e)) & 1u) parts[to * D] = __uint_as_float(u[e]) + (__uint_as_float(v[e]) + low);
          }
        }
      }
      tc_fence_before();
      bar_any(bar, false);   // sNeg and sNorm are read
      if (lane == 0) mbar_arrive(drained);
      ++seg;
      walk_next(k, p);
    }
  }
  // ---- teardown: every MMA done, then the tensor memory is freed ------------------------------
  if (warp == kMmaWarp && lane == 0) {
    volatile int dummy = 0;   // not the flag: a CTA that gave up waits for its MMAs all the same
    if (!mbar_wait(done, 0, kDrainLimit, &dummy)) *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) atomicOr(a.batch.err, DEV_ERR_WAIT_TIMEOUT);   // whichever warp's wait ran out
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- joining: a row's parts to its home, in order ----------------------------------------------------
// Only a unit that some worker goes on with has parts, so the blocks look at the workers: kSplit of them (blockIdx.y) take the
// rows of the unit that worker blockIdx.x of its class (blockIdx.z) is the first to go on with, if any.  (Looking at all rows
// of the list took 40 us for 6400 rows of 32 heads with nothing to join.)
constexpr int kJoinThreads = 256, kSplit = 8;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const PrefixArgs p) {
  constexpr int kCols = D / 4, kAtOnce = kJoinThreads / kCols, kFew = 4;
  griddep_launch();
  griddep_wait();
  const AttnArgs<__half>& a = p.a;
  const int col = threadIdx.x % kCols, group = a.shape.group, lane = threadIdx.x & 31, worker = blockIdx.x;
  const uint32_t mates = D == 128 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16);   // a row's lanes
  const int planned = *a.prefix.planned;
  // the class's last group that begins before the worker's share does, found by every warp
  const bool tall = blockIdx.z > 0;
  const PrefixGroup* const info = a.prefix.info + (tall ? a.tab.seqs : 0);
  int g = -1;
  for (int g0 = 0; g0 < planned; g0 += 32) {
    bool before = false;
    if (g0 + lane < planned) {
      const PrefixGroup& x = info[g0 + lane];
      before = x.units > 0 && x.base < worker * x.per;
    }
    const uint32_t found = __ballot_sync(0xffffffffu, before);
    if (found) g = g0 + 31 - __clz(found);
  }
  if (g < 0) return;
  const PrefixGroup at = info[g];
  const int64_t in = worker * at.per - at.base, unit = (in - 1) / at.tiles, start = at.base + unit * at.tiles;   // of the tile before the share
  const int h = static_cast<int>(unit / at.units), u = static_cast<int>(unit - static_cast<int64_t>(h) * at.units);
  if (h >= a.pool.heads || start / at.per + 1 != worker) return;   // past the group, or not the first
  const int count = static_cast<int>((start + at.tiles - 1) / at.per) - (worker - 1);
  if (count == 0) return;            // the share begins with the next unit
  const ClassRows list = class_rows(a.prefix, a.tab, a.batch, g, tall);
  const int rows = min(at.rows, list.list * group - u * at.rows);
  for (int rr = blockIdx.y * kAtOnce + threadIdx.x / kCols; rr < rows; rr += kSplit * kAtOnce) {
    const int r = u * at.rows + rr, x = r / group;
    const int64_t i = static_cast<int64_t>(place_of(a.prefix, list, at.first_row + x)) * a.q_heads + h * group + r - x * group;
    float* const home = a.prefix.home + i * D + 4 * col;
    const int64_t extra = at.extra + static_cast<int64_t>(worker) * at.stride + rr;
    float2 s = a.prefix.home_stat[i];
    float4 o = *reinterpret_cast<const float4*>(home);
    float m = s.x, l = s.y;
    for (int k0 = 0; k0 < count; k0 += kFew) {
      float2 st[kFew];
      float4 v[kFew];
#pragma unroll
      for (int k = 0; k < kFew; ++k) {
        st[k] = make_float2(-INFINITY, 0.0f);
        v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (k0 + k < count) {
          const int64_t row = extra + static_cast<int64_t>(k0 + k) * at.stride;
          st[k] = a.prefix.extra_stat[row];
          v[k] = *reinterpret_cast<const float4*>(a.prefix.extra + row * D + 4 * col);
        }
      }
      const float top = fmaxf(fmaxf(m, fmaxf(st[0].x, st[1].x)), fmaxf(st[2].x, st[3].x)), base = top == -INFINITY ? 0.0f : top;
      const float f0 = exp2f(m - base);
      l *= f0;
      o = make_float4(o.x * f0, o.y * f0, o.z * f0, o.w * f0);
#pragma unroll
      for (int k = 0; k < kFew; ++k) {
        const float f = exp2f(st[k].x - base);
        l = fmaf(st[k].y, f, l);
        o = make_float4(fmaf(v[k].x, f, o.x), fmaf(v[k].y, f, o.y), fmaf(v[k].z, f, o.z), fmaf(v[k].w, f, o.w));
      }
      m = top;
    }
    *reinterpret_cast<float4*>(home) = o;
    __syncwarp(mates);       // all have read it
    if (col == 0) a.prefix.home_stat[i] = make_float2(m, l);
  }
}

// ---- the plan of a call with chunks ------------------------------------------------------------------
// One CTA: who takes part, how many rows of steps and of chunks each group has and where a sequence's rows begin among those
// of its kind (a warp adds them up, 32 sequences at a time), the line, and where a call shares the list's places in order,
// steps first.  20 chunks over two prefixes: 7 us.
constexpr int kPlanThreads = 1024, kNear = 1024;
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PrefixArgs p) {
  __shared__ PrefixLine line;
  __shared__ int32_t near_member[kNear], near_rows[kNear], near_count[2][kNear];
  __shared__ bool near_split[kNear];
  griddep_launch();
  griddep_wait();
  const AttnArgs<__half>& a = p.a;
  const Prefix& x = a.prefix;
  const int seqs = a.tab.seqs, lane = threadIdx.x & 31, groups = groups_of(x, seqs);
  int32_t* const count[2] = {groups <= kNear ? near_count[0] : x.steps, groups <= kNear ? near_count[1] : x.chunks};
  if (threadIdx.x == 0) line.alone[0] = line.alone[1] = 0;
  for (int g = threadIdx.x; g < groups; g += blockDim.x) count[0][g] = count[1][g] = 0;
  for (int i = threadIdx.x; i < seqs; i += blockDim.x) {
    int n;
    const int g = shared_tokens(a, groups, i, n) > 0 ? x.group[i] : -1;
    if (i < kNear) {
      near_member[i] = g;
      near_rows[i] = n;
    } else {
      x.member[i] = g;
    }
  }
  auto member = [&](int i) { return i < kNear ? near_member[i] : x.member[i]; };
  auto rows_of = [&](int i) { return i < kNear ? near_rows[i] : a.batch.cu[i + 1] - a.batch.cu[i]; };
  __syncthreads();
  if (threadIdx.x < 32)
    for (int i0 = 0; i0 < seqs; i0 += 32) {
      const int i = i0 + lane;
      const int g = i < seqs ? member(i) : -1;
      if (!__any_sync(0xffffffffu, g >= 0)) continue;
      const int n = g < 0 ? 0 : rows_of(i);
      const bool chunk = static_cast<int64_t>(n) * a.shape.group > kStepRows;
      const uint32_t mates = __match_any_sync(0xffffffffu, g < 0 ? -1 : 2 * g + (chunk ? 1 : 0));   // the same kind of one group
      int mine = 0, all = 0;
#pragma unroll
      for (int l = 0; l < 32; ++l) {
        const int m = __shfl_sync(0xffffffffu, n, l);
        if ((mates >> l) & 1u) {
          all += m;
          if (l < lane) mine += m;
        }
      }
      if (g >= 0) mine += count[chunk][g];
      __syncwarp();
      if (g >= 0) {
        x.before[i] = mine;
        if (lane == __ffs(mates) - 1) count[chunk][g] += all;
      }
      __syncwarp();
    }
  __syncthreads();
  for (int g = threadIdx.x; g < groups; g += blockDim.x) {
    const int list = shared_group(x, a.tab, a.batch, g).list, steps = min(count[0][g], list), chunks = min(count[1][g], list - steps);   // (lists that contradict themselves)
    const bool split = static_cast<int64_t>(chunks) * a.shape.group > kPrefixFew;
    x.chunks[g] = chunks;
    x.steps[g] = split ? steps : -1;
    if (g < kNear) near_split[g] = split;
  }
  __syncthreads();
  auto split = [&](int g) { return g < kNear ? near_split[g] : x.steps[g] >= 0; };
  prefix_line<true>(p, line, [&](int, int i, int& n, int& tall) {
    const int g = member(i);
    n = rows_of(i);
    tall = g >= 0 && split(g) && static_cast<int64_t>(n) * a.shape.group > kStepRows ? 1 : 0;
    return g < 0 ? 0 : x.tokens[i];
  });
  if (!line.worth[0] && !line.worth[1]) return;
  for (int i = threadIdx.x >> 5; i < seqs; i += blockDim.x / 32) {   // a warp a sequence
    const int g = member(i);
    if (g < 0 || !split(g)) continue;
    const int n = rows_of(i);
    const SharedGroup s = shared_group(x, a.tab, a.batch, g);
    const int to = (static_cast<int64_t>(n) * a.shape.group > kStepRows ? x.steps[g] : 0) + x.before[i], from = s.first + x.first[i];
    for (int r = lane; r < n && to + r < s.list; r += 32) x.order[s.first + to + r] = from + r;
  }
}

template <int D>
fg_status launch(const PrefixArgs& p, cudaStream_t st) {
  using S = Smem<D>;
  static bool set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !set[dev]) {
    if (cudaFuncSetAttribute(prefix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes) != cudaSuccess)
      return check_launch("prefix_kernel smem attribute");
    set[dev] = true;
  }
  Trace tr(KC_ATTN_PAGED, st);
  return paged::launch("prefix_kernel", true, prefix_kernel<D>, static_cast<unsigned>(p.workers), kThreads, S::kBytes, st, p, wait_limit());
}

}  // namespace

fg_status paged_prefix_plan(const PrefixArgs& p, cudaStream_t st) {
  Trace tr(KC_ATTN_PAGED_PLAN, st);
  const unsigned threads = p.a.tab.seqs <= 224 ? 256 : kPlanThreads;   // a thread a sequence, and a warp
  return paged::launch("prefix_plan_kernel", true, prefix_plan_kernel, 1, threads, 0, st, p);
}

fg_status paged_prefix_join(const PrefixArgs& p, int head_dim, cudaStream_t st) {
  Trace tr(KC_ATTN_COMBINE, st);
  const dim3 grid(static_cast<unsigned>(p.workers), kSplit, p.tile.workers > 0 ? 2 : 1);
  return paged::launch("prefix_join_kernel", true, head_dim == 128 ? prefix_join_kernel<128> : prefix_join_kernel<64>, grid, kJoinThreads, 0, st, p);
}

fg_status paged_prefix(const PrefixArgs& p, int head_dim, cudaStream_t st) { return head_dim == 128 ? launch<128>(p, st) : launch<64>(p, st); }

}  // namespace paged
}  // namespace fg
