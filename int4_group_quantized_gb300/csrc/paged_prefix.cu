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
//   O^T[dim][row] += V^T P^T, V restored to fp16 (its 128-byte-swizzled rows are
//     the A operand, MN-major) and P as two fp16, value and remainder, side by
//     side as 2 N columns, added when the sums leave: no rounding of P that counts.
// What is left is V's rounding to fp16 and the result's.
//
// One CTA an SM walks its share of the line of tiles (paged_prefix.cuh), 128 keys a
// tile.  Warps 0..7: softmax, a key a thread, half of the rows each group of four
// warps; 8..11: K's codes into tensor memory, a key a thread, and a segment's Q;
// 12..14: V; 15: the MMAs.  Two stages of everything.  A row's maximum is known to
// all threads of its half: the segment's first tile finds it, a later tile takes
// it as it is and looks only whether a weight has left fp16 (a vote of the half);
// then the tile finds its maximum, the sums are rescaled and the weights formed
// again.  The normaliser stays with the threads (a key's share of every row's)
// until the segment ends.
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
static_assert(kThreads == 512 && kPrefixRows == 64, "the layout below");
constexpr float kLift = 4.0f;          // a row's largest weight is 2^4 or more when its maximum is found (paged_tile.cu)
constexpr uint32_t kMostHalf = 0x7800u;   // 2^15 as fp16: weights up to it stand

template <int D>
struct Smem {
  static constexpr int kPanel = kKeys * 128;            // 128 rows of 128 bytes
  static constexpr int kV = D / 64 * kPanel;
  static constexpr int kP = 2 * kPanel;                 // 2 N <= 128 columns
  static constexpr int kQPanel = kPrefixRows * 128;
  static constexpr int kQ = D / 64 * kQPanel;
  static constexpr int kSums = kPrefixRows * 8;         // (sum q of group 0, 1) of two rows side by side
  static constexpr int kBytes = 1024 + 2 * (kV + kP + kQ) + 2 * kSums + 4 * kPrefixRows * 2 + 4 * kPrefixRows * 4 + 256;
};

// A share's walk over its segments: parts of one unit's key tiles.
struct Walk {
  int64_t left;
  int g, h, u, x, x1;
  SharedGroup s;
  PrefixGroup at;
};
__device__ __forceinline__ void walk_begin(Walk& k, const PrefixArgs& p, const PrefixLine& line) {
  const int64_t o0 = blockIdx.x * line.per;
  k.left = 0;
  if (o0 >= line.total) return;
  k.left = line.per < line.total - o0 ? line.per : line.total - o0;
  k.g = line.g;
  k.at = line.at;
  k.s = shared_group(p.a.prefix, p.a.tab, p.a.batch, k.g);
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
      do k.s = shared_group(p.a.prefix, p.a.tab, p.a.batch, ++k.g);
      while (k.s.list == 0 || (p.tile.workers > 0 && static_cast<int64_t>(k.s.list) * p.a.shape.group > kPrefixFew));
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
// 64 codes of one group through fp16(fmaf(q, scale, min)) into row r of a swizzled panel; every 8 dims in the order (0, 4),
// (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ void restore_group(const uint4& lo, const uint4& hi, float scale, float mn, uint8_t* prow, int r) {
  const float2 lo2 = both(scale * 16777216.0f), hi2 = both(scale * 1048576.0f), m2 = both(mn);
  const uint32_t words[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t x = words[c], y = x >> 8;
    const uint4 o = make_uint4(q4::cvt_f16x2(q4::fma_f32x2(halves(x & 0x000F000Fu), lo2, m2)), q4::cvt_f16x2(q4::fma_f32x2(halves(x & 0x00F000F0u), hi2, m2)),
                               q4::cvt_f16x2(q4::fma_f32x2(halves(y & 0x000F000Fu), lo2, m2)), q4::cvt_f16x2(q4::fma_f32x2(halves(y & 0x00F000F0u), hi2, m2)));
    *reinterpret_cast<uint4*>(prow + ((c ^ (r & 7)) << 4)) = o;
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
  float* const sSum = reinterpret_cast<float*>(sQ + 2 * S::kQ);            // [segment % 2][row / 2][group][row % 2]
  float* const sNeg = sSum + 2 * S::kSums / 4;                             // [row] minus the maximum
  uint32_t* const sTop = reinterpret_cast<uint32_t*>(sNeg + kPrefixRows);  // [row] a tile's largest score, as an ordered key
  float* const sNorm = reinterpret_cast<float*>(sTop + kPrefixRows);       // [quarter][row]
  uint64_t* const bars = reinterpret_cast<uint64_t*>(sNorm + 4 * kPrefixRows);
  uint64_t* const kfull = bars;        // [stage] K's codes of the tile are in tensor memory
  uint64_t* const sfull = bars + 2;    // [stage] S^T of the tile is, and K's place is free
  uint64_t* const sfree = bars + 4;    // [stage] the softmax warps have read it, and the rows' sums
  uint64_t* const vfull = bars + 6;    // [stage] V of the tile is in shared memory
  uint64_t* const pfull = bars + 8;    // [stage] P is
  uint64_t* const pvdone = bars + 10;  // [stage] P V of the tile has completed
  uint64_t* const qfull = bars + 12;   // [segment % 2] Q of the segment is in shared memory
  uint64_t* const drained = bars + 14; // O of the segment has been read
  uint64_t* const done = bars + 15;    // every MMA has completed
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(bars + 16);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  __shared__ PrefixLine line;

  const AttnArgs<__half>& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kfull[i], kKeyWarps);
      mbar_init(&sfull[i], 1);
      mbar_init(&sfree[i], kSoftWarps);
      mbar_init(&vfull[i], 4);
      mbar_init(&pfull[i], kSoftWarps);
      mbar_init(&pvdone[i], 1);
      mbar_init(&qfull[i], kKeyWarps);
    }
    mbar_init(drained, kSoftWarps);
    mbar_init(done, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch();
  griddep_wait();
  prefix_line(p, line);
  Walk k;
  walk_begin(k, p, line);

  const int psl = a.pool.ps_log2, psm = (1 << psl) - 1;
  // page number of a key's table entry (not looked at before `there`), and the key's place in a page of head h
  auto entry = [&](const Walk& w, int j) { return j < w.s.tokens ? a.tab.table[w.s.leader * a.tab.stride + (j >> psl)] : -1; };
  auto there = [&](int page) { return static_cast<uint32_t>(page) < static_cast<uint32_t>(a.tab.pages); };
  auto slot = [&](int page, int h, int j) {
    return ((static_cast<int64_t>(page) * a.pool.heads + h) << psl) + (j & psm);
  };

  if (warp >= kFirstKey && warp < kFirstValue) {
    // ---- K's codes, a key a thread; a segment's Q before its first tile -------------------
    const int quarter = warp & 3, r = 32 * quarter + lane;
    int n = 0, seg = 0;
    uint4 code[2 * NG];
    auto load = [&](const Walk& w, int x, int page) {
      const int j = (x << kPrefixKeysLog2) + r;
      const bool on = j < w.s.tokens && there(page);
      if (j < w.s.tokens && !on) atomicOr(a.batch.err, DEV_ERR_PAGE);
      const uint4* c = reinterpret_cast<const uint4*>(a.pool.codes[0] + slot(on ? page : 0, w.h, on ? j : 0) * (D / 2));
#pragma unroll
      for (int e = 0; e < 2 * NG; ++e) code[e] = on ? c[e] : make_uint4(0u, 0u, 0u, 0u);
    };
    bool ok = true;
    while (k.left > 0 && ok) {
      // Q and the sums of this segment's place were last used two segments ago: by S of a tile two or more before this
      // one, and by the softmax that followed it
      if (n >= 2) ok = mbar_wait(&sfree[n & 1], ((n >> 1) - 1) & 1, wait_limit, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      int page = entry(k, (k.x << kPrefixKeysLog2) + r);
      load(k, k.x, page);
      page = entry(k, ((k.x + 1) << kPrefixKeysLog2) + r);
      {
        uint8_t* const q = sQ + (seg & 1) * S::kQ;
        float* const sum = sSum + (seg & 1) * (S::kSums / 4);
        constexpr int kPieces = D / 8;                    // 16 bytes each, a lane a piece
        const int pc = lane % kPieces, all = k.s.list * a.shape.group, r0 = k.u * k.at.rows;
        for (int i = quarter * (32 / kPieces) + lane / kPieces; i < k.at.rows; i += kKeyWarps * (32 / kPieces)) {
          const int row = r0 + i, x = row / a.shape.group;
          const bool on = row < all;
          const __half* from = a.q + static_cast<int64_t>(on ? listed_row(a.prefix, a.batch, k.s.first + x) : 0) * a.ldq +
                               static_cast<int64_t>(k.h * a.shape.group + (on ? row - x * a.shape.group : 0)) * D + 8 * pc;
          const uint4 v = on ? *reinterpret_cast<const uint4*>(from) : make_uint4(0u, 0u, 0u, 0u);
          // every 8 dims in the codes' order
          *reinterpret_cast<uint4*>(q + (pc >> 3) * S::kQPanel + i * 128 + (((pc & 7) ^ (i & 7)) << 4)) =
              make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
          const float2 f0 = halves(v.x), f1 = halves(v.y), f2 = halves(v.z), f3 = halves(v.w);
          float s = ((f0.x + f0.y) + (f1.x + f1.y)) + ((f2.x + f2.y) + (f3.x + f3.y));
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);   // rows are a multiple of 16: every lane comes as often
          if ((pc & 7) == 0) sum[(i >> 1) * 4 + (pc >> 3) * 2 + (i & 1)] = s;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&qfull[seg & 1]);
      }
      for (int x = k.x; x < k.x1; ++x, ++n) {
        ok = n < 2 || mbar_wait(&sfull[n & 1], ((n >> 1) - 1) & 1, wait_limit, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t to = tmem + kCodes + 64 * (n & 1) + (static_cast<uint32_t>(32 * quarter) << 16);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          uint32_t o[32];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t w[4] = {code[2 * g + e].x, code[2 * g + e].y, code[2 * g + e].z, code[2 * g + e].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              o[16 * e + 4 * c] = w[c] & 0x000F000Fu;
              o[16 * e + 4 * c + 1] = (w[c] >> 4) & 0x000F000Fu;
              o[16 * e + 4 * c + 2] = (w[c] >> 8) & 0x000F000Fu;
              o[16 * e + 4 * c + 3] = (w[c] >> 12) & 0x000F000Fu;
            }
          }
          tmem_st_32x32b_x32(to + 32 * g, o);
        }
        if (x + 1 < k.x1) {
          load(k, x + 1, page);
          page = entry(k, ((x + 2) << kPrefixKeysLog2) + r);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kfull[n & 1]);
      }
      ++seg;
      walk_next(k, p);
    }
  } else if (warp >= kFirstValue && warp < kMmaWarp) {
    // ---- V, 32 keys a task, four tasks a tile, dealt round the warps ------------------------
    Walk w = k;              // of the task that is loaded next
    int x = k.x, at = 0, n = warp - kFirstValue;   // its tile, that tile's number, the task in hand
    const int tasks = k.left > 0 ? static_cast<int>(4 * k.left) : 0;
    auto go_to = [&](int tile) {   // the walk at the tile of that number
      while (at < tile) {
        ++at;
        if (++x == w.x1) {
          walk_next(w, p);
          x = w.x;
          if (w.left == 0) return;
        }
      }
    };
    uint4 code[2 * NG];
    float scale[NG], mn[NG];
    int page = -1, j = 0, h = 0;
    bool in = false;
    auto look_up = [&](int task) {   // the lane's key and its table entry
      in = task < tasks;
      if (!in) return;
      go_to(task >> 2);
      j = (x << kPrefixKeysLog2) + 32 * (task & 3) + lane;
      h = w.h;
      in = j < w.s.tokens;
      page = entry(w, j);
    };
    auto load = [&]() {
      const bool on = in && there(page);
      const int64_t s = slot(on ? page : 0, h, on ? j : 0);
      const uint4* c = reinterpret_cast<const uint4*>(a.pool.codes[1] + s * (D / 2));
#pragma unroll
      for (int e = 0; e < 2 * NG; ++e) code[e] = on ? c[e] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int g = 0; g < NG; ++g) scale[g] = mn[g] = 0.0f;
      if (on) {
        load_meta(scale, a.pool.scales[1], s * (4 * NG));
        load_meta(mn, a.pool.mins[1], s * (4 * NG));
      }
    };
    look_up(n);
    load();
    look_up(n + kValueWarps);
    for (; n < tasks; n += kValueWarps) {
      const int g = n >> 2, r = 32 * (n & 3) + lane;
      bool ok = g < 2 || mbar_wait(&pvdone[g & 1], ((g >> 1) - 1) & 1, wait_limit, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint8_t* const to = sV + (g & 1) * S::kV + r * 128;
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        // a group whose scale is not finite is NaN for all rows: they all see the key
        const float sc = fabsf(scale[q]) < INFINITY ? scale[q] : __uint_as_float(0x7fffffffu);
        restore_group(code[2 * q], code[2 * q + 1], sc, mn[q], to + q * S::kPanel, r);
      }
      load();
      look_up(n + 2 * kValueWarps);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&vfull[g & 1]);
    }
  } else if (warp == kMmaWarp) {
    // ---- MMA issuer --------------------------------------------------------------------
    if (lane == 0) {
      const uint32_t q_lo = static_cast<uint32_t>(smem_desc_sw128(smem_u32(sQ), 16, 1024));
      const uint32_t v_lo = static_cast<uint32_t>(smem_desc_sw128(smem_u32(sV), D == 128 ? S::kPanel : 0, 1024));   // 64 dims: twice the same
      const uint32_t p_lo = static_cast<uint32_t>(smem_desc_sw128(smem_u32(sP), S::kPanel, 1024));
      int n = 0, seg = 0;
      bool ok = true, pending = false;
      auto wait = [&](uint64_t* bar, int phase) {
        if (ok) ok = mbar_wait(bar, phase & 1, wait_limit, abort_flag);
        return ok;
      };
      // P V of tile g; first: of its segment, whose number is `of` and whose unit has `rows` rows
      auto issue_o = [&](int g, bool first, int of, int rows) {
        if (first && of > 0 && !wait(drained, of - 1)) return;
        if (!wait(&vfull[g & 1], g >> 1) || !wait(&pfull[g & 1], g >> 1)) return;
        tc_fence_after();
        const uint32_t idesc = idesc_f16(128, 0, 1, 1) + (static_cast<uint32_t>(rows >> 2) << 17);   // 2 rows columns
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          mma_ss(tmem + kOut, v_lo + (g & 1) * (S::kV >> 4) + kk * (2048 >> 4), kDescHi, p_lo + (g & 1) * (S::kP >> 4) + kk * (2048 >> 4), kDescHi, idesc,
                 !first || kk > 0);
        mma_commit(&pvdone[g & 1]);
      };
      bool first = false;   // of the tile before this one
      int of = 0, rows = 16;
      while (k.left > 0 && ok) {
        const uint32_t idesc = idesc_f16(128, 0, 0, 0) + (static_cast<uint32_t>(k.at.rows >> 3) << 17);
        if (!wait(&qfull[seg & 1], seg >> 1)) break;
        for (int x = k.x; x < k.x1; ++x, ++n) {
          if (!wait(&kfull[n & 1], n >> 1)) break;
          if (n >= 2 && !wait(&sfree[n & 1], (n >> 1) - 1)) break;
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts(tmem + kScore + 128 * (n & 1) + 64 * g, tmem + kCodes + 64 * (n & 1) + 32 * g + 8 * kk,
                     q_lo + (((seg & 1) * S::kQ + g * S::kQPanel + 32 * kk) >> 4), kDescHi, idesc, kk > 0);
          mma_commit(&sfull[n & 1]);
          if (pending) issue_o(n - 1, first, of, rows);
          if (!ok) break;
          pending = true;
          first = x == k.x;
          of = seg;
          rows = k.at.rows;
        }
        ++seg;
        walk_next(k, p);
      }
      if (ok && pending) issue_o(n - 1, first, of, rows);
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
    // the key's scales and minima of K, in units of the exponent
    float ks[NG], km[NG];
    bool here = false;
    auto load = [&](const Walk& w, int x, int page) {
      const int j = (x << kPrefixKeysLog2) + r;
      here = j < w.s.tokens && there(page);
#pragma unroll
      for (int g = 0; g < NG; ++g) ks[g] = km[g] = 0.0f;
      if (here) {
        const int64_t s = slot(page, w.h, j) * (4 * NG);
        load_meta(ks, a.pool.scales[0], s);
        load_meta(km, a.pool.mins[0], s);
      }
    };
    while (k.left > 0) {
      const int rows = k.at.rows / 2, chunks = rows / 8, first = half * rows;   // of this half
      const float* const sum = sSum + (seg & 1) * (S::kSums / 4) + first * 2;
      float2 l[16];        // the normaliser's part of this key and those 128 after it, of two rows each
#pragma unroll
      for (int i = 0; i < 16; ++i) l[i] = both(0.0f);
      int page = entry(k, (k.x << kPrefixKeysLog2) + r);
      load(k, k.x, page);
      page = entry(k, ((k.x + 1) << kPrefixKeysLog2) + r);
      ok = mbar_wait(&qfull[seg & 1], (seg >> 1) & 1, wait_limit, abort_flag);   // the rows' sums
      bool gave_up = false;
      for (int x = k.x; x < k.x1; ++x, ++n) {
        const int st = n & 1;
        const uint32_t ts = tmem + kScore + 128 * st + lanes + first;
        float2 s2[NG], m2[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          // a code in the MMA is c * 2^-24; a scale that is not finite makes the key's scores NaN
          s2[g] = both(fabsf(ks[g]) < INFINITY ? ks[g] * (a.scale_log2 * 16777216.0f) : __uint_as_float(0x7fffffffu));
          m2[g] = both(km[g] * a.scale_log2);
        }
        const bool on = here;
        if (x + 1 < k.x1) {
          load(k, x + 1, page);
          page = entry(k, ((x + 2) << kPrefixKeysLog2) + r);
        }
        ok = ok && mbar_wait(&sfull[st], (n >> 1) & 1, wait_limit, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        // scores of rows 8 c .. 8 c + 7 of the half, on top of from(row)
        auto scores = [&](int c, float2 (&z)[4], auto from) {
          uint32_t u[8], v[8];
          tmem_ld8(ts + 8 * c, u);
          if (NG == 2) tmem_ld8(ts + 64 + 8 * c, v);
          else
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0u;
          arrived(u, v);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 q = *reinterpret_cast<const float4*>(sum + 4 * (4 * c + e));
            float2 t = q4::fma_f32x2(m2[0], make_float2(q.x, q.y), from(8 * c + 2 * e));
            if (NG == 2) t = q4::fma_f32x2(m2[NG - 1], make_float2(q.z, q.w), t);
            t = q4::fma_f32x2(s2[0], make_float2(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1])), t);
            if (NG == 2) t = q4::fma_f32x2(s2[NG - 1], make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), t);
            z[e] = t;
          }
        };
        auto below = [&](int i) {   // minus the maximum of rows i, i + 1 of the half; a key that is not there weighs nothing
          const float2 m = *reinterpret_cast<const float2*>(sNeg + first + i);
          return on ? m : both(-INFINITY);
        };
        // the tile's largest score of every row of the half, as ordered keys (two barriers around it)
        auto find = [&]() {
          if (quarter == 0 && lane < rows) sTop[first + lane] = 0u;
          bar_any(bar, false);
          if (ok)
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
              float2 z[4];
              scores(c, z, [](int) { return both(0.0f); });
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float f = on ? (e & 1 ? z[e / 2].y : z[e / 2].x) : -INFINITY;
                const uint32_t b = __float_as_uint(f), key = f != f ? 0u : b & 0x80000000u ? ~b : b | 0x80000000u;
                const uint32_t top = __reduce_max_sync(0xffffffffu, key);
                if (lane == e) atomicMax(sTop + first + 8 * c + e, top);
              }
            }
          bar_any(bar, false);
        };
        auto top_of = [&](int i) {
          const uint32_t key = sTop[first + i];
          return key == 0u ? -INFINITY : __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
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
        if (ok && n >= 2) ok = mbar_wait(&pvdone[st], ((n >> 1) - 1) & 1, wait_limit, abort_flag);   // P's place is free
        ok = __all_sync(0xffffffffu, ok);
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
            reinterpret_cast<float*>(sTop)[first + lane] = !ask ? 1.0f : old == INFINITY ? 0.0f : ex2_approx(neg - old);
          }
          bar_any(bar, false);
          const float* const shrink = reinterpret_cast<const float*>(sTop) + first;
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
          mbar_arrive(&sfree[st]);
        }
      }
      if (gave_up) break;
      // ---- the segment's rows: their parts ------------------------------------------------
      ok = mbar_wait(&pvdone[(n - 1) & 1], ((n - 1) >> 1) & 1, wait_limit, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      {   // the normaliser: a row's 32 keys of the warp to one lane, the four warps in order
        float v[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          v[2 * i] = l[i].x;
          v[2 * i + 1] = l[i].y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
          for (int i = 0; i < o; ++i) {
            const bool up = lane & o;
            v[i] = (up ? v[i + o] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + o], o);
          }
        if (lane < rows) sNorm[quarter * kPrefixRows + first + lane] = v[0];
      }
      if (bar_any(bar, !ok)) break;
      // where row `first` + lane of the unit goes
      const int row = k.u * k.at.rows + first + lane;
      const bool real = lane < rows && row < k.s.list * a.shape.group, home = k.x == 0;
      const int lx = real ? row / a.shape.group : 0;
      const int64_t place = home ? static_cast<int64_t>(k.s.first + lx) * a.q_heads + k.h * a.shape.group + (real ? row - lx * a.shape.group : 0)
                                 : static_cast<int64_t>(blockIdx.x) * kPrefixRows + first + lane;
      if (quarter == 0 && real) {
        const float* const c = sNorm + first + lane;
        (home ? a.prefix.home_stat : a.prefix.extra_stat)[place] =
            make_float2(-sNeg[first + lane], (c[0] + c[kPrefixRows]) + (c[2 * kPrefixRows] + c[3 * kPrefixRows]));
      }
      const uint32_t reals = __ballot_sync(0xffffffffu, real);
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
            if ((reals >> (8 * c + e)) & 1u) parts[to * D] = __uint_as_float(u[e]) + __uint_as_float(v[e]);
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

fg_status paged_prefix(const PrefixArgs& p, int head_dim, cudaStream_t st) { return head_dim == 128 ? launch<128>(p, st) : launch<64>(p, st); }

}  // namespace paged
}  // namespace fg
