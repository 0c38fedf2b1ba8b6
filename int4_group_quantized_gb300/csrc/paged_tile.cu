// Paged attention of chunks on tcgen05 (FlexGen notes, "背景知识": Softmax(x_Q
// x_K^T / sqrt(h1)) x_V per head, causal; "5. 近似方法": K and V stored in
// 4-bit groups of 64 and converted back to FP16), fp16 activations, sequences
// of more than 16 rows per K/V head.
//
// A unit is 256 rows (token t, query head g of the K/V head's group: row t *
// group + g), so that every restored K/V tile of 128 keys feeds two MMA tiles
// of 128 rows; one persistent CTA per SM walks its share of the line of tiles
// (paged_sched.cuh).  Roles:
//   * seven warps restore: a tile is eight tasks (K or V of 32 keys, a key a
//     lane), dealt round the warps in order.  A task's codes are loaded into
//     registers a task ahead, its page number two; they go through
//     fp16(fmaf(q, scale, min)) -- a masked nibble is the subnormal fp16 c *
//     2^-24, exact in fp32, then one paired fp32 FMA and one rounding -- into
//     the 128-byte-swizzled rows the MMA reads (K: K-major panels, V: MN-major
//     blocks; the same bytes).  A pair of a code word's halves holds dims (0,
//     4), (1, 5), (2, 6), (3, 7); Q is laid out in the same order and O is
//     taken apart in it;
//   * two groups of four softmax warps (one row a thread) keep a maximum and
//     the sum in base 2, write P (fp16) into tensor memory as the second MMA's
//     A operand, look for a new maximum (and rescale O there) only when the
//     known one no longer serves, and finish or hand on a share's rows;
//   * one thread issues S = Q K^T (M = N = 128) and O += P V for both groups in
//     turn, so that one group's softmax runs under the other's MMAs.
// Tensor memory: S of each group, O of each group, and P: in the columns of its
// S at head_dim 128 (S of the next tile is issued after the P V that reads it,
// in the order of one thread's MMAs of one shape), in columns of its own at 64.
//
// Rows see a key by position alone, so masks are words of bits per row, made
// only for tiles at an edge.  A V group that restores to NaN enters the product
// as zeros and is remembered for the rows that see it (0 * NaN would reach all).
// Every wait is bounded; on timeout the CTA raises the device error word, lets
// its MMAs finish and frees its tensor memory.
//
// Measured: a chunk of 2048 rows over 16384 tokens, 32 heads of 128, 452 to 460
// us (1.13 PFLOP/s, 59% of what a large bf16 library product reaches); a batch of
// 12 chunks (7 to 554 rows, 32 query heads on 8, a window of 1000 with 4 sinks)
// 118 to 119 us; 64 chunks of 20 rows over 300 to 600 tokens, 8 heads, 62 us.  A tile takes 3400 cycles where its four MMA batches take 2200:
// the protocol with its MMAs alone, no softmax and no restoring, takes 362 us
// of the chunk's 450; with every exponential replaced by a multiply-add it takes
// as long, without the restoring's arithmetic 424: a group's S, softmax and P V
// follow one another, and so do their barriers (250 cycles each).  A segment
// costs 10000 cycles more (walk, Q, first S, first softmax, O), a launch 25000
// before its first P V.  Other splits when a tile took a quarter longer: 24
// softmax and restoring warps of 80 registers 715 us against 588, two issuing
// warps 562 against 470.
#include <math.h>

#include <algorithm>

#include "paged_attn.cuh"
#include "q4_dev.cuh"
#include "tc_ptx.cuh"

namespace fg {
namespace paged {
namespace {

using namespace tc;

constexpr int kKeysLog2 = 7;
constexpr int kKeys = 1 << kKeysLog2;
constexpr int kRows = kTileRows;
constexpr int kSoftWarps = 8;      // warps 0..3: rows 0..127, warps 4..7: rows 128..255
constexpr int kRestoreWarps = 7;   // warps 8..14
constexpr int kMmaWarp = 15;
constexpr int kThreads = 16 * 32;
// Weights P = 2^(s - m) with m kLift below the largest score known when m was found: the largest weight of a row is 2^4
// or more, so that small ones keep their bits down to 2^-18 of it, and thousands of 2^-26 beside one large weight still add
// up (without the lift they were rounded to zero).  A higher lift leaves less room above a first tile's maximum, and more
// tiles look for theirs: the 12 chunks above 118.0 us with 3 or 4, 118.4 with 5, 124.6 with 6, 140 with 8 (the chunk 457
// to 458 with any).
constexpr float kLift = 4.0f;
constexpr float kMostSum = 60000.0f;   // a tile's row sum up to which its weights stand as fp16; where m is the tile's own, at most 128 * 2^4

template <int D>
struct Smem {
  static constexpr int kPanels = D / 64;
  static constexpr int kPanel = 128 * 128;              // 128 rows of 128 bytes
  static constexpr int kQ = kPanels * kPanel;           // one group's
  static constexpr int kK = kPanels * kPanel;
  static constexpr int kStage = 2 * kK;                 // K, then V
  static constexpr int kFlags = 4 * 16;                 // of a tile: whether any is set, absent keys, NaN value groups 0 and 1
  static constexpr int kOut = 32 * 128;                 // a softmax warp's rows on their way out, 128 bytes of each
  static constexpr int kBytes = 1024 + 2 * kQ + 2 * kStage + kSoftWarps * kOut + 4 * kFlags + 256;
  static_assert(kBytes + sizeof(OwnPlan) + sizeof(Line) + 64 <= 232448, "shared memory of one CTA");
};

// A share's walk over its segments: parts of one unit's key tiles.
// What a launch attends to: sequences alone, sequences behind their shared prefixes (Table::skip), or the prefixes: then an
// "i" is a group, whose rows all stand behind its tokens, and its rows' parts are left for the sequences.
enum : int { kAlone = 0, kBehind = 1, kPrefix = 2 };
struct Walk {
  int left;              // tiles of the share still to come
  int i, h, u, x;        // sequence (or group), head, unit, tile of the unit
  int units;
  Seq s;
  Unit un;
  Span sp;
  int x1;                // the current segment: tiles x .. x1 - 1
};
__device__ __forceinline__ void walk_unit(Walk& k, const AttnArgs<__half>& a) {
  k.un = unit_of<kRows>(k.s, a.shape.group, k.u);
  k.sp = span_of<kKeysLog2>(k.un.p0, k.un.p1, k.s.keys, a.shape.window, a.shape.sinks);
}
template <int MODE>
__device__ __forceinline__ void walk_seq(Walk& k, const AttnArgs<__half>& a) {
  if (MODE == kPrefix) {
    const ClassRows g = class_rows(a.prefix, a.tab, a.batch, k.i, true);   // of a split group: rows by Prefix::order
    k.s = Seq{g.first, g.list, g.tokens + g.list, g.tokens, 0};
  } else {
    k.s = seq_of<MODE == kBehind>(a.tab, a.batch, k.i);
  }
  k.units = static_cast<int>((static_cast<int64_t>(k.s.n) * a.shape.group + kRows - 1) / kRows);
  k.u = 0;
}
// Share w's first segment (left = 0: none).
template <int MODE>
__device__ __forceinline__ void walk_begin(Walk& k, const AttnArgs<__half>& a, const Line& pl, int w) {
  const int64_t total = pl.total, per = pl.per, o0 = w * per;
  k.left = 0;
  if (o0 >= total) return;
  int lo = 0, hi = a.tab.seqs;   // pre[lo] <= o0 < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pl.pre[mid] <= o0) lo = mid;
    else hi = mid;
  }
  k.i = lo;
  k.left = static_cast<int>(total - o0 < per ? total - o0 : per);
  walk_seq<MODE>(k, a);
  const int64_t all = pl.pre[lo + 1] - pl.pre[lo], in = o0 - pl.pre[lo];   // (32-bit divisions where they do: the short ones)
  const int64_t cost = all <= INT32_MAX ? static_cast<int>(all) / a.pool.heads : all / a.pool.heads;
  k.h = all <= INT32_MAX ? static_cast<int>(in) / static_cast<int>(cost) : static_cast<int>(in / cost);
  int64_t rest = in - k.h * cost;
  const int lane = threadIdx.x & 31;
  for (;; k.u += 32) {   // a unit a lane
    const Unit un = unit_of<kRows>(k.s, a.shape.group, min(k.u + lane, k.units - 1));
    const int n = k.u + lane < k.units ? span_of<kKeysLog2>(un.p0, un.p1, k.s.keys, a.shape.window, a.shape.sinks).n : 0;
    int64_t inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, rest < inc);
    if (past) {
      const int at = __ffs(past) - 1;
      k.u += at;
      rest -= __shfl_sync(0xffffffffu, inc - n, at);
      break;
    }
    rest -= __shfl_sync(0xffffffffu, inc, 31);
    if (k.u + 32 >= k.units) break;   // not reached: the share begins inside the item
  }
  walk_unit(k, a);
  k.x = static_cast<int>(rest);
  k.x1 = k.x + (k.left < k.sp.n - k.x ? k.left : k.sp.n - k.x);
}
// On to the next segment.
template <int MODE>
__device__ __forceinline__ void walk_next(Walk& k, const AttnArgs<__half>& a, const Line& pl) {
  k.left -= k.x1 - k.x;
  if (k.left == 0) return;
  if (++k.u == k.units) {
    k.u = 0;
    if (++k.h == a.pool.heads) {
      do ++k.i;
      while (pl.pre[k.i + 1] == pl.pre[k.i]);
      k.h = 0;
      walk_seq<MODE>(k, a);
    }
  }
  walk_unit(k, a);
  k.x = 0;
  k.x1 = k.left < k.sp.n ? k.left : k.sp.n;
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
// Waits for this thread's tensor-memory loads; the registers named are not
// read before it.
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
  asm volatile(""
               : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
// 16 bytes into shared memory, zeros where not `there` (then the address is not read).
__device__ __forceinline__ void cp16_zfill(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16u : 0u) : "memory");
}
// 16 consecutive columns (tmem_arrived before they are read).
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Bits c of a word with c < n, for any n.
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// The MMAs with their descriptors as a running low word (the start address
// field; offsets inside the CTA's allocation never carry out of it) and one
// high word: a couple of instructions an MMA for the issuing thread.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool acc) {
  asm volatile(
      "{ .reg .pred p; .reg .b64 x, y; setp.ne.b32 p, %5, 0; mov.b64 x, {%1, %3}; mov.b64 y, {%2, %3};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p; }" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; .reg .b64 y; setp.ne.b32 p, %5, 0; mov.b64 y, {%2, %3};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p; }" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
      : "memory");
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
// 64 codes (32 bytes) of one group through fp16(fmaf(q, scale, min)) into row
// r of a swizzled panel.
__device__ __forceinline__ void restore_group(const uint4& lo, const uint4& hi, float scale, float mn, uint8_t* prow, int r) {
  // a masked nibble is c * 2^-24 or 16 c * 2^-24; scaling by powers of two is exact
  const float2 lo2 = make_float2(scale * 16777216.0f, scale * 16777216.0f), hi2 = make_float2(scale * 1048576.0f, scale * 1048576.0f);
  const float2 m2 = make_float2(mn, mn);
  const uint32_t words[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t x = words[c], y = x >> 8;
    const uint4 o = make_uint4(q4::cvt_f16x2(q4::fma_f32x2(halves(x & 0x000F000Fu), lo2, m2)),
                               q4::cvt_f16x2(q4::fma_f32x2(halves(x & 0x00F000F0u), hi2, m2)),
                               q4::cvt_f16x2(q4::fma_f32x2(halves(y & 0x000F000Fu), lo2, m2)),
                               q4::cvt_f16x2(q4::fma_f32x2(halves(y & 0x00F000F0u), hi2, m2)));
    *reinterpret_cast<uint4*>(prow + ((c ^ (r & 7)) << 4)) = o;
  }
}

// One key's row of K or V as it is stored.
template <int NG>
struct Raw {
  uint4 code[2 * NG];
  float scale[NG], mn[NG];
  float vscale[NG];      // of its value, with K
  bool absent;           // the table has no page for it
};
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

template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1) tile_kernel(const AttnArgs<__half> a, const ClassPlan pl, uint32_t wait_limit, const bool own_plan, const bool every) {
  using S = Smem<D>;
  constexpr int NG = D / 64;
  constexpr uint32_t kIdescS = idesc_f16(128, 128, 0, 0);   // A = Q (K-major), B = K (K-major)
  constexpr uint32_t kIdescO = idesc_f16(128, D, 0, 1);     // A = P (tensor memory), B = V (MN-major)
  constexpr uint32_t kO = 256;                              // S: 0 and 128; O: 256 and 256 + D
  constexpr uint32_t kP = D == 128 ? 0 : 384, kPStep = D == 128 ? 128 : 64;
  constexpr uint32_t kTmemCols = 512;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = sm;
  uint8_t* sKV = sQ + 2 * S::kQ;
  uint8_t* sOut = sKV + 2 * S::kStage;
  uint32_t* sFlags = reinterpret_cast<uint32_t*>(sOut + kSoftWarps * S::kOut);   // [tile % 4][any, absent, nan 0, nan 1][4]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sOut + kSoftWarps * S::kOut + 4 * S::kFlags);
  uint64_t* qfull = bars;         // [group] Q of the segment is in place
  uint64_t* kfull = bars + 2;     // [stage]
  uint64_t* vfull = bars + 4;
  // Release c (barrier c % 2) says that S of tile c and P V of tile c - 1 have read their operands: K's place of tile c and
  // V's of tile c - 1 are free.
  uint64_t* freed = bars + 6;
  uint64_t* sfull = bars + 10;    // [group] S of the tile is in tensor memory
  uint64_t* pfull = bars + 12;    // [group] P of the tile is
  uint64_t* odone = bars + 14;    // [group] the segment's last P V has completed
  uint64_t* done = bars + 16;     // every MMA has
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 17);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = blockIdx.x;

  if (MODE == kPrefix) {   // often there is nothing: then it ends before it takes tensor memory
    griddep_launch();
    griddep_wait();
    if (pl.head[0] == 0) return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&qfull[i], 4);
      mbar_init(&kfull[i], 4);
      mbar_init(&vfull[i], 4);
      mbar_init(&freed[i], 1);
      mbar_init(&sfull[i], 2);   // the commit, and the issuer itself: it has seen K's barrier, and so the tile's flags
      mbar_init(&pfull[i], 4);
      mbar_init(&odone[i], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (MODE != kPrefix) {
    griddep_launch();
    griddep_wait();
  }
  __shared__ OwnPlan own;
  __shared__ Line line;   // not in registers: it is read between segments only
  {
    const Line x = own_plan ? make_line<false, kRows, kKeysLog2, MODE == kBehind>(own, a.tab, a.batch, a.shape, a.pool.heads, pl.workers, every)
                            : Line{pl.pre, pl.head[0], pl.head[1]};
    if (threadIdx.x == 0) line = x;
    __syncthreads();
  }

  Walk k;
  walk_begin<MODE>(k, a, line, w);

  if (warp >= kSoftWarps && warp < kSoftWarps + kRestoreWarps) {
    // ---- restoring warps: task n is K (n % 8 < 4) or V of 32 keys of tile n / 8 ------------
    const int tasks = 8 * k.left;
    int n = warp - kSoftWarps;
    Walk nx = k;             // at the tile of task `seen`, the next to be looked up
    int nxx = k.left > 0 ? k.x : 0, seen = n;
    const int psl = a.pool.ps_log2, psm = (1 << psl) - 1;
    const uint32_t page_codes = static_cast<uint32_t>(a.pool.heads) * (D / 2) << psl;   // bytes of a page in a codes array
    const uint32_t page_meta = static_cast<uint32_t>(a.pool.heads) * (4 * NG) << psl;   // and in a (min or scale) array
    // the segment's table row, its head's first row in a page, and the keys that its rows see
    const int32_t* row = nullptr;
    int head_row = 0, last = -1, lo = 0;
    auto enter = [&]() {
      row = MODE == kPrefix ? a.tab.table + a.prefix.leader[nx.i] * a.tab.stride : a.tab.table + nx.i * a.tab.stride + nx.s.off;
      head_row = nx.h << psl;
      last = min(nx.un.p1, nx.s.keys - 1);
      lo = a.shape.window > 0 && nx.un.p0 >= a.shape.window ? nx.un.p0 - a.shape.window + 1 : 0;
    };
    // The segment's rows of Q on their way into L2, by one warp, two tiles before the softmax warps read them.
    auto fetch_q = [&]() {
      if (warp != kSoftWarps) return;
      const int base = nx.h * a.shape.group;
      for (int r = lane; r < nx.un.rows; r += 32) {
        const int row_ = nx.un.r0 + r, t = row_ / a.shape.group;
        const __half* p = a.q + static_cast<int64_t>(MODE == kPrefix ? listed_row(a.prefix, a.batch, a.prefix.order[nx.s.row0 + t]) : nx.s.row0 + t) * a.ldq + static_cast<int64_t>(base + row_ - t * a.shape.group) * D;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
        if (D == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + 64));
      }
    };
    if (tasks > 0) {
      enter();
      fetch_q();
    }
    // the lane's key of task `seen`: the table's entry (not looked at before the load below) and its row in a page (-1: no
    // row of the unit sees the key)
    auto look_up = [&](int& page, int& off) {
      page = off = -1;
      if (seen >= tasks) return;
      const int j = (nx.sp.tile(nxx) << kKeysLog2) + 32 * (seen & 3) + lane;
      if (j <= last && (j >= lo || j < a.shape.sinks)) {
        page = row[j >> psl];
        off = head_row + (j & psm);
      }
      // on by 7 tasks: a tile further, unless the task was a tile's first
      if ((seen & 7) != 0 && ++nxx == nx.x1) {
        walk_next<MODE>(nx, a, line);
        nxx = nx.x;
        if (nx.left > 0) {
          enter();
          fetch_q();
        }
      }
      seen += kRestoreWarps;
    };
    // K's task loads the scales of V too: it writes the tile's flags
    auto load = [&](Raw<NG>& v, bool value, int page, int off) {
#pragma unroll
      for (int g = 0; g < NG; ++g) v.scale[g] = v.mn[g] = v.vscale[g] = 0.0f;
      v.absent = false;
      if (off >= 0 && static_cast<uint32_t>(page) < static_cast<uint32_t>(a.tab.pages)) {
        const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(page)) * page_codes + static_cast<uint32_t>(off) * (D / 2);
        const uint64_t am = static_cast<uint64_t>(static_cast<uint32_t>(page)) * page_meta + static_cast<uint32_t>(off) * (4 * NG);
        const uint4* c = reinterpret_cast<const uint4*>((value ? a.pool.codes[1] : a.pool.codes[0]) + at);
#pragma unroll
        for (int e = 0; e < 2 * NG; ++e) v.code[e] = c[e];
        load_meta(v.scale, value ? a.pool.scales[1] : a.pool.scales[0], am);
        load_meta(v.mn, value ? a.pool.mins[1] : a.pool.mins[0], am);
        if (!value) load_meta(v.vscale, a.pool.scales[1], am);
      } else {
#pragma unroll
        for (int e = 0; e < 2 * NG; ++e) v.code[e] = make_uint4(0u, 0u, 0u, 0u);
        if (off >= 0) {
          v.absent = true;
          atomicOr(a.batch.err, DEV_ERR_PAGE);
        }
      }
    };
    auto restore = [&](Raw<NG>& v) {   // task n
      const int g = n >> 3, st = g & 1, quarter = n & 3, r = 32 * quarter + lane;
      const bool value = n & 4;
      const int c = value ? g - 1 : g - 2;   // the release that frees the place
      bool ok = g < 2 || mbar_wait(&freed[c & 1], (c >> 1) & 1, wait_limit, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return false;
      if (value) {
#pragma unroll
        for (int q = 0; q < NG; ++q)
          if (!(fabsf(v.scale[q]) < INFINITY)) v.scale[q] = v.mn[q] = 0.0f;   // such a group is NaN: see its flag
      } else {
        // A slot of the ring of four is free: S of tile g - 2 is complete, so every softmax warp is past tile g - 4.
        uint32_t* f = sFlags + (g & 3) * 16 + quarter;
        const uint32_t absent = __ballot_sync(0xffffffffu, v.absent);
        const uint32_t nan0 = __ballot_sync(0xffffffffu, !(fabsf(v.vscale[0]) < INFINITY));
        const uint32_t nan1 = __ballot_sync(0xffffffffu, !(fabsf(v.vscale[NG - 1]) < INFINITY));
        if (lane == 0) {
          f[0] = absent | nan0 | nan1;
          f[4] = absent;
          f[8] = nan0;
          f[12] = NG == 2 ? nan1 : 0u;
        }
      }
      uint8_t* p = sKV + st * S::kStage + (value ? S::kK : 0) + r * 128;
#pragma unroll
      for (int q = 0; q < NG; ++q) restore_group(v.code[2 * q], v.code[2 * q + 1], v.scale[q], v.mn[q], p + q * S::kPanel, r);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(value ? &vfull[st] : &kfull[st]);
      return true;
    };
    Raw<NG> v;
    int page, off;
    look_up(page, off);
    load(v, n & 4, page, off);
    look_up(page, off);
    while (n < tasks && restore(v)) {
      n += kRestoreWarps;
      load(v, n & 4, page, off);   // on its way while the warp waits for the task's place
      look_up(page, off);
    }
  } else if (warp == kMmaWarp) {
    // ---- MMA issuer --------------------------------------------------------------------
    if (lane == 0) {
      const uint64_t kd = smem_desc_sw128(smem_u32(sKV), 16, 1024), vd = smem_desc_sw128(smem_u32(sKV) + S::kK, S::kPanel, 1024);
      const uint32_t q_lo = static_cast<uint32_t>(smem_desc_sw128(smem_u32(sQ), 16, 1024)), k_lo = static_cast<uint32_t>(kd);
      const uint32_t k_hi = static_cast<uint32_t>(kd >> 32), v_lo = static_cast<uint32_t>(vd), v_hi = static_cast<uint32_t>(vd >> 32);
      auto issue_s = [&](int grp, int g) {
        const uint32_t qa = q_lo + grp * (S::kQ >> 4), ka = k_lo + (g & 1) * (S::kStage >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk / 4) * S::kPanel + (kk % 4) * 32) >> 4;
          mma_ss(tmem + 128 * grp, qa + off, ka + off, k_hi, kIdescS, kk > 0);
        }
        mbar_arrive(&sfull[grp]);
        mma_commit(&sfull[grp]);
      };
      auto issue_o = [&](int grp, int g, bool first) {
        const uint32_t va = v_lo + (g & 1) * (S::kStage >> 4), pa = tmem + kP + kPStep * grp;
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          mma_ts(tmem + kO + D * grp, pa + 8 * kk, va + kk * (2048 >> 4), v_hi, kIdescO, (!first || kk > 0) ? 1u : 0u);
      };
      bool ok = true;
      int g = 0, gb = 0, n = 0, nb = 0;   // tiles and segments, of group 1 too
      auto wait = [&](uint64_t* bar, int phase) {
        if (ok) ok = mbar_wait(bar, phase & 1, wait_limit, abort_flag);
        return ok;
      };
      // A wait takes some 250 cycles even where it is over (the MMAs' operand reads fill shared memory) and an MMA is taken
      // every 64, few of them ahead: so the next batch's barrier is looked at before a batch is issued, and waited for after
      // it only where it was not over yet.
      auto look = [&](uint64_t* bar, int phase) { return mbar_test(bar, phase & 1); };
      while (k.left > 0 && ok) {
        const bool two = k.un.rows > 128;
        if (!wait(&qfull[0], n) || !wait(&kfull[g & 1], g >> 1)) break;
        tc_fence_after();
        issue_s(0, g);
        if (two) {
          if (!wait(&qfull[1], nb)) break;
          tc_fence_after();
          issue_s(1, g);
        }
        mma_commit(&freed[g & 1]);
        if (!wait(&vfull[g & 1], g >> 1)) break;
        for (int x = k.x; x < k.x1 && ok; ++x, ++g) {
          const bool first = x == k.x, last = x + 1 == k.x1;
          if (!wait(&pfull[0], g)) break;
          tc_fence_after();
          const uint32_t k_in = last ? 1u : look(&kfull[(g + 1) & 1], (g + 1) >> 1);
          issue_o(0, g, first);
          const uint32_t p_in = two ? look(&pfull[1], gb) : 1u;
          if (last) {
            mma_commit(&odone[0]);
          } else {
            if (!k_in && !wait(&kfull[(g + 1) & 1], (g + 1) >> 1)) break;
            tc_fence_after();
            issue_s(0, g + 1);
          }
          const uint32_t v_in = last ? 1u : look(&vfull[(g + 1) & 1], (g + 1) >> 1);
          if (two) {
            if (!p_in && !wait(&pfull[1], gb)) break;
            tc_fence_after();
            issue_o(1, g, first);
            if (last) mma_commit(&odone[1]);
            else issue_s(1, g + 1);
            ++gb;
          }
          if (!last) {
            mma_commit(&freed[(g + 1) & 1]);
            if (!v_in && !wait(&vfull[(g + 1) & 1], (g + 1) >> 1)) break;
          }
        }
        ++n;
        nb += two;
        walk_next<MODE>(k, a, line);
      }
      mma_commit(done);
    }
    __syncwarp();
  } else {
    // ---- softmax warps: row r of group grp -------------------------------------------------
    const int grp = warp >> 2, quarter = warp & 3;
    const int rr = 32 * quarter + lane, r = 128 * grp + rr;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    const uint32_t ts = trow + 128 * grp, to = trow + kO + D * grp, tp = trow + kP + kPStep * grp;
    // A warp brings its 32 rows of Q into shared memory a row over kPieces lanes, 16 bytes each.
    constexpr int kPieces = D / 8, kAtOnce = 32 / kPieces;
    const int pc = lane % kPieces, row_w = r - lane;
    uint8_t* const qt = sQ + grp * S::kQ + 32 * quarter * 128;
    auto piece = [&](int n) { return reinterpret_cast<uint4*>(qt + (pc >> 3) * S::kPanel + n * 128 + (((pc & 7) ^ (n & 7)) << 4)); };
    // where the lane's row begins in rows ld apart
    auto place = [&](int64_t ld) {
      const int row = k.un.r0 + (r < k.un.rows ? r : 0), tok = row / a.shape.group;
      return (MODE == kPrefix ? listed_row(a.prefix, a.batch, a.prefix.order[k.s.row0 + tok]) : k.s.row0 + tok) * ld + static_cast<int64_t>(k.h * a.shape.group + row - tok * a.shape.group) * D;
    };
    uint8_t* const stage = sOut + warp * S::kOut;
    bool ok = true;
    int4 rec = make_int4(-1, 0, 0, 0);
    int g0 = 0;            // the CTA's tiles before the segment
    int cnt = 0, seg = 0;  // this group's tiles and segments
    // the segment that ends: its rows, sums, and where they go
    bool whole_item = false, from_start = false;
    int rows = -1;         // -1: none
    int64_t dst = 0;
    float m = -INFINITY;
    float2 l2 = make_float2(0.0f, 0.0f);
    uint32_t nans = 0;
    int home = -1;         // kBehind: where the row's shared prefix left its sums (rows times heads are below 2^31)
    while (true) {
      // A round ends one segment and works on the next.  S of the last tile is complete, so Q's place is free: the next Q is
      // on its way while the last P V runs, and its first S runs while O is written.
      while (k.left > 0 && grp == 1 && k.un.rows <= 128) {
        g0 += k.x1 - k.x;
        walk_next<MODE>(k, a, line);
      }
      const bool more = k.left > 0;
      if (more) {
        const int64_t src = place(a.ldq);
        // (loops here and below: code that runs once a segment is fetched anew each time, and straight code costs its length)
#pragma unroll 2
        for (int i = 0; i < 32; i += kAtOnce) {
          const int n = i + lane / kPieces;
          const __half* from = a.q + __shfl_sync(0xffffffffu, src, n) + 8 * pc;
          cp16_zfill(smem_u32(piece(n)), from, row_w + n < k.un.rows);
        }
        cp_async_commit();
      }
      if (rows >= 0) {
        ok = mbar_wait(&odone[grp], seg & 1, kDrainLimit, abort_flag);   // of an MMA that the issuer is at: it gives up, or this comes
        ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        if (!ok) break;
        ++seg;
        tc_fence_after();
      }
      if (more) {   // Q has every 8 dims in the order (0, 4), (1, 5), (2, 6), (3, 7): a lane's own pieces
        cp_async_wait<0>();
#pragma unroll 2
        for (int i = 0; i < 32; i += kAtOnce) {
          uint4* q = piece(i + lane / kPieces);
          const uint4 v = *q;
          *q = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                          __byte_perm(v.y, v.w, 0x7632));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&qfull[grp]);
        __syncwarp();   // collective loads follow
      }
      if (rows >= 0) {
        // ---- the segment's rows: finished, or this share's partial ------------------------
        float l = l2.x + l2.y;
        float own = 1.0f, other = 0.0f;   // factors of its own sums and of its prefix's
        if (MODE == kBehind && home >= 0) {
          const float2 st = a.prefix.home_stat[home];
          const float top = fmaxf(m, st.x), base = top == -INFINITY ? 0.0f : top;
          own = exp2f(m - base);
          other = exp2f(st.x - base);
          l = l * own + st.y * other;
          m = top;
        }
        const float f = !whole_item ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t slot = (static_cast<int64_t>(w) * 2 + (from_start ? 1 : 0)) * kRows + row_w;   // of the warp's first row
        float* const parts = MODE != kPrefix ? pl.part + slot * D : from_start ? a.prefix.home : a.prefix.extra;   // kPrefix: dst is the lane's row
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t u[32];
          tmem_ld_32x32b_x32(to + 32 * c, u);
          tmem_arrived(u);
          const float fc = (nans >> (c >> 1)) & 1u ? __uint_as_float(0x7fffffffu) : f;   // a NaN group's columns
          float v[32];         // of 8 columns dims 0..7 lie at 0, 2, 4, 6, 1, 3, 5, 7
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(u[(e & 24) + ((e & 7) < 4 ? 2 * (e & 7) : 2 * (e & 7) - 7)]) * (MODE == kBehind ? fc * own : fc);
          if (MODE == kBehind) {
            if (home >= 0) {
              const float* x = a.prefix.home + static_cast<int64_t>(home) * D + 32 * c;
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 y = *reinterpret_cast<const float4*>(x + e);
                v[e] = fmaf(y.x, other * f, v[e]);
                v[e + 1] = fmaf(y.y, other * f, v[e + 1]);
                v[e + 2] = fmaf(y.z, other * f, v[e + 2]);
                v[e + 3] = fmaf(y.w, other * f, v[e + 3]);
              }
            }
            __syncwarp();   // collective loads follow
          }
          if (whole_item) {
            if (r < rows) {
              uint4* out = reinterpret_cast<uint4*>(a.out + dst + 32 * c);
#pragma unroll
              for (int e = 0; e < 32; e += 8)
                out[e / 8] = make_uint4(q4::cvt_f16x2(make_float2(v[e], v[e + 1])), q4::cvt_f16x2(make_float2(v[e + 2], v[e + 3])),
                                        q4::cvt_f16x2(make_float2(v[e + 4], v[e + 5])), q4::cvt_f16x2(make_float2(v[e + 6], v[e + 7])));
            }
            __syncwarp();   // the next round begins with a collective load
            continue;
          }
          // A partial's 32 columns go through shared memory and leave eight lanes a row: a row a lane takes a line of the L1
          // per lane and store (8500 cycles for the partial, 6500 to 7900 this way; whole rows, half the bytes and no
          // second pass, are faster straight out).
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                make_uint4(__float_as_uint(v[4 * e]), __float_as_uint(v[4 * e + 1]), __float_as_uint(v[4 * e + 2]), __float_as_uint(v[4 * e + 3]));
          __syncwarp();
#pragma unroll 4
          for (int i = 0; i < 32; i += 4) {
            const int n = i + (lane >> 3);
            const uint4 x = *reinterpret_cast<const uint4*>(stage + n * 128 + (((lane & 7) ^ (n & 7)) << 4));
            const int64_t to = MODE == kPrefix ? __shfl_sync(0xffffffffu, dst, n) : n;
            if (row_w + n < rows) *reinterpret_cast<uint4*>(parts + to * D + 32 * c + 4 * (lane & 7)) = x;
          }
          __syncwarp();
        }
        if (!whole_item && r < rows) (MODE != kPrefix ? pl.stat + slot : from_start ? a.prefix.home_stat : a.prefix.extra_stat)[MODE == kPrefix ? dst : lane] = make_float2(m, l);
      }
      if (!more) break;
      const int tiles = k.x1 - k.x;
      const bool on = r < k.un.rows;
      const int p = k.s.len - k.s.n + (k.un.r0 + (on ? r : 0)) / a.shape.group;   // the row's position
      const int whole_hi = min(k.un.p0, k.s.keys - 1) - (kKeys - 1), sink_hi = a.shape.sinks - kKeys;
      const int whole_lo = a.shape.window > 0 ? k.un.p1 - a.shape.window + 1 : 0;
      m = -INFINITY;
      l2 = make_float2(0.0f, 0.0f);
      nans = 0;
      for (int x = 0; x < tiles; ++x, ++cnt) {
        // tcgen05.ld/st are warp-collective: every branch around them is taken by the whole warp
        ok = mbar_wait(&sfull[grp], cnt & 1, wait_limit, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const int t0 = k.sp.tile(k.x + x) << kKeysLog2;
        const uint32_t* flags = sFlags + ((g0 + x) & 3) * 16;
        const uint4 any = *reinterpret_cast<const uint4*>(flags);
        const bool odd = (any.x | any.y | any.z | any.w) != 0;
        // every row of the unit sees all of the tile
        const bool whole = !odd && t0 <= whole_hi && (t0 >= whole_lo || t0 <= sink_hi);
        uint32_t see[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        if (!whole) {
          const int hi = min(p, k.s.keys - 1) - t0 + 1;                               // columns below it are not later than the row
          const int lo = a.shape.window > 0 && p >= a.shape.window ? p - a.shape.window + 1 - t0 : 0;   // columns below it lie behind the window
          const int sk = a.shape.sinks - t0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            see[c] = bits_below(hi - 32 * c) & (~bits_below(lo - 32 * c) | bits_below(sk - 32 * c)) & ~flags[4 + c];
            nans |= ((see[c] & flags[8 + c]) ? 1u : 0u) | ((see[c] & flags[12 + c]) ? 2u : 0u);
          }
        }
        if (!whole) {   // what the row does not see becomes -inf, in place
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t u[32];
            tmem_ld_32x32b_x32(ts + 32 * c, u);
            tmem_arrived(u);
            const uint32_t word = c == 0 ? see[0] : c == 1 ? see[1] : c == 2 ? see[2] : see[3];
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((word >> e) & 1u)) u[e] = 0xff800000u;
            tmem_st_32x32b_x32(ts + 32 * c, u);
          }
          tmem_st_wait();
        }
        // P = 2^(s - m) for the m known so far.  A segment's first tile finds m; a later one takes it as it is and
        // looks at the row's sum only: while that stays below kMostSum no weight has left fp16, and a larger maximum changes
        // nothing but the scale of sums that are divided in the end.  Otherwise (or with no key seen before) the tile finds
        // its maximum, the sums are rescaled, and the weights are formed again.
        uint32_t pk[64];
        float2 lt = make_float2(0.0f, 0.0f);
        bool find = x == 0;
        while (true) {
          if (find) {
            float mx = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t u[32];
              tmem_ld_32x32b_x32(ts + 32 * c, u);
              tmem_arrived(u);
              float m4[4] = {mx, mx, mx, mx};
#pragma unroll
              for (int e = 0; e < 32; e += 8)
#pragma unroll
                for (int q = 0; q < 4; ++q) m4[q] = fmaxf(m4[q], fmaxf(__uint_as_float(u[e + 2 * q]), __uint_as_float(u[e + 2 * q + 1])));
              mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            }
            // only for a row that asks: its bits do not depend on its neighbours
            mx = x == 0 || m == -INFINITY || !(lt.x + lt.y <= kMostSum) ? fmaxf(m, fmaf(mx, a.scale_log2, -kLift)) : m;
            if (x > 0) {
              const float alpha = mx == -INFINITY ? 1.0f : ex2_approx(m - mx);
              l2 = make_float2(l2.x * alpha, l2.y * alpha);
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t u[16];
                tmem_ld_32x32b_x16(to + 16 * c, u);
                tmem_arrived(u);
#pragma unroll
                for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * alpha);
                tmem_st_32x32b_x16(to + 16 * c, u);
              }
            }
            m = mx;
          }
          const float negm = m == -INFINITY ? 0.0f : -m;
          const float2 sc2 = make_float2(a.scale_log2, a.scale_log2), nm2 = make_float2(negm, negm);
          lt = make_float2(0.0f, 0.0f);
          float2 lb = lt;
          uint32_t ua[16], ub[16];
          auto weigh = [&](const uint32_t (&u)[16], int c) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float2 v = q4::fma_f32x2(make_float2(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1])), sc2, nm2);
              v = make_float2(ex2_approx(v.x), ex2_approx(v.y));
              if (e & 1) lb = add_f32x2(lb, v);
              else lt = add_f32x2(lt, v);
              pk[8 * c + e] = q4::cvt_f16x2(v);
            }
          };
          tmem_ld_32x32b_x16(ts, ua);
#pragma unroll
          for (int c = 0; c < 8; c += 2) {   // a load runs under the chunk before it
            tmem_arrived(ua);
            tmem_ld_32x32b_x16(ts + 16 * c + 16, ub);
            weigh(ua, c);
            tmem_arrived(ub);
            if (c < 6) tmem_ld_32x32b_x16(ts + 16 * c + 32, ua);
            weigh(ub, c + 1);
          }
          lt = add_f32x2(lt, lb);
          const bool again = !find && __any_sync(0xffffffffu, m == -INFINITY || !(lt.x + lt.y <= kMostSum));
          if (!again) break;
          find = true;
        }
        l2 = add_f32x2(l2, lt);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_st_32x32b_x16(tp + 16 * c, *reinterpret_cast<const uint32_t(*)[16]>(pk + 16 * c));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[grp]);
      }
      if (!ok) break;
      from_start = k.x == 0;
      whole_item = MODE != kPrefix && from_start && k.x1 == k.sp.n;
      rows = k.un.rows;
      if (MODE == kPrefix) {
        const int row = k.un.r0 + (r < rows ? r : 0), t = row / a.shape.group;
        dst = from_start ? static_cast<int64_t>(a.prefix.order[k.s.row0 + t]) * a.q_heads + k.h * a.shape.group + row - t * a.shape.group
                         : a.prefix.info[a.tab.seqs + k.i].extra + static_cast<int64_t>(w) * kRows + r;
      } else {
        dst = place(a.ldo);
      }
      if (MODE == kBehind) {
        home = -1;
        if (from_start && r < rows && a.tab.skip[k.i] > 0) {
          const int row = k.un.r0 + r, t = row / a.shape.group;
          home = static_cast<int>(prefix_home(a.prefix, k.i, t, k.h * a.shape.group + row - t * a.shape.group, a.q_heads));
        }
        __syncwarp();
      }
      if (MODE != kPrefix && from_start && !whole_item) {
        // the item's first tile in the line: the share's first tiles, then those of the segments before it
        const int64_t per = line.per, start = w * per + g0;
        rec = make_int4(k.i, k.h, k.u, static_cast<int>((start + k.sp.n - 1) / per));
      }
      g0 += tiles;
      walk_next<MODE>(k, a, line);
    }
    cp_async_wait<0>();   // none is left in flight where a wait ran out
    if (MODE != kPrefix && threadIdx.x == 0) pl.rec[w] = rec;
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

template <int D, int MODE>
fg_status launch_kernel(const AttnArgs<__half>& a, const ClassPlan& pl, bool own_plan, bool every, cudaStream_t st) {
  using S = Smem<D>;
  static bool set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !set[dev]) {
    if (cudaFuncSetAttribute(tile_kernel<D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes) != cudaSuccess)
      return check_launch("tile_kernel smem attribute");
    set[dev] = true;
  }
  Trace tr(KC_ATTN_PAGED, st);
  // Early behind the plan alone.  As a call's first launch or behind the steps the CTAs then would not take the SMs in
  // order, so that neighbours in the line share a head's keys in L2 (a chunk of 2048 rows 459 us, 464 early; 63 single
  // tokens beside a chunk of 512 362 and 367).
  return paged::launch("tile_kernel", every && !own_plan, tile_kernel<D, MODE>, static_cast<unsigned>(pl.workers), kThreads, S::kBytes, st, a, pl, wait_limit(), own_plan, every);
}

template <int D>
fg_status launch(const AttnArgs<__half>& a, const ClassPlan& pl, bool own_plan, bool every, cudaStream_t st) {
  return a.tab.skip != nullptr ? launch_kernel<D, kBehind>(a, pl, own_plan, every, st) : launch_kernel<D, kAlone>(a, pl, own_plan, every, st);
}

}  // namespace

fg_status paged_attention_tile(const AttnArgs<__half>& a, const ClassPlan& pl, int head_dim, bool own_plan, bool every, cudaStream_t st) {
  return head_dim == 128 ? launch<128>(a, pl, own_plan, every, st) : launch<64>(a, pl, own_plan, every, st);
}

fg_status paged_prefix_tile(const AttnArgs<__half>& a, const ClassPlan& pl, int head_dim, cudaStream_t st) {
  return head_dim == 128 ? launch_kernel<128, kPrefix>(a, pl, false, true, st) : launch_kernel<64, kPrefix>(a, pl, false, true, st);
}

}  // namespace paged
}  // namespace fg
