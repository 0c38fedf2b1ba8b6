// How the paged attention's work is dealt out.
//
// An item is one unit of rows of one sequence (RU rows, the query heads of a
// K/V head side by side: row t * group + g) against the keys it sees, for one
// K/V head; its cost is a number of key tiles (KT keys).  All items in a line,
// sequence by sequence, head by head, unit by unit, make T tiles, and worker w
// takes tiles [w * per, (w + 1) * per): equal work whatever the lengths are,
// and neighbouring workers read the same head's keys.  An item inside one
// worker's share is finished there; one that crosses shares leaves a partial
// (sums, maximum and normaliser) with each, joined in order afterwards.  A
// worker's first segment goes to its slot 0 when it began before, its last to
// slot 1 when it ends later, so two slots a worker are enough.
#pragma once

#include <stdint.h>

#include "paged.cuh"

namespace fg {
namespace paged {

// Sequences with at most this many rows (rows times group) are steps: the
// warp-level kernel takes them (a warp holds 8 or 16 rows); longer ones go to
// the tile kernels, whose units are 256 rows.  At 16 rows (8 K/V heads of 128, 4
// tokens of 4 query heads each): 32 sequences of 4000 tokens 67 us as steps,
// 122 to 125 as chunks (head_dim 64: 44 and 103), 4 sequences of 500 tokens 15.9
// and 20.2 us; the chunks' kernel is ahead only for one long sequence (30000
// tokens 62.7 and 53.5).
constexpr int kStepRows = 16;
constexpr int kMaxSplits = 128;   // shares an item may cross (the join reads them one after another)

struct AttnShape {
  int group;            // query heads per K/V head
  int max_q;
  int window, sinks;    // window 0: none; both at most 2^30
};

// What a class of items shares: header and prefix sums written by the plan.
struct ClassPlan {
  int64_t* head;        // [0] tiles in all, [1] tiles of a share
  int64_t* pre;         // [seqs + 1] tiles before sequence i
  int4* rec;            // [workers] the item that begins in a share and ends later: (sequence or -1, head, unit, last share)
  float* part;          // [workers][2][rows][D] sums
  float2* stat;         // [workers][2][rows] (maximum, normaliser)
  int rows;             // rows of a slot
  int workers;
};

// Key tiles that the rows at positions p0 .. p1 see: the first ns, then those
// from t0 on; n in all, at least one (a unit that sees nothing still writes its
// zeros).
struct Span {
  int ns, t0, n;
  __device__ __forceinline__ int tile(int x) const { return x < ns ? x : t0 + x - ns; }
};
template <int KTL>
__device__ __forceinline__ Span span_of(int p0, int p1, int keys, int window, int sinks) {
  const int last = p1 < keys - 1 ? p1 : keys - 1;
  Span s{0, 0, 1};
  if (last < 0) return s;
  int lo = window > 0 && p0 >= window ? p0 - window + 1 : 0;
  lo = lo < last ? lo : last;
  const int t1 = last >> KTL, t0 = lo >> KTL;
  const int se = sinks < last + 1 ? sinks : last + 1;
  const int ns = (se + (1 << KTL) - 1) >> KTL;
  if (window == 0 || ns >= t0) {
    s.n = t1 + 1;
  } else {
    s.ns = ns;
    s.t0 = t0;
    s.n = ns + t1 - t0 + 1;
  }
  return s;
}

// Unit u of a sequence: its rows and their positions.
struct Unit {
  int r0, rows;         // rows r0 .. r0 + rows - 1 of the sequence's n * group
  int p0, p1;
};
template <int RU>
__device__ __forceinline__ Unit unit_of(const Seq& s, int group, int u) {
  Unit x;
  const int64_t all = static_cast<int64_t>(s.n) * group;
  x.r0 = u * RU;
  x.rows = static_cast<int>(all - x.r0 < RU ? all - x.r0 : RU);
  const int base = s.len - s.n;
  x.p0 = base + x.r0 / group;
  x.p1 = base + (x.r0 + x.rows - 1) / group;
  return x;
}

// Tiles of a step (a sequence of at most kStepRows rows) for one K/V head.
constexpr int kStepTileLog2 = 5;
__device__ __forceinline__ int step_tiles(const Seq& s, const AttnShape& sh) {
  return span_of<kStepTileLog2>(s.len - s.n, s.len - 1, s.keys, sh.window, sh.sinks).n;
}
// Tiles of a share: equal shares, but no item over more than kMaxSplits of
// them, and at least `few`.
__device__ __forceinline__ int64_t share_of(int64_t total, int longest, int workers, int few) {
  const int64_t a = (total + workers - 1) / workers, b = (longest + kMaxSplits - 1) / kMaxSplits;
  const int64_t c = a > b ? a : b;
  return c > few ? c : few;
}
constexpr int kStepFew = 2;   // a step's share: at least 64 tokens, so that a warp's copies of one tile run under another's sums

// Tiles of a sequence's units for one K/V head, every `stride`-th from u0 on.
template <int RU, int KTL>
__device__ __forceinline__ int64_t units_tiles(const Seq& s, const AttnShape& sh, int u0, int stride) {
  const int64_t all = static_cast<int64_t>(s.n) * sh.group;
  const int units = static_cast<int>((all + RU - 1) / RU);
  int64_t c = 0;
  for (int u = u0; u < units; u += stride) {
    const Unit x = unit_of<RU>(s, sh.group, u);
    c += span_of<KTL>(x.p0, x.p1, s.keys, sh.window, sh.sinks).n;
  }
  return c;
}
// The most tiles that a unit of the sequence may see: the last one's, but for a
// few where it is short and a window cuts them all.
template <int RU, int KTL>
__device__ __forceinline__ int longest_unit(const Seq& s, const AttnShape& sh) {
  const Unit x = unit_of<RU>(s, sh.group, static_cast<int>((static_cast<int64_t>(s.n) * sh.group - 1) / RU));
  return span_of<KTL>(x.p0, x.p1, s.keys, sh.window, sh.sinks).n + 4;
}

// Where a kernel reads its class's line.
struct Line {
  const int64_t* pre;
  int64_t total, per;
};
// Calls over at most kOwnPlan sequences make the line in every CTA, by all its
// warps, instead of by a launch before: step (at most kStepRows rows) or tile
// class of a call that has both, or all sequences (`every`).  Steps of 64
// sequences 21.9 us this way and 23.9 with the launch, of 128 30.8 and 33.0;
// chunks of 20 rows of 64 sequences 63.8 and 65.6, of 128 105.9 and 107.3.
constexpr int kOwnPlan = 128;
struct OwnPlan {
  int64_t pre[kOwnPlan + 1];
  int64_t per;
  int longest;
};
template <bool STEP, int RU, int KTL>
__device__ __forceinline__ Line make_line(OwnPlan& o, const Table& t, const Batch& b, const AttnShape& sh, int heads, int workers,
                                          bool every) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if (threadIdx.x == 0) o.longest = 0;
  __syncthreads();
  for (int i0 = warp; i0 < t.seqs; i0 += 32 * nw) {   // a lane a sequence, the warps in turn (a warp counts its chunks one by one)
    const int i = i0 + nw * lane;
    Seq s{0, 0, 0, 0};
    if (i < t.seqs) {
      s = seq_of(t, b, i);
      if (s.n > sh.max_q) {
        if (blockIdx.x == 0) atomicOr(b.err, DEV_ERR_BATCH);
        s.n = 0;
      }
    }
    const bool step = static_cast<int64_t>(s.n) * sh.group <= kStepRows;
    const bool on = s.n > 0 && (every || step == STEP);
    int64_t mine = 0;
    if (STEP) {
      if (on) mine = step_tiles(s, sh);
      if (on) atomicMax(&o.longest, static_cast<int>(mine));
    } else {
      if (on) atomicMax(&o.longest, longest_unit<RU, KTL>(s, sh));
      uint32_t todo = __ballot_sync(0xffffffffu, on);
      while (todo) {                                       // a chunk's units: the lanes together
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        Seq c{0, 0, 0, 0};
        c.n = __shfl_sync(0xffffffffu, s.n, src);
        c.len = __shfl_sync(0xffffffffu, s.len, src);
        c.keys = __shfl_sync(0xffffffffu, s.keys, src);
        int64_t tiles = units_tiles<RU, KTL>(c, sh, lane, 32);
#pragma unroll
        for (int f = 16; f > 0; f >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, f);
        if (lane == src) mine = tiles;
      }
    }
    if (i < t.seqs) o.pre[i] = mine * heads;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t at = 0;
    for (int i0 = 0; i0 < t.seqs; i0 += 32) {
      const int i = i0 + lane;
      const int64_t c = i < t.seqs ? o.pre[i] : 0;
      int64_t inc = c;
#pragma unroll
      for (int f = 1; f < 32; f <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, inc, f);
        if (lane >= f) inc += up;
      }
      if (i < t.seqs) o.pre[i] = at + inc - c;
      at += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
      o.pre[t.seqs] = at;
      o.per = share_of(at, o.longest, workers, STEP ? kStepFew : 1);
    }
  }
  __syncthreads();
  return Line{o.pre, o.pre[t.seqs], o.per};
}

}  // namespace paged
}  // namespace fg
