// Paged attention with fp32 activations (FlexGen notes, "背景知识": Softmax(x_Q
// x_K^T / sqrt(h1)) x_V per head, causal; "5. 近似方法": K and V stored in 4-bit
// groups of 64), on the CUDA cores: everything in fp32, K and V restored as
// fmaf(q, scale, min).
//
// A unit is 16 rows of one K/V head; a CTA of 128 threads walks its share of
// the line of tiles (paged_sched.cuh), 64 keys a tile.  A thread restores one K
// or one V row of the tile (its codes loaded a tile ahead) into shared memory;
// then half a warp owns two rows: 2 x 4 scores a thread (keys 16 apart, so that
// the rows it reads lie four banks apart), the running maximum and sum over the
// half warp, the weights through shared memory, and 2 x D/16 outputs a thread.
// Bound by the FMAs' operands: ten shared-memory wavefronts for 32 FMAs a warp.
// 3 sequences of 300 to 777 tokens, 5 to 67 rows, 12 heads of 64: 23.9 us by
// graph replay, two tiles a CTA of 8 to 10 thousand cycles each; the rest is
// launch, plan and the first loads (9000 cycles) and the join.
#include <math.h>

#include "paged_attn.cuh"
#include "q4_dev.cuh"
#include "tc_ptx.cuh"

namespace fg {
namespace paged {
namespace {

constexpr int kKeysLog2 = kF32KeysLog2;
constexpr int kKeys = 1 << kKeysLog2;
constexpr int kRows = kF32Rows;
constexpr int kThreads = 128;
static_assert(kKeys == 64 && kRows == 16, "the thread layout below");

template <int D>
struct Smem {
  static constexpr int kRow = D + 4;          // floats; rows start four banks apart
  float q[kRows][kRow];
  float k[kKeys][kRow];
  float v[kKeys][kRow];
  float p[kRows][kKeys + 4];
  uint32_t absent[2], nan[2][2];              // keys of the tile: no page; value group g is NaN
};

template <int D>
__global__ void __launch_bounds__(kThreads) f32_kernel(const AttnArgs<float> a, const ClassPlan pl, const bool own_plan) {
  constexpr int NG = D / 64, CW = D / 16;     // output columns of a thread: 4 (cx + 16 i), i < D / 64
  extern __shared__ __align__(16) uint8_t raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
  const int tid = threadIdx.x, lane = tid & 31;
  const int ry = tid >> 4, cx = tid & 15;     // rows 2 ry, 2 ry + 1
  const int w = blockIdx.x;

  tc::griddep_launch();
  tc::griddep_wait();
  __shared__ OwnPlan own;
  const Line line = own_plan ? make_line<false, kRows, kKeysLog2>(own, a.tab, a.batch, a.shape, a.pool.heads, pl.workers, true)
                             : Line{pl.pre, pl.head[0], pl.head[1]};
  const int64_t total = line.total, per = line.per, o0 = w * per;
  if (o0 >= total) {
    if (tid == 0) pl.rec[w] = make_int4(-1, 0, 0, 0);
    return;
  }
  // the share's first segment
  int i, h, u, x, left, units;
  Seq s;
  Unit un;
  Span sp;
  auto enter_unit = [&]() {
    un = unit_of<kRows>(s, a.shape.group, u);
    sp = span_of<kKeysLog2>(un.p0, un.p1, s.keys, a.shape.window, a.shape.sinks);
  };
  auto enter_seq = [&]() {
    s = seq_of(a.tab, a.batch, i);
    units = static_cast<int>((static_cast<int64_t>(s.n) * a.shape.group + kRows - 1) / kRows);
    u = 0;
  };
  {
    int lo = 0, hi = a.tab.seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (line.pre[mid] <= o0) lo = mid;
      else hi = mid;
    }
    i = lo;
    left = static_cast<int>(total - o0 < per ? total - o0 : per);
    enter_seq();
    const int64_t all = line.pre[lo + 1] - line.pre[lo], in = o0 - line.pre[lo];   // (32-bit divisions where they do: the short ones)
    const int64_t cost = all <= INT32_MAX ? static_cast<int>(all) / a.pool.heads : all / a.pool.heads;
    h = all <= INT32_MAX ? static_cast<int>(in) / static_cast<int>(cost) : static_cast<int>(in / cost);
    int64_t rest = in - h * cost;
    enter_unit();
    while (rest >= sp.n) {
      rest -= sp.n;
      ++u;
      enter_unit();
    }
    x = static_cast<int>(rest);
  }
  int4 rec = make_int4(-1, 0, 0, 0);
  int64_t at = o0;

  // a thread's row of the tile: K of key tid, or V of key tid - 64
  const bool value = tid >= kKeys;
  const int key = tid & (kKeys - 1);
  uint4 code[2 * NG];
  float scale[NG], mn[NG];
  bool absent;
  auto load = [&](int xx) {
    const int j = (sp.tile(xx) << kKeysLog2) + key;
    const int last = min(un.p1, s.keys - 1);
    const int lo = a.shape.window > 0 && un.p0 >= a.shape.window ? un.p0 - a.shape.window + 1 : 0;
    absent = false;
    int page = -1;
    if (j <= last && (j >= lo || j < a.shape.sinks)) {
      page = page_of(a.tab, i, j);
      if (page < 0) {
        absent = true;
        if (!value) atomicOr(a.batch.err, DEV_ERR_PAGE);
      }
    }
    if (page >= 0) {
      const int64_t slot = slot_of(a.pool, page, h, j);
      const uint4* c = reinterpret_cast<const uint4*>((value ? a.pool.codes[1] : a.pool.codes[0]) + slot * (D / 2));
#pragma unroll
      for (int e = 0; e < 2 * NG; ++e) code[e] = c[e];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        scale[g] = ((value ? a.pool.scales[1] : a.pool.scales[0]) + slot * NG)[g];
        mn[g] = ((value ? a.pool.mins[1] : a.pool.mins[0]) + slot * NG)[g];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 2 * NG; ++e) code[e] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int g = 0; g < NG; ++g) scale[g] = mn[g] = 0.0f;
    }
  };
  auto restore = [&]() {
    bool bad[2] = {false, false};
    if (value)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        bad[g] = !(fabsf(scale[g]) < INFINITY);
        if (bad[g]) scale[g] = mn[g] = 0.0f;
      }
    const uint32_t ab = __ballot_sync(0xffffffffu, absent), b0 = __ballot_sync(0xffffffffu, bad[0]), b1 = __ballot_sync(0xffffffffu, bad[1]);
    if (lane == 0) {
      if (value) {
        sm.nan[0][key >> 5] = b0;
        sm.nan[1][key >> 5] = b1;
      } else {
        sm.absent[key >> 5] = ab;
      }
    }
    float* dst = value ? sm.v[key] : sm.k[key];
#pragma unroll
    for (int e = 0; e < 2 * NG; ++e) {
      const uint32_t words[4] = {code[e].x, code[e].y, code[e].z, code[e].w};
      const float sc = scale[e >> 1], m = mn[e >> 1];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int n = 0; n < 8; n += 4)
          *reinterpret_cast<float4*>(dst + 32 * e + 8 * c + n) =
              make_float4(__fmaf_rn(static_cast<float>((words[c] >> (4 * n)) & 15u), sc, m),
                          __fmaf_rn(static_cast<float>((words[c] >> (4 * n + 4)) & 15u), sc, m),
                          __fmaf_rn(static_cast<float>((words[c] >> (4 * n + 8)) & 15u), sc, m),
                          __fmaf_rn(static_cast<float>((words[c] >> (4 * n + 12)) & 15u), sc, m));
    }
  };

  while (left > 0) {
    const int x1 = x + (left < sp.n - x ? left : sp.n - x);
    const int x0 = x;
    const bool from_start = x0 == 0, to_end = x1 == sp.n;
    // Q of the unit's rows; a thread's two rows
    load(x);           // on its way under Q
    __syncthreads();   // the rows before are done with
    for (int e = tid; e < kRows * D / 4; e += kThreads) {
      const int r = e / (D / 4), c = e % (D / 4), row = un.r0 + (r < un.rows ? r : 0), t = row / a.shape.group;
      const float4 q = *reinterpret_cast<const float4*>(a.q + static_cast<int64_t>(s.row0 + t) * a.ldq +
                                                        static_cast<int64_t>(h * a.shape.group + row - t * a.shape.group) * D + 4 * c);
      *reinterpret_cast<float4*>(&sm.q[r][4 * c]) = r < un.rows ? q : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    int pos[2];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, o[2][CW];
    uint32_t nans[2] = {0u, 0u};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      pos[r] = s.len - s.n + (un.r0 + 2 * ry + r) / a.shape.group;
#pragma unroll
      for (int c = 0; c < CW; ++c) o[r][c] = 0.0f;
    }
    for (; x < x1; ++x) {
      const int t0 = sp.tile(x) << kKeysLog2;
      restore();
      __syncthreads();
      if (x + 1 < x1) load(x + 1);
      // scores
      float sc[2][4];
      float2 s2[2][4];   // even and odd dims
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) s2[r][c] = make_float2(0.0f, 0.0f);
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 q[2], k[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) q[r] = *reinterpret_cast<const float4*>(&sm.q[2 * ry + r][d]);
#pragma unroll
        for (int c = 0; c < 4; ++c) k[c] = *reinterpret_cast<const float4*>(&sm.k[cx + 16 * c][d]);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            s2[r][c] = q4::fma_f32x2(make_float2(q[r].x, q[r].y), make_float2(k[c].x, k[c].y), s2[r][c]);
            s2[r][c] = q4::fma_f32x2(make_float2(q[r].z, q[r].w), make_float2(k[c].z, k[c].w), s2[r][c]);
          }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[r][c] = s2[r][c].x + s2[r][c].y;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int kk = cx + 16 * c, j = t0 + kk, p = pos[r];
          const bool see = j <= p && j < s.keys && (a.shape.window == 0 || j > p - a.shape.window || j < a.shape.sinks) &&
                           !((sm.absent[kk >> 5] >> (kk & 31)) & 1u);
          if (see) {
            nans[r] |= ((sm.nan[0][kk >> 5] >> (kk & 31)) & 1u) | (((sm.nan[1][kk >> 5] >> (kk & 31)) & 1u) << 1);
            sc[r][c] *= a.scale;
          } else {
            sc[r][c] = -INFINITY;
          }
          mx = fmaxf(mx, sc[r][c]);
        }
#pragma unroll
        for (int f = 8; f > 0; f >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, f));
        const float nm = fmaxf(m[r], mx), base = nm == -INFINITY ? 0.0f : nm;
        const float alpha = expf(m[r] - base);   // 0 where nothing was seen before
        m[r] = nm;
        l[r] *= alpha;
#pragma unroll
        for (int c = 0; c < CW; ++c) o[r][c] *= alpha;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float p = expf(sc[r][c] - base);
          l[r] += p;
          sm.p[2 * ry + r][cx + 16 * c] = p;
        }
      }
      __syncwarp();   // a row's weights are its half warp's own
#pragma unroll 2
      for (int kk = 0; kk < kKeys; kk += 4) {
        float4 p[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) p[r] = *reinterpret_cast<const float4*>(&sm.p[2 * ry + r][kk]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float4 v = *reinterpret_cast<const float4*>(&sm.v[kk + e][64 * g + 4 * cx]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float f = e == 0 ? p[r].x : e == 1 ? p[r].y : e == 2 ? p[r].z : p[r].w;
              o[r][4 * g] = fmaf(f, v.x, o[r][4 * g]);
              o[r][4 * g + 1] = fmaf(f, v.y, o[r][4 * g + 1]);
              o[r][4 * g + 2] = fmaf(f, v.z, o[r][4 * g + 2]);
              o[r][4 * g + 3] = fmaf(f, v.w, o[r][4 * g + 3]);
            }
          }
      }
      __syncthreads();   // K, V and the flags are read
    }
    // ---- the segment's rows: finished, or this share's partial
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int f = 8; f > 0; f >>= 1) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], f);
        nans[r] |= __shfl_xor_sync(0xffffffffu, nans[r], f);
      }
      const int n = 2 * ry + r;
      if (n >= un.rows) continue;
      const bool whole = from_start && to_end;
      const float f = !whole ? 1.0f : l[r] == 0.0f ? 0.0f : 1.0f / l[r];
      const int row = un.r0 + n, t = row / a.shape.group;
      const int64_t slot = (static_cast<int64_t>(w) * 2 + (from_start ? 1 : 0)) * pl.rows + n;
      float* dst = whole ? a.out + static_cast<int64_t>(s.row0 + t) * a.ldo +
                               static_cast<int64_t>(h * a.shape.group + row - t * a.shape.group) * D
                         : pl.part + slot * D;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float4 v = make_float4(o[r][4 * g] * f, o[r][4 * g + 1] * f, o[r][4 * g + 2] * f, o[r][4 * g + 3] * f);
        if ((nans[r] >> g) & 1u) v.x = v.y = v.z = v.w = __uint_as_float(0x7fffffffu);
        *reinterpret_cast<float4*>(dst + 64 * g + 4 * cx) = v;
      }
      if (!whole && cx == 0) pl.stat[slot] = make_float2(m[r] * 1.44269504f, l[r]);   // the join works in base 2
    }
    if (from_start && !to_end) rec = make_int4(i, h, u, static_cast<int>((at + sp.n - 1) / per));
    at += x1 - x0;
    left -= x1 - x0;
    if (left == 0) break;
    if (++u == units) {
      u = 0;
      if (++h == a.pool.heads) {
        do ++i;
        while (line.pre[i + 1] == line.pre[i]);
        h = 0;
        enter_seq();
      }
    }
    enter_unit();
    x = 0;
  }
  if (tid == 0) pl.rec[w] = rec;
}

template <int D>
fg_status launch(const AttnArgs<float>& a, const ClassPlan& pl, bool own_plan, cudaStream_t st) {
  constexpr int bytes = sizeof(Smem<D>);
  static bool set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (bytes > 48 * 1024 && dev >= 0 && dev < 64 && !set[dev]) {
    if (cudaFuncSetAttribute(f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
      return check_launch("f32_kernel smem attribute");
    set[dev] = true;
  }
  Trace tr(KC_ATTN_PAGED, st);
  return paged::launch("f32_kernel", true, f32_kernel<D>, static_cast<unsigned>(pl.workers), kThreads, bytes, st, a, pl, own_plan);
}

}  // namespace

// CTAs that fit an SM's shared memory (44 and 81 KB each)
int f32_workers(int head_dim, int sms) { return sms * (head_dim == 128 ? 2 : 4); }

fg_status paged_attention_f32(const AttnArgs<float>& a, const ClassPlan& pl, int head_dim, bool own_plan, cudaStream_t st) {
  return head_dim == 128 ? launch<128>(a, pl, own_plan, st) : launch<64>(a, pl, own_plan, st);
}

}  // namespace paged
}  // namespace fg
