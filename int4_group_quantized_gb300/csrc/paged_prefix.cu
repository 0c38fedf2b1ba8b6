// Attention of a group's rows over the prefix that its sequences share (FlexGen
// notes, "背景知识" attention; "5. 近似方法" 4-bit K/V), first and plainly: a row a
// thread, a key after another, everything in fp32.
#include <math.h>

#include "paged_prefix.cuh"
#include "q4_dev.cuh"
#include "tc_ptx.cuh"

namespace fg {
namespace paged {
namespace {

constexpr int kKeys = 32;   // of a step

template <int D>
__global__ void __launch_bounds__(kPrefixRows) prefix_kernel(const PrefixArgs p) {
  constexpr int NG = D / 64;
  __shared__ PrefixLine line;
  __shared__ float k[kKeys][D], v[kKeys][D];
  __shared__ int there[kKeys];
  tc::griddep_launch();
  tc::griddep_wait();
  prefix_line(p, line);
  const AttnArgs<__half>& a = p.a;
  const int tid = threadIdx.x, w = blockIdx.x, group = a.shape.group, psl = a.pool.ps_log2;
  const int64_t o0 = w * line.per;
  if (o0 >= line.total) return;
  int64_t left = min(line.per, line.total - o0);
  int g = line.g;
  PrefixGroup at = line.at;
  SharedGroup s = shared_group(a.prefix, a.tab, a.batch, g);
  int64_t in = o0 - at.base;
  int h = static_cast<int>(in / (static_cast<int64_t>(at.units) * at.tiles));
  in -= static_cast<int64_t>(h) * at.units * at.tiles;
  int u = static_cast<int>(in / at.tiles), x0 = static_cast<int>(in - static_cast<int64_t>(u) * at.tiles);
  while (true) {
    const int x1 = static_cast<int>(min(static_cast<int64_t>(at.tiles), x0 + left));
    const int r = u * at.rows + tid;
    const bool on = tid < at.rows && r < s.list * group;
    const int x = on ? r / group : 0, gh = on ? r - x * group : 0, row = on ? listed_row(a.prefix, a.batch, s.first + x) : 0;
    const __half* q = a.q + row * a.ldq + static_cast<int64_t>(h * group + gh) * D;
    float o[D], m = -INFINITY, l = 0.0f;
#pragma unroll 8
    for (int c = 0; c < D; ++c) o[c] = 0.0f;
    for (int j0 = x0 << kPrefixKeysLog2; j0 < min(x1 << kPrefixKeysLog2, s.tokens); j0 += kKeys) {
      __syncthreads();
      for (int e = tid; e < kKeys * D; e += kPrefixRows) {
        const int j = e / D, c = e % D;
        const int page = j0 + j < s.tokens ? page_of(a.tab, s.leader, j0 + j) : -1;
        if (c == 0) there[j] = page >= 0;
        if (c == 0 && page < 0 && j0 + j < s.tokens) atomicOr(a.batch.err, DEV_ERR_PAGE);
        const int64_t slot = page < 0 ? 0 : slot_of(a.pool, page, h, j0 + j);
        for (int kv = 0; kv < 2; ++kv) {
          const int code = (a.pool.codes[kv][slot * (D / 2) + c / 2] >> (4 * (c & 1))) & 15;
          const float sc = a.pool.scales[kv][slot * NG + c / 64], mn = a.pool.mins[kv][slot * NG + c / 64];
          const float val = kv && !(fabsf(sc) < INFINITY) ? __uint_as_float(0x7fffffffu) : fmaf(static_cast<float>(code), sc, mn);
          (kv ? v : k)[j][c] = page < 0 ? 0.0f : val;
        }
      }
      __syncthreads();
      if (!on) continue;
      for (int j = 0; j < kKeys; ++j) {
        if (!there[j]) continue;
        float sum = 0.0f;
        for (int c = 0; c < D; ++c) sum = fmaf(__half2float(q[c]), k[j][c], sum);
        sum *= a.scale_log2;
        const float top = fmaxf(m, sum), base = top == -INFINITY ? 0.0f : top, f = exp2f(m - base), e = exp2f(sum - base);
        l = fmaf(l, f, e);
        for (int c = 0; c < D; ++c) o[c] = fmaf(o[c], f, e * v[j][c]);
        m = top;
      }
    }
    if (on) {
      const int64_t home = static_cast<int64_t>(s.first + x) * a.q_heads + h * group + gh, extra = static_cast<int64_t>(w) * kPrefixRows + tid;
      float* to = x0 == 0 ? a.prefix.home + home * D : a.prefix.extra + extra * D;
      for (int c = 0; c < D; ++c) to[c] = o[c];
      (x0 == 0 ? a.prefix.home_stat[home] : a.prefix.extra_stat[extra]) = make_float2(m, l);
    }
    left -= x1 - x0;
    if (left == 0) return;
    x0 = 0;
    if (++u == at.units) {
      u = 0;
      if (++h == a.pool.heads) {
        h = 0;
        const int64_t next = at.base + static_cast<int64_t>(a.pool.heads) * at.units * at.tiles;
        do s = shared_group(a.prefix, a.tab, a.batch, ++g);
        while (s.list == 0 || (p.tile.workers > 0 && s.list * group > kPrefixFew));
        at = prefix_group(s, group, false);
        at.base = next;
      }
    }
  }
}

}  // namespace

fg_status paged_prefix(const PrefixArgs& p, int head_dim, cudaStream_t st) {
  Trace tr(KC_ATTN_PAGED, st);
  return paged::launch("prefix_kernel", true, head_dim == 128 ? prefix_kernel<128> : prefix_kernel<64>, static_cast<unsigned>(p.workers), kPrefixRows,
                       0, st, p);
}

}  // namespace paged
}  // namespace fg
