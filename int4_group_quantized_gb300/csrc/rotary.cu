// Rotary positions of rows: the frequencies (host) and the rotation.
//
// Bound by the rows' bytes, read and written once.  A block takes two rows:
// their cosines and sines go into shared memory once for all heads, a thread
// then moves 16 bytes of each half (or 16 bytes of neighbouring pairs).  20
// thousand rows of 40 heads of 128, half of each rotated: 72 us for 410 MB, 84%
// of a copy's rate (10 thousand fp32 rows 63, 96%); 64 rows of 64 heads 6.3, a launch.
#include <math.h>

#include <algorithm>

#include "fg_internal.cuh"
#include "rotary.cuh"
#include "tc_ptx.cuh"

namespace fg {
namespace {

using namespace rotary;

constexpr int kThreads = 256;
constexpr int kMostRot = 65536;

__device__ __forceinline__ void load8(const float* p, float2 (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = make_float2(a.x, a.y);
  v[1] = make_float2(a.z, a.w);
  v[2] = make_float2(b.x, b.y);
  v[3] = make_float2(b.z, b.w);
}
__device__ __forceinline__ void load8(const __half* p, float2 (&v)[4]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
}
__device__ __forceinline__ void store8(float* p, const float2 (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}
__device__ __forceinline__ void store8(__half* p, const float2 (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 h = __float22half2_rn(v[e]);
    w[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ float get(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

template <typename T>
struct RotateArgs {
  const T* x;
  T* out;
  const int32_t* pos;
  const uint64_t* turns;
  int64_t rows, ldx, ldo;
  int heads, d, rot;
  float scale;
  int part;        // heads of a block
  bool copy;       // the dims past rot go to out
};

// 16 bytes at a time.  kRows rows and `part` heads a block; a head has rot / 16
// pieces that turn (HALF: eight dims of each half; PAIRS: rot / 8, eight dims side by side) and,
// where out is other memory, (d - rot) / 8 that are copied.  A thread has one
// piece of every (threads / pieces)-th head, in all rows at once: their loads are on
// their way together, and nothing is divided in the loop (with a piece after another,
// found by two divisions each, the 72 us above were 116; with four rows a block 74, eight 84;
// two rows in six blocks an SM, 40 registers, 79).
constexpr int kRows = 2;
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const RotateArgs<T> a) {
  extern __shared__ __align__(16) float cs[];   // [kRows][cosines, sines][rot / 2]
  tc::griddep_launch();
  tc::griddep_wait();
  const int pairs = a.rot / 2;
  const int parts = (a.heads + a.part - 1) / a.part;
  const int64_t row0 = blockIdx.x / parts * static_cast<int64_t>(kRows);
  const int h0 = static_cast<int>(blockIdx.x % parts) * a.part;
  const int rows = static_cast<int>(a.rows - row0 < kRows ? a.rows - row0 : kRows), h1 = min(a.heads, h0 + a.part);
  for (int i = threadIdx.x; i < rows * pairs; i += kThreads) {
    const int r = i / pairs, p = i - r * pairs;
    const float2 v = cos_sin(phase_of(a.pos[row0 + r], a.turns[p]), a.scale);
    cs[2 * r * pairs + p] = v.x;
    cs[(2 * r + 1) * pairs + p] = v.y;
  }
  __syncthreads();
  const int turn = HALF ? a.rot / 16 : a.rot / 8, per = turn + (a.copy ? (a.d - a.rot) / 8 : 0), step = kThreads / per;
  const int j = threadIdx.x % per, first = threadIdx.x / per;
  if (first >= step) return;
  const bool turns = j < turn, two = HALF && turns;
  const int at = turns ? 8 * j : a.rot + 8 * (j - turn);
  const T* x = a.x + row0 * a.ldx + at;
  T* out = a.out + row0 * a.ldo + at;
  for (int h = h0 + first; h < h1; h += step) {
    const int64_t off = static_cast<int64_t>(h) * a.d;
    float2 u[kRows][4], v[kRows][4];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (r < rows) {
        load8(x + r * a.ldx + off, u[r]);
        if (two) load8(x + r * a.ldx + off + pairs, v[r]);
      }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (r < rows) {
        const float* c = cs + 2 * r * pairs;
        const float* s = c + pairs;
        if (two) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            turn2(u[r][e], v[r][e], *reinterpret_cast<const float2*>(c + 8 * j + 2 * e), *reinterpret_cast<const float2*>(s + 8 * j + 2 * e));
          store8(out + r * a.ldo + off + pairs, v[r]);
        } else if (turns) {
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            float2 p = make_float2(u[r][e].x, u[r][e + 1].x), q = make_float2(u[r][e].y, u[r][e + 1].y);
            turn2(p, q, *reinterpret_cast<const float2*>(c + 4 * j + e), *reinterpret_cast<const float2*>(s + 4 * j + e));
            u[r][e] = make_float2(p.x, q.x);
            u[r][e + 1] = make_float2(p.y, q.y);
          }
        }
        store8(out + r * a.ldo + off, u[r]);
      }
  }
}

// Any strides and any even rot: a thread a pair, or an element past rot, of
// one row and all its heads.  The same 20 thousand rows with rows of an odd length
// 158 us, of halves of 128 dims 126; 60 dims of each head rotated 210: a pair's two
// elements are neighbours' loads of 2 bytes, and the dims past rot too.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads) rotate_any_kernel(const RotateArgs<T> a) {
  tc::griddep_launch();
  tc::griddep_wait();
  const int pairs = a.rot / 2, per = pairs + (a.copy ? a.d - a.rot : 0);
  const int64_t items = a.rows * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < items; i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t r = i / per;
    const int j = static_cast<int>(i - r * per);
    const T* x = a.x + r * a.ldx;
    T* out = a.out + r * a.ldo;
    if (j >= pairs) {
      for (int h = 0; h < a.heads; ++h) out[static_cast<int64_t>(h) * a.d + a.rot + j - pairs] = x[static_cast<int64_t>(h) * a.d + a.rot + j - pairs];
      continue;
    }
    const float2 v = cos_sin(phase_of(a.pos[r], a.turns[j]), a.scale);
    for (int h = 0; h < a.heads; ++h) {
      const int64_t p = static_cast<int64_t>(h) * a.d + (HALF ? j : 2 * j), q = p + (HALF ? pairs : 1);
      float u = get(x + p), w = get(x + q);
      turn1(u, w, v.x, v.y);
      put(out + p, u);
      put(out + q, w);
    }
  }
}

template <class... P, class... A>
fg_status launch(const char* what, void (*kernel)(P...), unsigned grid, size_t smem, cudaStream_t st, A&&... args) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  Trace tr(KC_ROTATE, st);
  cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  return check_launch(what);
}

template <typename T>
fg_status rotate(const fg_rotary& r, const void* x, int64_t rows, int64_t ldx, int32_t heads, int32_t d, const int32_t* pos, void* out,
                 int64_t ldo, cudaStream_t st) {
  RotateArgs<T> a{static_cast<const T*>(x), static_cast<T*>(out), pos, r.turns, rows, ldx, ldo, heads, d, r.rot, r.scale, heads, x != out && r.rot < d};
  const bool half = r.layout == FG_ROTARY_HALF;
  const size_t smem = static_cast<size_t>(kRows) * r.rot * sizeof(float);
  const int64_t blocks = (rows + kRows - 1) / kRows, sms = num_sms();
  const int per = (half ? r.rot / 16 : r.rot / 8) + (a.copy ? (d - r.rot) / 8 : 0);   // pieces of a head
  if (d % 8 == 0 && per <= kThreads && r.rot % (half ? 16 : 8) == 0 && ldx % 8 == 0 && ldo % 8 == 0 && aligned(x, 16) && aligned(out, 16) && smem <= 48 * 1024 &&
      static_cast<int64_t>(heads) * d <= (1 << 28)) {
    // few rows: the heads of a block of rows go to as many blocks as give every SM two
    const int64_t parts = std::min<int64_t>(heads, std::max<int64_t>(1, 2 * sms / blocks));
    a.part = static_cast<int>((heads + parts - 1) / parts);
    const int64_t grid = blocks * ((heads + a.part - 1) / a.part);
    if (grid <= INT32_MAX)
      return launch("rotate_kernel", half ? rotate_kernel<T, true> : rotate_kernel<T, false>, static_cast<unsigned>(grid), smem, st, a);
  }
  const int64_t items = rows * (r.rot / 2 + (a.copy ? d - r.rot : 0));
  const int64_t grid = std::min<int64_t>((items + kThreads - 1) / kThreads, sms * 16);
  return launch("rotate_any_kernel", half ? rotate_any_kernel<T, true> : rotate_any_kernel<T, false>, static_cast<unsigned>(grid), 0, st, a);
}

}  // namespace

fg_status check_rotary(const fg_rotary* r, int32_t head_dim) {
  if (!r) return fail(FG_ERR_ARG, "null rotation");
  if (!r->turns) return fail(FG_ERR_ARG, "rotation: null turns");
  if (!aligned(r->turns, 8)) return fail(FG_ERR_ALIGN, "rotation: turns need 8-byte alignment");
  if (r->layout != FG_ROTARY_HALF && r->layout != FG_ROTARY_PAIRS) return fail(FG_ERR_ARG, "rotation: layout %d", r->layout);
  if (r->rot < 2 || r->rot % 2 || r->rot > head_dim) return fail(FG_ERR_SHAPE, "rotation of %d of %d dims", r->rot, head_dim);
  if (!(fabsf(r->scale) < INFINITY)) return fail(FG_ERR_ARG, "rotation: scale");
  return FG_OK;
}

bool rows_meet(const void* x, int64_t ldx, int64_t xcols, const void* y, int64_t ldy, int64_t ycols, int64_t rows, fg_dtype dt) {
  const char *xb = static_cast<const char*>(x), *yb = static_cast<const char*>(y);
  const int64_t e = static_cast<int64_t>(dtype_bytes(dt)), xn = ((rows - 1) * ldx + xcols) * e, yn = ((rows - 1) * ldy + ycols) * e;
  if (xb >= yb + yn || yb >= xb + xn) return false;
  // columns of one buffer's rows may lie side by side
  const int64_t row = ldx * e, off = rows > 1 && ldx == ldy ? ((yb - xb) % row + row) % row : 0;
  return off < xcols * e || off + ycols * e > row;
}

fg_status check_apart(const void* x, int64_t ldx, const void* out, int64_t ldo, int64_t rows, int64_t cols, fg_dtype dt) {
  if (x == out ? (rows > 1 && ldx != ldo) : rows_meet(x, ldx, cols, out, ldo, cols, rows, dt))
    return fail(FG_ERR_ARG, "rotated rows go to the rows themselves, with their stride, or to memory apart from them");
  return FG_OK;
}

}  // namespace fg

using namespace fg;

namespace {

// Frequencies as sums of two doubles (Knuth's and Dekker's error-free sums and products): a position multiplies what the
// last bits of a turn are off, so all 64 have to be right.  About 100 bits; built without contraction.
struct Wide {
  double hi, lo;
};
constexpr Wide kTau = {6.283185307179586232, 2.4492935982947064e-16}, kLn2 = {0.6931471805599453094, 2.3190468138462996e-17};
constexpr double kMostTurns = 4294967296.0;   // of a position: 64 bits of the fraction are left

Wide joined(double a, double b) {   // |a| >= |b|
  const double s = a + b;
  return {s, b - (s - a)};
}
Wide wide(double a, double b = 0.0) {   // a + b
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
Wide operator+(Wide a, Wide b) {
  const Wide s = wide(a.hi, b.hi), t = wide(a.lo, b.lo), u = joined(s.hi, s.lo + t.hi);
  return joined(u.hi, u.lo + t.lo);
}
Wide operator-(Wide a) { return {-a.hi, -a.lo}; }
Wide operator*(Wide a, Wide b) {
  const double p = a.hi * b.hi;
  return joined(p, fma(a.hi, b.lo, fma(a.lo, b.hi, fma(a.hi, b.hi, -p))));
}
Wide operator/(Wide a, Wide b) {
  const double q = a.hi / b.hi;
  Wide r = a + -(b * wide(q));
  const double q2 = r.hi / b.hi;
  r = r + -(b * wide(q2));
  return wide(q) + wide(q2, r.hi / b.hi);
}
// 2^k (1 + y)^256, y the series of a 256th of what is left of x
Wide exp_wide(Wide x) {
  const double k = rint(x.hi / kLn2.hi);
  const Wide r = x + -(kLn2 * wide(k)), s = {ldexp(r.hi, -8), ldexp(r.lo, -8)};
  Wide y = wide(0.0);
  for (int n = 12; n > 0; --n) y = (wide(1.0) + y) * s / wide(n);
  for (int i = 0; i < 8; ++i) y = y * (wide(2.0) + y);
  y = wide(1.0) + y;
  return {ldexp(y.hi, static_cast<int>(k)), ldexp(y.lo, static_cast<int>(k))};
}
Wide log_wide(double x) {
  int k;
  const Wide m = wide(frexp(x, &k));
  Wide y = wide(log(m.hi));
  for (int i = 0; i < 2; ++i) y = y + (m * exp_wide(-y) + wide(-1.0));   // Newton
  return y + kLn2 * wide(k);
}
Wide share_of(Wide x) { return x.hi < 0.0 ? wide(0.0) : x.hi < 1.0 ? x : wide(1.0); }
// The fraction of a turn, in units of 2^-64, rounded.
uint64_t fraction(Wide t) {
  const Wide f = t + wide(-floor(t.hi));   // in (-2^-52, 1]
  const double h = ldexp(f.hi, 64), whole = floor(h);
  const uint64_t top = whole < 0.0 || whole >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(whole);   // (2^64 is a whole turn)
  return top + static_cast<uint64_t>(static_cast<int64_t>(rint((whole < 0.0 ? h : h - whole) + ldexp(f.lo, 64))));
}

}  // namespace

extern "C" {

fg_status fg_rotary_turns(int32_t rot, int32_t scaling, double base, double factor, double context, double low, double high,
                          uint64_t* turns, float* scale) {
  if (!turns || !scale) return fail(FG_ERR_ARG, "null pointer");
  if (scaling < FG_ROTARY_PLAIN || scaling > FG_ROTARY_RAMP) return fail(FG_ERR_ARG, "scaling %d", scaling);
  if (rot < 2 || rot % 2 || rot > kMostRot) return fail(FG_ERR_SHAPE, "rotation of %d dims", rot);
  if (!(base > 1.0 && base < INFINITY)) return fail(FG_ERR_ARG, "base %g", base);
  const bool banded = scaling == FG_ROTARY_BANDS || scaling == FG_ROTARY_RAMP;
  if (scaling != FG_ROTARY_PLAIN && !(factor > 0.0 && factor < INFINITY)) return fail(FG_ERR_ARG, "factor %g", factor);
  if (scaling == FG_ROTARY_RAMP && factor < 1.0) return fail(FG_ERR_ARG, "factor %g below 1", factor);
  if (scaling == FG_ROTARY_BASE && rot < 4) return fail(FG_ERR_SHAPE, "a rotation of two dims has no other base");
  if (banded && !(context > 0.0 && context < INFINITY && low > 0.0 && low < high && high < INFINITY))
    return fail(FG_ERR_ARG, "context %g, low %g, high %g", context, low, high);
  Wide ln_base = log_wide(base);
  if (scaling == FG_ROTARY_BASE) {
    ln_base = ln_base + log_wide(factor) * wide(rot) / wide(rot - 2);
    if (!(ln_base.hi < 709.0)) return fail(FG_ERR_ARG, "base %g stretched by %g", base, factor);   // near the largest double
  }
  double from = 0.0, to = 0.0;
  if (scaling == FG_ROTARY_RAMP) {
    auto pair_of = [&](double t) { return rot * log(context / (kTau.hi * t)) / (2.0 * log(base)); };
    from = std::max(0.0, floor(pair_of(high)));
    to = std::min(rot - 1.0, ceil(pair_of(low)));
  }
  for (int pass = 0; pass < 2; ++pass)   // looked at, then written
    for (int i = 0; i < rot / 2; ++i) {
      const Wide y = ln_base * wide(-2.0 * i) / wide(rot);
      if (!(y.hi < 709.0)) return fail(FG_ERR_ARG, "frequency %d", i);
      Wide f = exp_wide(y);
      Wide share = wide(1.0);   // of f, the rest of f / factor
      if (scaling == FG_ROTARY_LINEAR) share = wide(0.0);
      if (scaling == FG_ROTARY_BANDS) share = share_of((wide(context) * f / kTau + wide(-low)) / wide(high, -low));
      if (scaling == FG_ROTARY_RAMP) share = wide(1.0) + -share_of(wide(i, -from) / wide(std::max(to - from, 0.001)));
      if (share.hi < 1.0) f = share * f + (wide(1.0) + -share) * (f / wide(factor));
      const Wide t = f / kTau;
      if (!(t.hi < kMostTurns)) return fail(FG_ERR_ARG, "frequency %d of %g", i, f.hi);
      if (pass == 1) turns[i] = fraction(t);
    }
  *scale = scaling == FG_ROTARY_RAMP ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.0f;
  return FG_OK;
}

fg_status fg_rotate(const fg_rotary* r, const void* x, fg_dtype dt, int64_t rows, int64_t ldx, int32_t heads, int32_t head_dim,
                    const int32_t* pos, void* out, int64_t ldo, cudaStream_t stream) {
  if (dt != FG_F16 && dt != FG_F32) return fail(FG_ERR_ARG, "dtype");
  if (rows < 0 || heads < 0 || head_dim < 0) return fail(FG_ERR_ARG, "negative sizes");
  if (head_dim > kMostRot || heads > 65535 || rows > (int64_t(1) << 40)) return fail(FG_ERR_UNSUPPORTED, "more than 65536 dims, 65535 heads or 2^40 rows");
  FG_TRY(check_rotary(r, head_dim));
  if (rows == 0 || heads == 0) return FG_OK;
  if (!x || !out || !pos) return fail(FG_ERR_ARG, "null pointer");
  const int64_t h1 = static_cast<int64_t>(heads) * head_dim;
  if (rows > 1 && (ldx < h1 || ldo < h1)) return fail(FG_ERR_SHAPE, "row stride below heads * head_dim = %lld", (long long)h1);
  if (!aligned(x, dtype_bytes(dt)) || !aligned(out, dtype_bytes(dt)) || !aligned(pos, 4)) return fail(FG_ERR_ALIGN, "rows or positions");
  FG_TRY(check_apart(x, ldx, out, ldo, rows, h1, dt));
  if (dt == FG_F16) return rotate<__half>(*r, x, rows, ldx, heads, head_dim, pos, out, ldo, stream);
  return rotate<float>(*r, x, rows, ldx, heads, head_dim, pos, out, ldo, stream);
}

}  // extern "C"
