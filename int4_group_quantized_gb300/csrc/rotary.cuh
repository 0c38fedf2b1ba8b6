// Rotary positions, device side: cosine and sine of a position's angle to more
// than fp32, and the rotation of a pair.
//
// An angle is a 64-bit fraction of a turn (position times turns, wrapping): the
// turns' own rounding, 2^-65 a step, is all that a far position adds up (2^-34
// turns at 2^31).  Its top 8 bits, rounded, name one of
// 256 angles whose cosine and sine stand in a table as sums of two fp32; the
// rest, at most 1/512 turn (0.0123), goes through the addition theorem,
//   cos(a + d) = C + C (cos d - 1) - S sin d,   sin(a + d) = S + S (cos d - 1) + C sin d,
// with cos d - 1 and sin d - d from their series and the one large product (S d,
// C d) kept as a sum of two fp32.  What is left out is below 2^-36, so the fp32
// that comes out is the nearest one but for one angle in some thousands, and
// rows rotated here and elsewhere agree in their bits (and codes) but there.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace fg {
namespace rotary {

struct alignas(16) TurnEntry {
  float ch, cl, sh, sl;   // cosine = ch + cl, sine = sh + sl
};
struct TurnTable {
  TurnEntry e[256];
};

// Series at |x| <= pi/4, in double, for the table.
constexpr double series(double x, bool sine) {
  double term = sine ? x : 1.0, sum = term;
  for (int k = sine ? 3 : 2; k < 28; k += 2) {
    term *= -x * x / (k * (k - 1));
    sum += term;
  }
  return sum;
}
constexpr TurnEntry turn_entry(int k) {
  constexpr double kPi = 3.14159265358979323846;
  const int octant = (k + 32) / 64 % 4;                       // quarter turn that k lies around
  const double x = (k - 64 * ((k + 32) / 64)) * (kPi / 128.0);
  const double c0 = series(x, false), s0 = series(x, true);
  const double c = octant == 0 ? c0 : octant == 1 ? -s0 : octant == 2 ? -c0 : s0;
  const double s = octant == 0 ? s0 : octant == 1 ? c0 : octant == 2 ? -s0 : -c0;
  TurnEntry t{};
  t.ch = static_cast<float>(c);
  t.cl = static_cast<float>(c - static_cast<double>(t.ch));
  t.sh = static_cast<float>(s);
  t.sl = static_cast<float>(s - static_cast<double>(t.sh));
  return t;
}
constexpr TurnTable turn_table() {
  TurnTable t{};
  for (int k = 0; k < 256; ++k) t.e[k] = turn_entry(k);
  return t;
}
static __device__ const TurnTable kTurnTable = turn_table();

// a + b as a rounded sum and what the rounding left out.
__device__ __forceinline__ float two_sum(float a, float b, float& rest) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  rest = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
  return s;
}
// (hi + lo) * scale, rounded to fp32 once but for far bits.
__device__ __forceinline__ float scaled(float hi, float lo, float scale) {
  float rest;
  const float v = two_sum(hi, lo, rest), p = __fmul_rn(v, scale);
  return __fadd_rn(p, __fmaf_rn(rest, scale, __fmaf_rn(v, scale, -p)));
}

// scale * (cosine, sine) of the angle `phase` / 2^64 turns.
__device__ __forceinline__ float2 cos_sin(uint64_t phase, float scale) {
  constexpr float kTau = 6.28318530717958647692f;
  constexpr float kTauLow = static_cast<float>(6.28318530717958647692 - static_cast<double>(kTau));
  const uint64_t k = (phase + (uint64_t(1) << 55)) >> 56;
  const int64_t d = static_cast<int64_t>(phase - (k << 56));           // in [-2^55, 2^55)
  const float hi = __int2float_rn(static_cast<int>(d >> 25));          // of 2^-39 turns
  const float lo = __int2float_rn(static_cast<int>(d - (static_cast<int64_t>(__float2int_rn(hi)) << 25)));   // of 2^-64
  const float h = hi * 1.8189894035458565e-12f, l = lo * 5.421010862427522e-20f;
  const float x = __fmul_rn(h, kTau);                                  // d in radians: x + xl
  const float xl = __fmaf_rn(h, kTau, -x) + __fmaf_rn(h, kTauLow, l * kTau);
  const float x2 = x * x;
  const float sl = __fmaf_rn(x * x2, __fmaf_rn(x2, 1.0f / 120.0f, -1.0f / 6.0f), xl);   // sin d - x
  const float cm = __fmaf_rn(x2, __fmaf_rn(x2, 1.0f / 24.0f, -0.5f), -x * xl);          // cos d - 1
  const TurnEntry t = kTurnTable.e[k & 255];
  float rest;
  const float ps = __fmul_rn(t.sh, x), pse = __fmaf_rn(t.sh, x, -ps);
  const float c = two_sum(t.ch, -ps, rest);
  const float cl = rest + (__fmaf_rn(t.ch, cm, __fmaf_rn(-t.sh, sl, __fmaf_rn(-t.sl, x, t.cl))) - pse);
  const float pc = __fmul_rn(t.ch, x), pce = __fmaf_rn(t.ch, x, -pc);
  const float s = two_sum(t.sh, pc, rest);
  const float sll = rest + (__fmaf_rn(t.sh, cm, __fmaf_rn(t.ch, sl, __fmaf_rn(t.cl, x, t.sl))) + pce);
  return make_float2(scaled(c, cl, scale), scaled(s, sll, scale));
}
__device__ __forceinline__ uint64_t phase_of(int pos, uint64_t turns) { return static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns; }

// a c - b s and a s + b c of two pairs at once, each operation rounded by
// itself.  (Both sums are differences taken by an FMA with -1: a paired product
// with a paired sum after it came out contracted, in a quarter of the values.)
__device__ __forceinline__ void turn2(float2& a, float2& b, float2 c, float2 s) {
  float2 x, y;
  asm("{ .reg .b64 a, b, c, s, n, p, q; mov.b64 a, {%4, %5}; mov.b64 b, {%6, %7}; mov.b64 c, {%8, %9}; mov.b64 s, {%10, %11};\n"
      "mov.b64 n, {%12, %12};\n"
      "mul.rn.f32x2 p, a, c; mul.rn.f32x2 q, b, s; fma.rn.f32x2 p, q, n, p; mov.b64 {%0, %1}, p;\n"
      "xor.b64 b, b, 0x8000000080000000;\n"
      "mul.rn.f32x2 p, a, s; mul.rn.f32x2 q, b, c; fma.rn.f32x2 p, q, n, p; mov.b64 {%2, %3}, p; }"
      : "=f"(x.x), "=f"(x.y), "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(s.x), "f"(s.y), "f"(-1.0f));
  a = x;
  b = y;
}
__device__ __forceinline__ void turn1(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)), y = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
  a = x;
  b = y;
}

}  // namespace rotary
}  // namespace fg
