// Exponentials as fixed-point integers, for draws that have to be decided as in
// 64-bit arithmetic.
//
// A draw compares u * sum(e) with running sums of e_i = exp((l_i - m) / T).  Over
// a whole vocabulary an error of 2^-24 in the running sum moves 200,000
// boundaries by more than some of them are wide, so one draw in a few hundred
// would land on a neighbour.  FP64 is no way out (2 operations a clock and SM);
// here e is formed in pairs of fp32 (a value and its rounding error, Dekker 1971)
// with a relative error below 2^-36 and then rounded once to an integer multiple
// of 2^-shift.  Integer sums are exact and do not depend on their order, so a
// row can be split over any number of threads and CTAs and still give the same
// bits.
//
// exp((l - m) / T) = 2^y, y = (l - m) * (log2 e / T) in a pair; the table-driven
// method of Tang (1989): y = n + j / 32 + f, |f| <= 1 / 64, 2^y = 2^n * 2^(j/32)
// * (1 + p(f)) with 2^(j/32) in a pair and p the Taylor series of 2^f - 1 to the
// fifth power (next term below 2^-48), its linear term in a pair.
#pragma once

#include <stdint.h>

namespace tail {

constexpr int EXP_TABLE = 32;
constexpr int EXP_MANT_BITS = 52;  // the significand below is an integer multiple of 2^-52

// 2^(j / 32) = first + second, second the fp32 rounding of the remainder
__device__ const float2 EXP2_TABLE[EXP_TABLE] = {
    {0x1.000000p+0f, 0x0.0p+0f},       {0x1.059b0ep+0f, -0x1.9d4f52p-25f}, {0x1.0b5586p+0f, 0x1.9f3122p-25f},
    {0x1.11301ep+0f, -0x1.fdb496p-25f}, {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f},
    {0x1.2387a6p+0f, 0x1.ceac48p-25f},  {0x1.29e9e0p+0f, -0x1.5c0424p-25f}, {0x1.306fe0p+0f, 0x1.4636e2p-25f},
    {0x1.371a74p+0f, -0x1.18aac6p-25f}, {0x1.3dea64p+0f, 0x1.824684p-25f},  {0x1.44e086p+0f, 0x1.8624b4p-30f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.5342b6p+0f, -0x1.2c5610p-25f}, {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f},
    {0x1.6247ecp+0f, -0x1.f8b550p-25f}, {0x1.6a09e6p+0f, 0x1.9fcef4p-26f},  {0x1.71f75ep+0f, 0x1.1d8beep-25f},
    {0x1.7a1148p+0f, -0x1.829fd0p-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f}, {0x1.8ace54p+0f, 0x1.15506ep-27f},
    {0x1.93737cp+0f, -0x1.e64744p-25f}, {0x1.9c4918p+0f, 0x1.51f848p-27f},  {0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b7f770p+0f, -0x1.a09438p-25f}, {0x1.c199bep+0f, -0x1.3d56b2p-27f},
    {0x1.cb720ep+0f, -0x1.8837ccp-27f}, {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.dfc974p+0f, -0x1.908c94p-25f},
    {0x1.ea4afap+0f, 0x1.52486cp-27f},  {0x1.f50766p+0f, -0x1.246eb0p-26f},
};

// log2(e) / T as a pair: the quotient and, from the exact remainder, the rest.  (An fp64 division by
// every thread kept the fp64 pipe, two operations a clock, busy for 41 of a kernel's 57 us.)  Below T = 2^-127
// the quotient passes fp32's largest value and counts as that: an infinite one would make 0 times infinity of
// the maximum's own exponent.
struct ExpScale {
  float h, l;
};
__device__ __forceinline__ ExpScale exp_scale(float temp) {
  constexpr float LH = 0x1.715476p+0f, LL = 0x1.4ae0c0p-26f;  // log2(e)
  ExpScale s;
  s.h = fminf(LH / temp, 3.402823466e38f);
  const float rest = fmaf(-s.h, temp, LH) + LL;
  s.l = s.h > 0.f && s.h < 3.402823466e38f ? rest / temp : 0.f;
  return s;
}

// The significand of exp((l - m) / T) in units of 2^-52 (below 2^54) and its
// binary exponent n <= 0: the value is mant * 2^(n - 52).  mant = 0 stands for
// anything below 2^-60, for l = -inf and for NaN.  l == m gives exactly 1, also
// when both are infinite.  `table` is EXP2_TABLE, in shared memory.
__device__ __forceinline__ int64_t exp_mant(float l, float m, ExpScale c, const float2* table, int& n) {
  n = 0;
  if (l == m) return int64_t(1) << EXP_MANT_BITS;
  const float d = l - m;  // with its rounding error: Knuth's two-sum
  const float dl = d - l;
  const float err = (l - (d - dl)) + (-m - dl);
  const float yh = d * c.h;
  if (!(yh >= -60.0f)) return 0;
  const float yl = fmaf(d, c.h, -yh) + fmaf(d, c.l, err * c.h);
  const int k = __float2int_rn(yh * 32.0f);
  n = k >> 5;
  const float2 t = table[k & 31];
  const float f0 = fmaf(static_cast<float>(k), -0.03125f, yh);  // exact
  const float fh = f0 + yl;
  const float fl = (f0 - fh) + yl;
  // 2^f - 1 = f ln 2 + f^2 (ln^2 2 / 2! + f ln^3 2 / 3! + ...)
  constexpr float L1H = 0x1.62e430p-1f, L1L = -0x1.05c610p-29f;
  const float a = fh * L1H;
  const float b = fmaf(fh, L1H, -a) + fmaf(fh, L1L, fl * L1H);
  float q = fmaf(fh, 0x1.5d87fep-10f, 0x1.3b2ab6p-7f);
  q = fmaf(fh, q, 0x1.c6b08ep-5f);
  q = fmaf(fh, q, 0x1.ebfbe0p-3f);
  const float s = fmaf(fh * fh, q, b);
  const float g = t.x * a;
  const float rest = fmaf(t.x, s, fmaf(t.x, a, -g)) + fmaf(t.y, a, t.y);
  const float e0 = t.x + g;
  const float e1 = ((t.x - e0) + g) + rest;
  const float eh = e0 + e1;
  const float el = (e0 - eh) + e1;
  // eh is in [0.98, 2): a multiple of 2^-24; |el| <= 2^-24
  return (static_cast<int64_t>(__float2int_rn(eh * 16777216.0f)) << (EXP_MANT_BITS - 24)) +
         __float2int_rn(el * 4503599627370496.0f);
}

// exp((l - m) / T) rounded to a multiple of 2^-shift, shift <= 52.
__device__ __forceinline__ int64_t exp_fixed(float l, float m, ExpScale c, const float2* table, int shift) {
  int n;
  const int64_t mant = exp_mant(l, m, c, table, n);
  const int r = EXP_MANT_BITS - shift - n;  // bits to drop
  if (r > 56) return 0;                     // below half a step: mant < 2^54
  return r > 0 ? (mant + (int64_t(1) << (r - 1))) >> r : mant;
}

// Two values at a time on the packed fp32 pipe (half the instructions): exp_fixed(l0), exp_fixed(l1)
// rounded to multiples of 2^-shift, off by at most one of them.  m is finite.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void unpack(F2 x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 sub(F2 a, F2 b) { return fma(b, f2(-1.f), a); }  // exact product: a - b rounded once

// (h 2^28 + w) / 2^r, rounded; r in [0, 56]: the value is below 2^54, and half of 2^r has to stay below 2^62.
// By 32-bit conversions and shifts: a conversion to 64 bits runs on the fp64 pipe.
__device__ __forceinline__ int64_t drop_bits(float h, float w, int r) {
  const int64_t mant = (static_cast<int64_t>(__float2int_rn(h)) << (EXP_MANT_BITS - 24)) + __float2int_rn(w);
  return (mant + ((int64_t(1) << r) >> 1)) >> r;
}

__device__ __forceinline__ void exp_fixed2(float l0, float l1, float m, ExpScale c, const float2* table, int shift,
                                           int64_t& r0, int64_t& r1) {
  const F2 l = f2(l0, l1), nm = f2(-m), ch = f2(c.h);
  const F2 d = add(l, nm), dl = sub(d, l);
  const F2 err = add(sub(l, sub(d, dl)), sub(nm, dl));
  const F2 yh = mul(d, ch);
  const F2 yl = add(fma(d, ch, mul(d, f2(-c.h))), fma(d, f2(c.l), mul(err, ch)));
  constexpr float ROUND = 12582912.0f;  // 1.5 * 2^23: its sum with a small number ends in that number's integer
  const F2 t = fma(yh, f2(32.0f), f2(ROUND));
  const F2 f0 = fma(sub(t, f2(ROUND)), f2(-0.03125f), yh);
  const F2 fh = add(f0, yl), fl = add(sub(f0, fh), yl);
  float t0, t1, y0, y1;
  unpack(t, t0, t1);
  unpack(yh, y0, y1);
  const int k0 = __float_as_int(t0) - __float_as_int(ROUND), k1 = __float_as_int(t1) - __float_as_int(ROUND);
  const float2 b0 = table[k0 & 31], b1 = table[k1 & 31];
  const F2 tx = f2(b0.x, b1.x), ty = f2(b0.y, b1.y);
  constexpr float L1H = 0x1.62e430p-1f, L1L = -0x1.05c610p-29f;
  const F2 a = mul(fh, f2(L1H)), na = mul(fh, f2(-L1H));
  const F2 b = add(fma(fh, f2(L1H), na), fma(fh, f2(L1L), mul(fl, f2(L1H))));
  F2 q = fma(fh, f2(0x1.5d87fep-10f), f2(0x1.3b2ab6p-7f));
  q = fma(fh, q, f2(0x1.c6b08ep-5f));
  q = fma(fh, q, f2(0x1.ebfbe0p-3f));
  const F2 s = fma(mul(fh, fh), q, b);
  const F2 g = mul(tx, a);
  const F2 rest = add(fma(tx, s, fma(tx, a, mul(tx, na))), fma(ty, a, ty));
  const F2 e0 = add(tx, g);
  const F2 e1 = add(add(sub(tx, e0), g), rest);
  const F2 eh = add(e0, e1), el = add(sub(e0, eh), e1);
  float h0, h1, w0, w1;
  unpack(mul(eh, f2(16777216.0f)), h0, h1);
  unpack(mul(el, f2(4503599627370496.0f)), w0, w1);
  // 2^y below half a step is 0, and so are -inf and NaN; what is left drops at most 53 bits (k >> 5 >= -(shift + 1))
  const float least = -static_cast<float>(shift + 1);
  r0 = y0 >= least ? drop_bits(h0, w0, EXP_MANT_BITS - shift - (k0 >> 5)) : 0;
  r1 = y1 >= least ? drop_bits(h1, w1, EXP_MANT_BITS - shift - (k1 >> 5)) : 0;
}

// Four of them; among logits of +inf (m too) each of those weighs 1 and the others nothing.
__device__ __forceinline__ void exp_fixed4(float4 l, float m, ExpScale c, const float2* table, int shift,
                                           int64_t (&r)[4]) {
  if (m == INFINITY) {
    r[0] = l.x == m ? int64_t(1) << shift : 0;
    r[1] = l.y == m ? int64_t(1) << shift : 0;
    r[2] = l.z == m ? int64_t(1) << shift : 0;
    r[3] = l.w == m ? int64_t(1) << shift : 0;
    return;
  }
  exp_fixed2(l.x, l.y, m, c, table, shift, r[0], r[1]);
  exp_fixed2(l.z, l.w, m, c, table, shift, r[2], r[3]);
}

// exp((l - m) / T) in fp32, scale = log2(e) / T: a relative error of a few 2^-24 times the exponent's
// size.  l == m gives 1; l = -inf 0, also where the scale is 0 (fmaxf takes the number beside a NaN).
__device__ __forceinline__ float exp_fast(float l, float m, float scale) {
  const float e = exp2f((l - m) * scale);
  return l == m ? 1.0f : fmaxf(e, 0.0f);
}

// exp((l - m) / T) in fp32 with a relative error of a few 2^-24 whatever the exponent's size: the exponent in a
// pair, exp2f of its first part and the second part's term of first order.
__device__ __forceinline__ float exp_single(float l, float m, ExpScale c) {
  if (l == m) return 1.0f;
  const float d = l - m, dl = d - l;
  const float err = (l - (d - dl)) + (-m - dl);
  const float yh = d * c.h;
  if (!(yh >= -150.0f)) return 0.0f;  // below fp32's smallest number, or NaN
  const float yl = fmaf(d, c.h, -yh) + fmaf(d, c.l, err * c.h);
  const float e = exp2f(yh);
  return fmaf(e * 0x1.62e430p-1f, yl, e);  // ln 2
}

// 2^e as fp64, e a normal exponent.
__device__ __forceinline__ double pow2_double(int e) {
  return __longlong_as_double(static_cast<long long>(1023 + e) << 52);
}

// exp((l - m) / T) as fp64 (a few values a row: fp64 is slow here).
__device__ __forceinline__ double exp_double(float l, float m, ExpScale c, const float2* table) {
  int n;
  const int64_t mant = exp_mant(l, m, c, table, n);
  return static_cast<double>(mant) * pow2_double(n - EXP_MANT_BITS);
}

// s * exp((l - m) / T) for s >= 0 in units of 2^-from, in units of 2^-to (rounded down).
__device__ __forceinline__ int64_t scale_fixed(int64_t s, int from, float l, float m, ExpScale c, const float2* table,
                                               int to) {
  int n;
  const uint64_t mant = static_cast<uint64_t>(exp_mant(l, m, c, table, n));
  const uint64_t hi = __umul64hi(static_cast<uint64_t>(s), mant), lo = static_cast<uint64_t>(s) * mant;
  const int r = from + EXP_MANT_BITS - n - to;  // bits to drop; at least 52
  if (r >= 128) return 0;
  return static_cast<int64_t>(r >= 64 ? hi >> (r - 64) : (hi << (64 - r)) | (lo >> r));
}

// The largest integer at most u * total: an integer sum S exceeds u * total iff it exceeds this.
__device__ __forceinline__ int64_t draw_threshold(float u, int64_t total) {
  return __double2ll_rd(static_cast<double>(u) * static_cast<double>(total));
}

// q * z, rounded down, for q in [0, 1] and 0 <= z < 2^62.
__device__ __forceinline__ int64_t prod_fixed(float q, int64_t z) {
  const uint32_t b = __float_as_uint(q);
  const uint32_t e = b >> 23;
  const uint32_t m = (b & 0x7fffffu) | (e ? 0x800000u : 0u);  // q = m * 2^(max(e, 1) - 150)
  const int r = 150 - static_cast<int>(e ? e : 1u);           // bits to drop: at least 23
  const uint64_t lo = static_cast<uint64_t>(m) * static_cast<uint32_t>(z);
  const uint64_t hi = static_cast<uint64_t>(m) * static_cast<uint32_t>(z >> 32) + (lo >> 32);
  if (r >= 96) return 0;
  return static_cast<int64_t>(r >= 32 ? hi >> (r - 32) : (hi << (32 - r)) | (static_cast<uint32_t>(lo) >> r));
}

}  // namespace tail
