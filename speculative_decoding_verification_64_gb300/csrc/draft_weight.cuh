// Weights exp((l - M) / T) exact enough that sums over a whole vocabulary name the same
// token as sums in 64-bit floating point do: each weight is a whole number of 2^-42 of the
// largest one, good to about 2^-35 of itself, and sums of them are exact, in any order.
//
// With c = log2(e) / T as a pair of floats, x = (l - M) c is cut at the nearest multiple of
// 2^-10: 2^x = 2^n 2^(j/1024) 2^f with |f| <= 2^-11.  2^(j/1024) comes from a table of
// pairs, 2^f - 1 = f (ln 2 + f (ln^2 2 / 2 + f ln^3 2 / 6)) with an error of 2^-49.  The
// difference l c - (M c + n + j / 1024) is one fused multiply-add, so that neither product
// is rounded on its own; M c itself is first rounded to a multiple of 2^-10, which scales
// all weights of a row alike.
#pragma once

#include "draft_common.cuh"

namespace specdec {

constexpr int kTable = 1024;

struct alignas(16) WeightTable {
  struct {
    float hi, lo;
  } at[kTable];
};

constexpr double exp_series(double x) {  // 0 <= x <= ln 2
  double term = 1.0, sum = 1.0;
  for (int i = 1; i < 24; ++i) {
    term *= x / i;
    sum += term;
  }
  return sum;
}

constexpr WeightTable make_table() {
  WeightTable t{};
  for (int j = 0; j < kTable; ++j) {
    const double y = exp_series(j * (0.693147180559945309417232121458 / kTable));
    t.at[j].hi = (float)y;
    t.at[j].lo = (float)(y - (double)t.at[j].hi);
  }
  return t;
}

#ifdef __CUDACC__

constexpr float kFixed = 0x1p42f;  // units of a weight of 1

// What a row's weights need.  (No 64-bit arithmetic: this GPU has little of it.)
struct WeightOf {
  float ch, cl;     // c = log2(e) / T
  float off;        // taken from the logits first: 0, or M where M c is large (the
                    // difference is exact then for every logit that weighs anything)
  float magic;      // 12288 - M c, a multiple of 2^-10
  float least;      // logits (less off) below count as this one, whose weight of 2^-60 is 0
                    // in fixed point
  float rest;       // M c less its rounding: the weight of M is 2^rest
};

__device__ __forceinline__ WeightOf weight_of(float M, float ch, float cl) {
  WeightOf w;
  w.ch = ch;
  w.cl = cl;
  float mc = M * ch, low = fmaf(M, cl, fmaf(M, ch, -mc));
  w.off = 0.0f;
  if (fabsf(mc) >= 2047.0f) {
    w.off = M;
    mc = low = 0.0f;
  }
  const float mr = rintf(mc * 1024.0f) * 0x1p-10f;
  w.magic = 12288.0f - mr;
  w.least = (M - w.off) - 60.0f / ch;
  w.rest = (mc - mr) + low;
  return w;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Two weights as a + b: a a multiple of 2^-20, b one of 2^-42 and not above 2^-20, so that
// float32 sums of eight are exact.
__device__ __forceinline__ void weight2(float2 l, const WeightOf &w, const float2 *table, float2 &a,
                                        float2 &b) {
  const float2 ch = both(w.ch), magic = both(w.magic);
  l = __fadd2_rn(l, both(-w.off));
  l = make_float2(fmaxf(l.x, w.least), fmaxf(l.y, w.least));
  const float2 t = __ffma2_rn(l, ch, magic);  // 12288 + x, rounded to a multiple of 2^-10
  const float2 at = __fadd2_rn(t, both(-w.magic));
  float2 f = __ffma2_rn(l, ch, make_float2(-at.x, -at.y));
  f = __ffma2_rn(l, both(w.cl), f);
  float2 m = __ffma2_rn(f, both(0.0555041087f), both(0.240226507f));
  m = __ffma2_rn(f, m, both(0.693147181f));
  m = __fmul2_rn(f, m);
  const uint32_t i0 = __float_as_uint(t.x), i1 = __float_as_uint(t.y);
  const float2 t0 = table[i0 & (kTable - 1)], t1 = table[i1 & (kTable - 1)];
  // (the bits of 12288.0 above the index leave nothing in the exponent's place)
  const uint32_t e0 = (i0 << 13) & 0xFF800000u, e1 = (i1 << 13) & 0xFF800000u;
  const float2 hi = make_float2(__uint_as_float(__float_as_uint(t0.x) + e0),
                                __uint_as_float(__float_as_uint(t1.x) + e1));
  const float2 s = make_float2(__uint_as_float(0x3F800000u + e0), __uint_as_float(0x3F800000u + e1));
  const float2 lo = __fmul2_rn(make_float2(t0.y, t1.y), s);
  const float2 v = __ffma2_rn(hi, m, lo);
  const float2 y = __fadd2_rn(hi, v);
  const float2 rest = __fadd2_rn(__fadd2_rn(hi, make_float2(-y.x, -y.y)), v);
  a = __fadd2_rn(__fadd2_rn(y, both(12.0f)), both(-12.0f));
  b = __fadd2_rn(__fadd2_rn(y, make_float2(-a.x, -a.y)), rest);
  b = __fadd2_rn(__fadd2_rn(b, both(0x1.8p-19f)), both(-0x1.8p-19f));
}

// a + b in fixed point (whole numbers).
__device__ __forceinline__ unsigned long long fixed_of(float a, float b) {
  return (unsigned long long)(__float2ll_rz(a * kFixed) + __float2ll_rz(b * kFixed));
}

__device__ __forceinline__ unsigned long long weight_fixed(float l, const WeightOf &w,
                                                           const float2 *table) {
  float2 a, b;
  weight2(both(l), w, table, a, b);
  return fixed_of(a.x, b.x);
}

// The least integer that is at least p Z, for p in [0, 1) and Z < 2^63.
__device__ __forceinline__ unsigned long long share_at_least(float p, unsigned long long Z) {
  if (!(p > 0.0f)) return 0ull;
  const unsigned long long f = uniform_target(p, Z);
  // p = mant * 2^-sh: f is all of p Z where mant Z has no bits below 2^sh
  const uint32_t u = __float_as_uint(p);
  const int e = (int)(u >> 23);
  const unsigned long long mant = (u & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  const int sh = e ? 150 - e : 149;
  const unsigned long long lo = mant * Z, hi = __umul64hi(mant, Z);
  bool more;
  if (sh >= 128) more = (lo | hi) != 0;
  else if (sh > 64) more = lo != 0 || (hi & ((1ull << (sh - 64)) - 1)) != 0;
  else if (sh == 64) more = lo != 0;
  else more = (lo & ((1ull << sh) - 1)) != 0;
  return f + (more ? 1 : 0);
}

#endif  // __CUDACC__

}  // namespace specdec
