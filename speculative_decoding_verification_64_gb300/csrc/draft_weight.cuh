// Weights exp((l - M) / T) for sums over a whole vocabulary that name a token: each weight is
// a whole number of 2^-42 of the largest one, good to 2^-43 of that and about 2^-35 of itself, and
// sums of them are exact, in any order.  A sum is that of 64-bit floating point to 2^-35 of
// itself and 2^-43 a token; the latter shows where a long tail of tokens stands some 30 T below
// the largest (each counts as 0 or as 2^-42): 1.5e-8 for 128256 tokens, 2^-24 for 2^19.
//
// With c = log2(e) / T as a pair of floats, x = (l - M) c is cut at the nearest multiple of
// 2^-10: 2^x = 2^n 2^(j/1024) 2^f with |f| <= 2^-11.  2^(j/1024) comes from a table of
// pairs, 2^f - 1 = f (ln 2 + f ln^2 2 / 2) with an error of 2^-37.  The difference
// l c - (M c + n + j / 1024) is one fused multiply-add, so that neither product is rounded on
// its own; M c itself is first rounded to a multiple of 2^-10, which scales all weights of a
// row alike.
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
    // (the upper part below the value, so that the lower one is positive and both can be
    // scaled by adding to their exponents)
    float hi = (float)(y - 0x1p-25);
    if ((double)hi >= y) hi = (float)(y - 0x1p-23);
    t.at[j].hi = hi;
    t.at[j].lo = (float)(y - (double)hi);
  }
  return t;
}

#ifdef __CUDACC__

constexpr float kFixed = 0x1p42f;  // fixed-point units of a weight of 1

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

// Two weights, each a + b with a a multiple of 2^-21 and b one of 2^-42 not above 2^-20: as
// the bits of 6 + a and of 3 * 2^-20 + b, which count those units from kBits6 and kBitsB.
// (Integer sums of them are exact, and cost less than float32 ones.)
constexpr uint32_t kBits6 = 0x40C00000u, kBitsB = 0x36400000u;

__device__ __forceinline__ void weight2(float2 l, const WeightOf &w, const float2 *table, uint32_t *a,
                                        uint32_t *b) {
  const float2 ch = both(w.ch);
  l = __fadd2_rn(l, both(-w.off));
  l = make_float2(fmaxf(l.x, w.least), fmaxf(l.y, w.least));
  const float2 t = __ffma2_rn(l, ch, both(w.magic));  // 12288 + x, rounded to a multiple of 2^-10
  const float2 at = __fadd2_rn(both(w.magic), make_float2(-t.x, -t.y));
  float2 f = __ffma2_rn(l, ch, at);
  f = __ffma2_rn(l, both(w.cl), f);
  // 2^f - 1 to 2^-37
  const float2 m = __fmul2_rn(f, __ffma2_rn(f, both(0.240226507f), both(0.693147181f)));
  const uint32_t i0 = __float_as_uint(t.x), i1 = __float_as_uint(t.y);
  const float2 t0 = table[i0 & (kTable - 1)], t1 = table[i1 & (kTable - 1)];
  // (the bits of 12288.0 above the index leave nothing in the exponent's place)
  const uint32_t e0 = (i0 << 13) & 0xFF800000u, e1 = (i1 << 13) & 0xFF800000u;
  const float2 hi = make_float2(__uint_as_float(__float_as_uint(t0.x) + e0),
                                __uint_as_float(__float_as_uint(t1.x) + e1));
  const float2 lo = make_float2(__uint_as_float(__float_as_uint(t0.y) + e0),
                                __uint_as_float(__float_as_uint(t1.y) + e1));
  const float2 v = __ffma2_rn(hi, m, lo);
  const float2 y = __fadd2_rn(__fadd2_rn(hi, both(6.0f)), v);
  // hi - a, with a within 2^-21 of hi + v: exact
  const float2 d = __fadd2_rn(hi, __fadd2_rn(both(6.0f), make_float2(-y.x, -y.y)));
  const float2 z = __fadd2_rn(__fadd2_rn(d, v), both(0x1.8p-19f));
  a[0] = __float_as_uint(y.x);
  a[1] = __float_as_uint(y.y);
  b[0] = __float_as_uint(z.x);
  b[1] = __float_as_uint(z.y);
}

// The fixed-point sum of n weights from the sums of their bits.
__device__ __forceinline__ unsigned long long fixed_sum(uint32_t a, uint32_t b, int n) {
  return ((unsigned long long)(a - (uint32_t)n * kBits6) << 21) +
         (unsigned long long)(long long)(int32_t)(b - (uint32_t)n * kBitsB);
}

__device__ __forceinline__ unsigned long long weight_fixed(float l, const WeightOf &w,
                                                           const float2 *table) {
  uint32_t a[2], b[2];
  weight2(both(l), w, table, a, b);
  return fixed_sum(a[0], b[0], 1);
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
