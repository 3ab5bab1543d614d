// Attention of drafted tokens over the 8-bit paged cache (specdec_attend).
//
// For one request and one head of k and v the R = N * G rows (node n, query
// head g of the group) all read the same cached tokens:
//     s = scale q . k (capped, biased), out = sum 2^(s' - m) v / sum 2^(s' - m),
// s' = s log2(e), with the running maximum m and sum of one pass.  Each cached
// byte is read once for 16 rows; with few rows the pass is bound by HBM.
//
// Streaming kernel.  A CTA of four warps takes one request, one k/v head, 16
// rows and one split of the tokens; a warp takes every fourth granule of 16
// tokens, with statistics of its own, so nothing waits on another warp until
// the four are joined at the end.  Codes go from global memory straight into
// the operand registers of m16n8k16 products, no shared memory between:
//   * the products' inner order is free, so for q k^T lane c of a quad owns 16
//     consecutive elements of a head instead of scattered pairs: one 16-byte
//     load fills the operand of four products;
//   * for p v the order of the output columns is free too: lane group g owns
//     D/8 consecutive elements of a head for its four tokens, and a byte
//     permute pairs neighbouring tokens.
// e4m3 codes widen to fp16 exactly.  q is scaled by a power of two per row, so
// that its largest element is in [2^10, 2^11): a bfloat16 is then exact in fp16
// but for elements below 2^-24 of that.  p goes into
// the products in fp16 (11 bits; bfloat16 would add as much error as the
// rounding of a bfloat16 result) around 2^6, so that weights down to 2^-20 of
// the largest keep all of them.  Float32 activations are split into two fp16
// terms each (22 bits) and the products repeated.  Maximum, sum and the
// accumulators are float32.
//
// A block's v scale, u = 2^k f with f in [1, 2), rides on the weights, whose fp16
// range has to fit what a row sees and nothing else: each row has a maximum m of its
// scores, for the sum, and one of s' - m + k, ko, for the outputs.  The products'
// weights are 2^(s' - m + k - ko) f: a token that the row does not see, or sees with
// next to no weight, leaves them alone whatever its size.  ko is an integer, so that the
// token of the largest score, which may hold most of the weight, has a power of two.
//
// The drafted tokens' own k and v take the same path as granules of 16 nodes,
// scaled to fp16 by a power of two per node (f = 1).  Where a mask hides part of a
// granule, non-finite v are taken out of the products (0 * NaN would reach rows
// that do not see them) and added to the rows that do.
//
// The tokens' granules, drafted ones last, are split over up to eight CTAs, a
// cluster, that join their partials through each other's shared memory: one
// launch.  More splits than that (few heads over a long cache) go through the
// workspace and a second kernel.
//
// Takes float32 calls, heads wider than 128 elements and small bfloat16 calls.
// Measured (8 heads of 128, G = 4): one request of 1 node over 777 tokens 20.5 us,
// of 5 over 2048 in float32 26.6 us.  Such calls are bound by latency: about 16 us
// pass before the first granule's products, in dependent loads and in code that
// is not in the instruction caches yet.
#include "attention_common.cuh"

namespace specdec {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;       // rows of one CTA
constexpr int kGran = 16;       // tokens of one granule
constexpr float kRaise = 8.0f;  // the maximum moves when a score passes it by this much
constexpr float kLift = 6.0f;   // p = 2^(s' - m + kLift) <= 2^14: inside fp16
constexpr unsigned kAll = 0xffffffffu;

// A partial: m[16], l[16], ko[16], then O[16][D]; a row's flags ride in l (< 0).
__host__ __device__ inline size_t partial_floats(int D) { return (size_t)kRows * (D + 3); }

__device__ __forceinline__ void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 2^k, k in [-126, 127].
__device__ __forceinline__ float pow2i(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// The exponent k of the unit that values of size up to `top` are carried in:
// top / 2^k is in [2^10, 2^11), clear of fp16's subnormals at both terms.
__device__ __forceinline__ int unit_exponent(float top) {
  return min(max((int)(__float_as_uint(top) >> 23) - 127 - 10, -126), 126);
}

// x = 2^k f: k, and f in [1, 2), for x >= 0 (f below 1 where x is below 2^-126).
__device__ __forceinline__ void split_unit(float x, float &k, float &f) {
  const uint32_t u = __float_as_uint(x);
  const bool normal = u >= 0x800000u;
  k = normal ? (float)((int)(u >> 23) - 127) : -126.0f;
  f = normal ? __uint_as_float((u & 0x7FFFFFu) | 0x3F800000u) : x * 0x1p126f;
}

// x 2^e for an e of any size (all factors are normal numbers; exact for an integer).
__device__ __forceinline__ float times_pow2(float x, float e) {
  const float whole = rintf(fminf(fmaxf(e, -252.0f), 252.0f));
  const int n = (int)whole, half = n / 2;
  return x * ex2_approx(e - whole) * pow2i(half) * pow2i(n - half);
}

__device__ __forceinline__ uint4 ldg_stream(const uint8_t *p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ uint2 ldg_stream8(const uint8_t *p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
               : "=r"(r.x), "=r"(r.y)
               : "l"(p));
  return r;
}

template <int DP, bool kF32, bool kPlain>
struct Kernel {
  static constexpr int KC = DP / 64;  // 16-byte pieces of a token that a lane takes for q k^T
  static constexpr int VB = DP / 8;   // consecutive elements that a lane takes for p v
  static constexpr int NT = DP / 8;   // 8-column tiles of the output
  static constexpr int KS = DP / 16;  // inner steps of q k^T
  static constexpr int U = 1;  // granules a warp has in flight

  struct Smem {
    uint4 q[KS][32];                    // A operands, in register order
    uint4 q_lo[kF32 ? KS : 1][32];      // the low terms of float32 activations
    float q_exp[kRows];                 // 2^e taken out of each row
    float o[2][kRows][DP + 4];          // joining of the warps; o[0]: the CTA's sums
    float m[kWarps][kRows], l[kWarps][kRows], ko[kWarps][kRows];
    float all_m[kRows], all_l[kRows], all_ko[kRows];   // the CTA's
    int bad[kWarps], all_bad;
  };

  const AttendParams &p;
  Smem &sm;
  const int lane, warp, g, c;
  int b, h, tile, split;
  int len, nodes, max_depth;
  // the thread's two rows (g and g + 8 of the CTA's 16)
  int node[2], pos[2];
  bool live[2];
  float rf[2], slope[2];
  float m[2], l[2], ko[2];  // maximum and sum of the scores; maximum with the units, from m
  float o[NT][4];

  __device__ Kernel(const AttendParams &p_, Smem &s_)
      : p(p_), sm(s_), lane(threadIdx.x & 31), warp(threadIdx.x >> 5), g((threadIdx.x & 31) >> 2),
        c(threadIdx.x & 3) {
    // splits are neighbours (a cluster's CTAs), then row tiles, which read the same tokens
    int i = blockIdx.x;
    split = i % p.splits;
    i /= p.splits;
    tile = i % p.row_tiles;
    i /= p.row_tiles;
    h = i % p.cache.Hkv;
    b = i / p.cache.Hkv;
  }

  __device__ __forceinline__ int row0() const { return tile * kRows; }

  __device__ __forceinline__ float act(const void *base, long long i) const {
    return load_elem(base, kF32 ? SPECDEC_F32 : SPECDEC_BF16, i);
  }

  // -------------------------------------------------------------------------
  // scores: products -> base-2 exponents, masked where hidden
  // -------------------------------------------------------------------------
  __device__ __forceinline__ float score(float dot, float k_unit, int i, int dist) const {
    // kPlain: neither cap nor bias, and rf carries log2(e)
    float s = dot * (k_unit * rf[i]);
    if (kPlain) return s;
    if (p.softcap > 0.0f) {
      const float y = s / p.softcap;
      if (kF32) {
        s = tanhf(y) * p.softcap;
      } else if (fabsf(y) < kTanhNear) {
        const float y2 = y * y;
        s *= fmaf(fmaf(fmaf(fmaf((float)kTanh4, y2, (float)kTanh3), y2, (float)kTanh2), y2,
                       (float)kTanh1), y2, 1.0f);
      } else {  // 1 - 2 / (1 + e^2y): absolute error below 2^-22
        s = (1.0f - __fdividef(2.0f, 1.0f + ex2_approx(y * (2.0f * kLog2e)))) * p.softcap;
      }
    }
    if (p.slopes) s -= slope[i] * (float)dist;
    return s * kLog2e;
  }

  // One granule's softmax: x[nt][0..3] are base-2 scores (hidden ones -inf), k[0..3]
  // the exponents of the v units of tokens 2c, 2c+1, 2c+8, 2c+9 (kSame: all alike).
  // The maxima move where a score passes them.  Lanes of a quad share rows.
  template <bool kSame>
  __device__ __forceinline__ void raise(const float (*x)[4], const float *k) {
    float to[2], at[2], best[2];  // m as it would be, where ko would stand from there, and the largest
    bool need = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = fmaxf(fmaxf(x[0][2 * i], x[0][2 * i + 1]), fmaxf(x[1][2 * i], x[1][2 * i + 1]));
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
      to[i] = fmaxf(m[i], top);
      at[i] = m[i] == -INFINITY ? -INFINITY : ko[i] + (m[i] - to[i]);
      const float from = to[i] == -INFINITY ? 0.0f : to[i];
      if (kSame) {
        best[i] = top - from + k[0];
      } else {
        best[i] = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) best[i] = fmaxf(best[i], x[j >> 1][2 * i + (j & 1)] - from + k[j]);
        best[i] = fmaxf(best[i], __shfl_xor_sync(kAll, best[i], 1));
        best[i] = fmaxf(best[i], __shfl_xor_sync(kAll, best[i], 2));
      }
      need |= top > m[i] + kRaise || best[i] > at[i] + kRaise;  // also the first time: -inf
    }
    if (__any_sync(kAll, need)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] *= m[i] == -INFINITY ? 0.0f : ex2_approx(m[i] - to[i]);
        ko[i] = fmaxf(floorf(at[i]), ceilf(best[i]));  // (nothing is lost by a smaller unit)
        const float f = at[i] == -INFINITY ? 0.0f : ex2_approx(at[i] - ko[i]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          o[j][2 * i] *= f;
          o[j][2 * i + 1] *= f;
        }
        m[i] = to[i];
      }
    }
  }

  // Adds p to l, and returns the products' weights as A operands; k and f: the v units
  // 2^k f of tokens 2c, 2c+1, 2c+8, 2c+9.
  __device__ __forceinline__ void weights(const float (*x)[4], const float *k, const float *f,
                                          uint32_t *a, uint32_t *a_lo) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float at = m[i] == -INFINITY ? 0.0f : m[i] - kLift;
      const float ato = ko[i] == -INFINITY ? 0.0f : ko[i];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const float x0 = x[nt][2 * i] - at, x1 = x[nt][2 * i + 1] - at;
        l[i] += ex2_approx(x0) + ex2_approx(x1);
        const float w0 = ex2_approx(x0 + (k[2 * nt] - ato)) * f[2 * nt];
        const float w1 = ex2_approx(x1 + (k[2 * nt + 1] - ato)) * f[2 * nt + 1];
        const uint32_t w = pack_half2(w0, w1);
        a[2 * nt + i] = w;
        if (kF32)
          a_lo[2 * nt + i] = pack_half2(w0 - half_bits_to_float(w & 0xFFFFu),
                                        w1 - half_bits_to_float(w >> 16));
      }
    }
  }

  // -------------------------------------------------------------------------
  // cached tokens
  // -------------------------------------------------------------------------
  struct Codes {
    uint4 k[2][KC];
    uint32_t v[4][VB / 4];
    float ks, vs;
  };

  __device__ __forceinline__ int block_of(int t) const {
    return p.block_shift >= 0 ? t >> p.block_shift : t / p.cache.block;
  }
  __device__ __forceinline__ int block_id(int t) const {
    return __ldg(p.cache.block_table + (long long)b * p.cache.max_blocks + block_of(t));
  }

  __device__ __forceinline__ void load(Codes &w, int t0, int id) const {
    const specdec_kv_cache &kv = p.cache;
    const long long cell = (long long)id * kv.Hkv + h;
    const int slot = t0 - block_of(t0) * kv.block;
    const uint8_t *k = reinterpret_cast<const uint8_t *>(kv.k) +
                       (cell * kv.block + slot) * kv.D;
    const uint8_t *v = reinterpret_cast<const uint8_t *>(kv.v) +
                       (cell * kv.block + slot) * kv.D;
    const int held = len - t0;  // tokens of this granule that exist
    w.ks = __ldg(kv.k_scale + cell);
    w.vs = __ldg(kv.v_scale + cell);
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int i = 0; i < KC; ++i) {
        const int t = nt * 8 + g, e = (c + 4 * i) * 16;
        w.k[nt][i] = (t < held && e < kv.D) ? ldg_stream(k + t * kv.D + e)
                                            : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = (j >> 1) * 8 + 2 * c + (j & 1), e = g * VB;
      if (VB == 8) {
        const uint2 x = (t < held && e < kv.D) ? ldg_stream8(v + t * kv.D + e) : make_uint2(0u, 0u);
        w.v[j][0] = x.x;
        w.v[j][1] = x.y;
      } else {
#pragma unroll
        for (int i = 0; i < VB / 16; ++i) {
          const uint4 x = (t < held && e + 16 * i < kv.D) ? ldg_stream(v + t * kv.D + e + 16 * i)
                                                          : make_uint4(0u, 0u, 0u, 0u);
          w.v[j][4 * i] = x.x;
          w.v[j][4 * i + 1] = x.y;
          w.v[j][4 * i + 2] = x.z;
          w.v[j][4 * i + 3] = x.w;
        }
      }
    }
  }

  __device__ __forceinline__ void dots(const Codes &w, float (*s)[4]) const {
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
#pragma unroll
    for (int i = 0; i < KC; ++i)
#pragma unroll
      for (int sub = 0; sub < 4; ++sub) {
        const uint4 qa = sm.q[i * 4 + sub][lane];
        const uint32_t a[4] = {qa.x, qa.y, qa.z, qa.w};
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const uint32_t word = sub == 0 ? w.k[nt][i].x : sub == 1 ? w.k[nt][i].y
                                : sub == 2 ? w.k[nt][i].z : w.k[nt][i].w;
          const uint32_t b0 = e4m3x2_to_half2(word & 0xFFFFu), b1 = e4m3x2_to_half2(word >> 16);
          mma16816(s[nt], a, b0, b1);
          if (kF32) {
            const uint4 ql = sm.q_lo[i * 4 + sub][lane];
            const uint32_t al[4] = {ql.x, ql.y, ql.z, ql.w};
            mma16816(s[nt], al, b0, b1);
          }
        }
      }
  }

  // Scores of the granule at t0 from its dots, hidden ones -inf.
  __device__ __forceinline__ void scores(float (*s)[4], float ks, int t0, bool partial) const {
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = e >> 1, t = t0 + nt * 8 + 2 * c + (e & 1);
        const float x = score(s[nt][e], ks, i, pos[i] - t);
        s[nt][e] = (partial && !sees(i, t)) ? -INFINITY : x;
      }
  }

  __device__ __forceinline__ bool sees(int i, int t) const {
    return live[i] && t < len && (p.window == 0 || pos[i] - t < p.window);
  }

  __device__ __forceinline__ void values(Codes &w, const uint32_t *a, const uint32_t *a_lo) {
#pragma unroll
    for (int q4 = 0; q4 < VB / 4; ++q4) {
      uint32_t b0[4], b1[4];
      const uint32_t x01 = __byte_perm(w.v[0][q4], w.v[1][q4], 0x5140);
      const uint32_t x23 = __byte_perm(w.v[0][q4], w.v[1][q4], 0x7362);
      const uint32_t y01 = __byte_perm(w.v[2][q4], w.v[3][q4], 0x5140);
      const uint32_t y23 = __byte_perm(w.v[2][q4], w.v[3][q4], 0x7362);
      b0[0] = e4m3x2_to_half2(x01 & 0xFFFFu);
      b0[1] = e4m3x2_to_half2(x01 >> 16);
      b0[2] = e4m3x2_to_half2(x23 & 0xFFFFu);
      b0[3] = e4m3x2_to_half2(x23 >> 16);
      b1[0] = e4m3x2_to_half2(y01 & 0xFFFFu);
      b1[1] = e4m3x2_to_half2(y01 >> 16);
      b1[2] = e4m3x2_to_half2(y23 & 0xFFFFu);
      b1[3] = e4m3x2_to_half2(y23 >> 16);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        mma16816(o[q4 * 4 + k], a, b0[k], b1[k]);
        if (kF32) mma16816(o[q4 * 4 + k], a_lo, b0[k], b1[k]);
      }
    }
  }

  // Element of the thread's output column: tile j, value e of its four.
  __device__ __forceinline__ int column(int j, int e) const { return (2 * c + (e & 1)) * VB + j; }

  // NaN codes of a partly hidden granule: out of the products, into the rows
  // that see their token.
  __device__ __forceinline__ void sift(Codes &w, int t0, int id) {
    unsigned hit = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q4 = 0; q4 < VB / 4; ++q4) {
        uint32_t keep = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (((w.v[j][q4] >> (8 * k)) & 0x7Fu) != 0x7Fu) keep |= 0xFFu << (8 * k);
        if (keep != kAll) hit |= 1u << ((j >> 1) * 8 + 2 * c + (j & 1));
        w.v[j][q4] &= keep;
      }
    hit = __reduce_or_sync(kAll, hit);
    const specdec_kv_cache &kv = p.cache;
    const uint8_t *v = reinterpret_cast<const uint8_t *>(kv.v) +
                       (((long long)id * kv.Hkv + h) * kv.block + t0 - block_of(t0) * kv.block) *
                           kv.D;
    while (hit) {
      const int t = __ffs(hit) - 1;
      hit &= hit - 1;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = column(j, e);
          if (d < kv.D && (v[t * kv.D + d] & 0x7Fu) == 0x7Fu && sees(e >> 1, t0 + t))
            o[j][e] = __int_as_float(0x7fc00000);
        }
    }
  }

  // Cached tokens [from, to): the warp's granules.  Returns false on a bad id.
  __device__ __forceinline__ bool cached(int from, int to) {
    constexpr int kStep = kGran * kWarps;
    int t0 = from + kGran * warp;
    int id[U];
    bool ok = true;
    auto fetch = [&](int t) {
      int i = t < to ? block_id(t) : 0;
      if (i < 0 || i >= p.cache.n_blocks) {
        ok = false;
        i = 0;
      }
      return i;
    };
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = fetch(t0 + u * kStep);
    Codes w[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t0 + u * kStep < to) load(w[u], t0 + u * kStep, id[u]);
    for (; t0 < to; t0 += U * kStep) {
      int next[U];
#pragma unroll
      for (int u = 0; u < U; ++u) next[u] = fetch(t0 + (U + u) * kStep);
      // the window's and the length's edges; with a tree's depth unknown, any
      // granule that the deepest possible node may not see whole
      float s[U][2][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * kStep;
        if (t < to) {
          const bool partial =
              t + kGran > len || (p.window > 0 && t <= len + p.N - 1 - p.window);
          dots(w[u], s[u]);
          scores(s[u], w[u].ks, t, partial);
          if (partial && p.window > 0) sift(w[u], t, id[u]);
        } else {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u][nt][e] = -INFINITY;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t0 + u * kStep < to) {
          float uk, uf;
          split_unit(w[u].vs, uk, uf);
          const float k[4] = {uk, uk, uk, uk}, f[4] = {uf, uf, uf, uf};
          raise<true>(s[u], k);
          uint32_t a[4], a_lo[4];
          weights(s[u], k, f, a, a_lo);
          values(w[u], a, a_lo);
        }
        if (t0 + (U + u) * kStep < to) load(w[u], t0 + (U + u) * kStep, next[u]);
        id[u] = next[u];
      }
    }
    return ok;
  }

  // -------------------------------------------------------------------------
  // the drafted tokens themselves
  // -------------------------------------------------------------------------
  // The node above a, -1 above a root.
  __device__ __forceinline__ int up_from(int a) const {
    if (!p.parent || a == 0) return a - 1;
    const int up = __ldg(p.parent + (long long)b * p.N + a);
    return up < a ? max(up, -1) : -1;
  }

  // Nodes of [j0, j0 + 16) that node n sees, as bits.
  __device__ __forceinline__ unsigned above(int n, int j0) const {
    unsigned bits = 0;
    int a = n;
    for (int step = 0; a >= j0 && (p.window == 0 || step < p.window); ++step) {
      if (a < j0 + kGran) bits |= 1u << (a - j0);
      a = up_from(a);
    }
    return bits;
  }

  // 4 consecutive activations; `wide`: on a multiple of their 4 elements
  __device__ __forceinline__ float4 act4(const void *base, long long at, bool wide) const {
    if (!wide) return act4_narrow(base, at);
    if (kF32) return __ldg(reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(base) + at));
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(reinterpret_cast<const unsigned short *>(base) + at));
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
  }
  static __device__ __noinline__ float4 act4_narrow(const void *base, long long at) {
    constexpr int dt = kF32 ? SPECDEC_F32 : SPECDEC_BF16;
    return make_float4(load_elem(base, dt, at), load_elem(base, dt, at + 1), load_elem(base, dt, at + 2),
                       load_elem(base, dt, at + 3));
  }
  __device__ __forceinline__ bool wide_rows(const void *base, long long stride) const {
    constexpr int bytes = kF32 ? 16 : 8;
    return ((reinterpret_cast<uintptr_t>(base) | (uintptr_t)(stride * (bytes / 4))) & (bytes - 1)) == 0;
  }
  static __device__ __forceinline__ float size_of(float x) {  // of what is finite
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.0f;
  }
  static __device__ __forceinline__ float top4(const float4 &x) {
    return fmaxf(fmaxf(size_of(x.x), size_of(x.y)), fmaxf(size_of(x.z), size_of(x.w)));
  }

  static __device__ __forceinline__ bool finite4(const float4 &x) {
    return finite(x.x) && finite(x.y) && finite(x.z) && finite(x.w);
  }

  // q . k of one row and one drafted token, from global memory, term by term.
  static __device__ __noinline__ float plain_dot(const void *q, long long q_at, const void *k,
                                                 long long k_at, int D) {
    constexpr int dt = kF32 ? SPECDEC_F32 : SPECDEC_BF16;
    float s = 0.0f;
#pragma unroll 1
    for (int e = 0; e < D; ++e) s = fmaf(load_elem(q, dt, q_at + e), load_elem(k, dt, k_at + e), s);
    return s;
  }

  __device__ __forceinline__ void drafted(int j0) {
    const specdec_kv_cache &kv = p.cache;
    const long long first = (long long)b * p.N + j0;
    const int held = min(nodes - j0, kGran);
    const bool k_wide = wide_rows(p.k_new, p.k_stride), v_wide = wide_rows(p.v_new, p.v_stride);
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);

    // q k^T, the node's k in units of its size
    float s[1][2][4], unit_k[2];
    unsigned odd = 0;  // tokens whose k is not finite
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const int t = nt * 8 + g;
      const long long at = (first + t) * p.k_stride + (long long)h * kv.D;
      float4 x[KC][4];
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < KC; ++i)
#pragma unroll
        for (int sub = 0; sub < 4; ++sub) {
          const int e = (c + 4 * i) * 16 + sub * 4;
          x[i][sub] = (t < held && e < kv.D) ? act4(p.k_new, at + e, k_wide) : zero;
        }
#pragma unroll
      for (int i = 0; i < KC; ++i)
#pragma unroll
        for (int sub = 0; sub < 4; ++sub) {
          top = fmaxf(top, top4(x[i][sub]));
          if (!finite4(x[i][sub])) odd |= 1u << t;
        }
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
      const int ex = unit_exponent(top);
      unit_k[nt] = pow2i(ex);
      const float inv = pow2i(-ex);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[0][nt][e] = 0.0f;
#pragma unroll
      for (int i = 0; i < KC; ++i)
#pragma unroll
        for (int sub = 0; sub < 4; ++sub) {
          const float4 y = make_float4(x[i][sub].x * inv, x[i][sub].y * inv, x[i][sub].z * inv,
                                       x[i][sub].w * inv);
          const uint32_t b0 = pack_half2(y.x, y.y), b1 = pack_half2(y.z, y.w);
          const uint4 qa = sm.q[i * 4 + sub][lane];
          const uint32_t a[4] = {qa.x, qa.y, qa.z, qa.w};
          mma16816(s[0][nt], a, b0, b1);
          if (kF32) {
            const uint32_t l0 = low_half2(y.x, y.y, b0), l1 = low_half2(y.z, y.w, b1);
            const uint4 ql = sm.q_lo[i * 4 + sub][lane];
            const uint32_t al[4] = {ql.x, ql.y, ql.z, ql.w};
            mma16816(s[0][nt], al, b0, b1);
            mma16816(s[0][nt], a, l0, l1);
          }
        }
    }
    unsigned see[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) see[i] = live[i] ? above(node[i], j0) : 0u;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = e >> 1, t = nt * 8 + 2 * c + (e & 1);
        // column t's unit is with the lanes of group t % 8
        const float unit = __shfl_sync(kAll, unit_k[nt], (2 * c + (e & 1)) * 4);
        const bool seen = (see[i] >> t) & 1u;
        const int dist = p.slopes && seen ? pos[i] - len - depth_of(j0 + t) : 0;
        s[0][nt][e] = seen ? score(s[0][nt][e], unit, i, dist) : -INFINITY;
      }
    odd = __reduce_or_sync(kAll, odd);
    if (odd) {  // infinities times the zeros of the other terms are not what q . k is
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll 1
        for (int n = 0; n < 4; ++n) {
          const int t = (n >> 1) * 8 + 2 * c + (n & 1);
          if (!(odd >> t & see[i] >> t & 1u)) continue;
          const int row = row0() + g + 8 * i;
          const float dot = plain_dot(p.q,
                                      ((long long)b * p.N + node[i]) * p.q_stride +
                                          (long long)(h * p.G + row - node[i] * p.G) * kv.D,
                                      p.k_new, (first + t) * p.k_stride + (long long)h * kv.D, kv.D);
          const float y = score(dot, __fdiv_rn(1.0f, sm.q_exp[g + 8 * i]), i,
                                p.slopes ? pos[i] - len - depth_of(j0 + t) : 0);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k == n) s[0][k >> 1][2 * i + (k & 1)] = y;
        }
      __syncwarp();
    }
    // p v, the node's v in units of its size; tokens 2c, 2c + 1, 2c + 8, 2c + 9
    float4 x[4][VB / 4];
    float unit_v[4], inv_v[4];  // the unit's exponent, and 1 / unit
    unsigned hit = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = (j >> 1) * 8 + 2 * c + (j & 1);
      const long long at = (first + t) * p.v_stride + (long long)h * kv.D;
#pragma unroll
      for (int i = 0; i < VB / 4; ++i) {
        const int e = g * VB + 4 * i;
        x[j][i] = (t < held && e < kv.D) ? act4(p.v_new, at + e, v_wide) : zero;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = (j >> 1) * 8 + 2 * c + (j & 1);
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < VB / 4; ++i) {
        float4 &y = x[j][i];
        top = fmaxf(top, top4(y));
        if (!finite4(y)) {
          hit |= 1u << t;
          y.x = finite(y.x) ? y.x : 0.0f;
          y.y = finite(y.y) ? y.y : 0.0f;
          y.z = finite(y.z) ? y.z : 0.0f;
          y.w = finite(y.w) ? y.w : 0.0f;
        }
      }
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
      const int ex = unit_exponent(top);
      unit_v[j] = (float)ex;
      inv_v[j] = pow2i(-ex);
    }
    hit = __reduce_or_sync(kAll, hit);
    raise<false>(s[0], unit_v);
    const float one[4] = {1.0f, 1.0f, 1.0f, 1.0f};
    uint32_t a[4], a_lo[4];
    weights(s[0], unit_v, one, a, a_lo);
#pragma unroll
    for (int i = 0; i < VB / 4; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int n = 4 * i + k;
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          y[j] = (k == 0 ? x[j][i].x : k == 1 ? x[j][i].y : k == 2 ? x[j][i].z : x[j][i].w) * inv_v[j];
        const uint32_t b0 = pack_half2(y[0], y[1]), b1 = pack_half2(y[2], y[3]);
        mma16816(o[n], a, b0, b1);
        if (kF32) {
          mma16816(o[n], a_lo, b0, b1);
          mma16816(o[n], a, low_half2(y[0], y[1], b0), low_half2(y[2], y[3], b1));
        }
      }
    if (hit) {  // infinities and NaN reach the rows that see their node, no others ...
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // ... and not under a score of -infinity
        unsigned none = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (s[0][k >> 1][2 * i + (k & 1)] == -INFINITY) none |= 1u << ((k >> 1) * 8 + 2 * c + (k & 1));
        none |= __shfl_xor_sync(kAll, none, 1);
        see[i] &= ~(none | __shfl_xor_sync(kAll, none, 2));
      }
    }
    while (hit) {
      const int t = __ffs(hit) - 1;
      hit &= hit - 1;
#pragma unroll 1
      for (int n = 0; n < 4 * NT; ++n) {
        const int d = column(n >> 2, n & 3);
        if (d < kv.D && ((see[(n >> 1) & 1] >> t) & 1u)) {
          const float y = act(p.v_new, (first + t) * p.v_stride + (long long)h * kv.D + d);
          if (!finite(y)) add_to(n >> 2, n & 3, y);
        }
      }
    }
  }

  // o[n][e] += y with n, e known only at run time (o stays in registers)
  __device__ __forceinline__ void add_to(int n, int e, float y) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j == n && k == e) o[j][k] += y;
  }

  // what fp16 left of (x0, x1); nothing where they are not finite
  __device__ __forceinline__ uint32_t low_half2(float x0, float x1, uint32_t hi) const {
    const float l0 = x0 - half_bits_to_float(hi & 0xFFFFu), l1 = x1 - half_bits_to_float(hi >> 16);
    return pack_half2(finite(l0) ? l0 : 0.0f, finite(l1) ? l1 : 0.0f);
  }

  __device__ __forceinline__ int depth_of(int n) const {
    if (!p.parent) return n;
    int depth = 0;
    for (int a = up_from(n); a >= 0; a = up_from(a)) ++depth;
    return depth;
  }

  // -------------------------------------------------------------------------
  __device__ __forceinline__ void run() {
    const int row0 = this->row0(), R = p.N * p.G;
    const specdec_kv_cache &kv = p.cache;
    int bad = 0;
    len = kv.length[b];
    if (len < 0 || (long long)len > (long long)kv.max_blocks * kv.block) {
      bad = SPECDEC_ROW_BAD_CACHE;
      len = 0;
    }
    nodes = p.N;
    if (p.n_nodes) {
      nodes = p.n_nodes[b];
      if (nodes < 0 || nodes > p.N) {
        bad |= SPECDEC_ROW_BAD_TREE;
        nodes = 0;
      }
    }
    if (p.parent) {
      bool wrong = false;
      for (int n = threadIdx.x; n < nodes; n += kThreads) {
        const int up = p.parent[(long long)b * p.N + n];
        wrong |= n == 0 ? up != -1 : (up < 0 || up >= n);
      }
      if (__syncthreads_or(wrong)) bad |= SPECDEC_ROW_BAD_TREE;
    }

    // q: rows to fp16 by a power of two each, in operand order; a lane takes 4
    // elements of a row (8 of 256), one lane's part of one step
    constexpr int kPer = DP > 128 ? 2 : 1, kMine = kRows / kWarps;
    const bool q_wide = wide_rows(p.q, p.q_stride);
    float4 qx[kMine][kPer];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int row = row0 + warp + kWarps * i, n = row / p.G;
      const bool in = row < R && n < nodes;
      const long long at = in ? ((long long)b * p.N + n) * p.q_stride +
                                    (long long)(h * p.G + row - n * p.G) * kv.D
                              : 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int e = 4 * (lane + 32 * k);
        qx[i][k] = (in && e < kv.D) ? act4(p.q, at + e, q_wide) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
    }
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int r = warp + kWarps * i;
      float top = 0.0f;
      bool all = true;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        top = fmaxf(top, top4(qx[i][k]));
        all &= finite4(qx[i][k]);
      }
      all = __all_sync(kAll, all);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
      const int ex = unit_exponent(top);
      const float inv = pow2i(-ex);
      // a q that is not finite makes its row NaN
      if (lane == 0) sm.q_exp[r] = all ? pow2i(ex) : __int_as_float(0x7fc00000);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int w = lane + 32 * k;
        if (w >= DP / 4) continue;
        const float4 x = make_float4(qx[i][k].x * inv, qx[i][k].y * inv, qx[i][k].z * inv,
                                     qx[i][k].w * inv);
        const int piece = w >> 2, sub = w & 3;           // 16-element piece, step in it
        const int cc = piece & 3, ks = (piece >> 2) * 4 + sub;
        uint32_t *dst = reinterpret_cast<uint32_t *>(&sm.q[ks][(r & 7) * 4 + cc]);
        const uint32_t x01 = pack_half2(x.x, x.y), x23 = pack_half2(x.z, x.w);
        dst[r >> 3] = x01;
        dst[2 + (r >> 3)] = x23;
        if (kF32) {
          dst = reinterpret_cast<uint32_t *>(&sm.q_lo[ks][(r & 7) * 4 + cc]);
          dst[r >> 3] = low_half2(x.x, x.y, x01);
          dst[2 + (r >> 3)] = low_half2(x.z, x.w, x23);
        }
      }
    }
    __syncthreads();

#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i, row = row0 + r;
      node[i] = row / p.G;
      live[i] = row < R && node[i] < nodes;
      pos[i] = len + (live[i] && (p.slopes || p.window > 0) ? depth_of(node[i]) : 0);
      rf[i] = (kPlain ? p.scale * kLog2e : p.scale) * sm.q_exp[r];
      slope[i] = (p.slopes && live[i]) ? p.slopes[h * p.G + row - node[i] * p.G] : 0.0f;
      m[i] = ko[i] = -INFINITY;
      l[i] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;

    if (nodes > 0) {
      // the split's share of the granules: those of the tokens that the window
      // leaves, then the drafted ones
      int from = p.window > 0 ? max(0, len - p.window + 1) : 0;
      from = from / kGran * kGran;
      const int cached_n = (len - from + kGran - 1) / kGran, all_n = cached_n + (nodes + kGran - 1) / kGran;
      const int share = (all_n + p.splits - 1) / p.splits;
      const int g0 = min(all_n, split * share), g1 = min(all_n, g0 + share);
      const int c1 = min(g1, cached_n);
      if (g0 < c1 && !cached(from + g0 * kGran, min(len, from + c1 * kGran)))
        bad |= SPECDEC_ROW_BAD_CACHE;
      // drafted ones go on where the cached ones leave the warps
      for (int i = max(g0, cached_n); i < g1; ++i)
        if ((i - g0) % kWarps == warp) drafted((i - cached_n) * kGran);
    }

    // quads hold parts of l; rows past the request's nodes took part unmasked
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!live[i]) {
        m[i] = ko[i] = -INFINITY;
        l[i] = 0.0f;
      }
      l[i] += __shfl_xor_sync(kAll, l[i], 1);
      l[i] += __shfl_xor_sync(kAll, l[i], 2);
      // maxima pass over NaN scores, sums do not: where all were NaN the row has a
      // maximum of 0 from here on, as one without would count as having seen nothing
      if (l[i] != l[i] && m[i] == -INFINITY) m[i] = ko[i] = 0.0f;
    }
    bad = __reduce_or_sync(kAll, bad);
    if (c == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sm.m[warp][g + 8 * i] = m[i];
        sm.l[warp][g + 8 * i] = l[i];
        sm.ko[warp][g + 8 * i] = ko[i];
      }
    }
    if (lane == 0) sm.bad[warp] = bad;
    __syncthreads();
    // every warp moves to the common maxima
    float all[2], all_o[2], sum[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      all[i] = all_o[i] = -INFINITY;
      for (int w = 0; w < kWarps; ++w) all[i] = fmaxf(all[i], sm.m[w][r]);
      for (int w = 0; w < kWarps; ++w)
        if (sm.m[w][r] > -INFINITY) all_o[i] = fmaxf(all_o[i], sm.m[w][r] - all[i] + sm.ko[w][r]);
      sum[i] = 0.0f;
      for (int w = 0; w < kWarps; ++w)
        if (sm.m[w][r] > -INFINITY) sum[i] += sm.l[w][r] * ex2_approx(sm.m[w][r] - all[i]);
      const float f = m[i] > -INFINITY ? ex2_approx(m[i] - all[i] + ko[i] - all_o[i]) : 0.0f;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        o[j][2 * i] = m[i] > -INFINITY ? o[j][2 * i] * f : 0.0f;
        o[j][2 * i + 1] = m[i] > -INFINITY ? o[j][2 * i + 1] * f : 0.0f;
      }
    }
    bad = 0;
    for (int w = 0; w < kWarps; ++w) bad |= sm.bad[w];
#pragma unroll
    for (int step = kWarps / 2; step >= 1; step >>= 1) {
      if (warp >= step && warp < 2 * step) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sm.o[warp - step][g + 8 * (e >> 1)][column(j, e)] = o[j][e];
      }
      __syncthreads();
      if (warp < step) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[j][e] += sm.o[warp][g + 8 * (e >> 1)][column(j, e)];
      }
      __syncthreads();
    }
    if (warp == 0) {  // the CTA's sums
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sm.o[0][g + 8 * (e >> 1)][column(j, e)] = o[j][e];
      if (c == 0)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sm.all_m[g + 8 * i] = all[i];
          sm.all_l[g + 8 * i] = sum[i];
          sm.all_ko[g + 8 * i] = all_o[i];
        }
      if (lane == 0) sm.all_bad = bad;
    }
    __syncwarp();
    const bool joined = p.splits > 1 && p.clustered;
    if (joined) {
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                       : "memory");
    } else {
      __syncthreads();
    }
    if (p.splits > 1 && !p.clustered) {
      float *part = p.part + ((((long long)b * kv.Hkv + h) * p.row_tiles + tile) * p.splits + split) *
                                 partial_floats(kv.D);
      for (int i = threadIdx.x; i < kRows * kv.D; i += kThreads)
        part[3 * kRows + i] = sm.o[0][i / kv.D][i % kv.D];
      if (threadIdx.x < kRows) {
        part[threadIdx.x] = sm.all_m[threadIdx.x];
        part[kRows + threadIdx.x] = bad ? -(float)bad : sm.all_l[threadIdx.x];
        part[2 * kRows + threadIdx.x] = sm.all_ko[threadIdx.x];
      }
      return;
    }
    // rows of this CTA: all of them, or its share of the cluster's
    const int parts = joined ? p.splits : 1, per = kRows / parts, r0 = joined ? split * per : 0;
    if (joined) {
      bad = 0;
      for (int s = 0; s < parts; ++s) bad |= __float_as_int(remote(reinterpret_cast<float *>(&sm.all_bad), s));
    }
    for (int i = warp; i < per; i += kWarps) {
      const int r = r0 + i, row = row0 + r;
      if (row >= R) break;
      const int n = row / p.G;
      const long long at = ((long long)b * p.N + n) * p.Hq + h * p.G + row - n * p.G;
      // (a part under a factor of 0 takes part all the same: its sums may be NaN)
      float f[8], fo[8], top = -INFINITY, top_o = -INFINITY, total = 0.0f;
      unsigned seen = 0;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        f[s] = s < parts ? (joined ? remote(&sm.all_m[r], s) : sm.all_m[r]) : -INFINITY;
        seen |= (unsigned)(f[s] > -INFINITY) << s;
        top = fmaxf(top, f[s]);
      }
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (seen >> s & 1u) {
          total += ex2_approx(f[s] - top) * (joined ? remote(&sm.all_l[r], s) : sm.all_l[r]);
          fo[s] = f[s] - top + (joined ? remote(&sm.all_ko[r], s) : sm.all_ko[r]);
          top_o = fmaxf(top_o, fo[s]);
        }
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (seen >> s & 1u) fo[s] = ex2_approx(fo[s] - top_o);
      const bool empty = bad || n >= nodes || top == -INFINITY;
      const float inv = empty ? 0.0f : 1.0f / total;
      for (int d = lane; d < kv.D; d += 32) {
        float x = 0.0f;
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (seen >> s & 1u) x += fo[s] * (joined ? remote(&sm.o[0][r][d], s) : sm.o[0][r][d]);
        store_out(at * kv.D + d, empty ? 0.0f : times_pow2(x * inv, top_o));
      }
      if (lane == 0 && p.lse)
        p.lse[at] = empty ? -INFINITY : (top - kLift + log2f(total)) * 0.6931471805599453f;
    }
    if (tile == 0 && h == 0 && r0 == 0 && threadIdx.x == 0) p.row_status[b] = bad;
    __syncwarp();
    if (joined)  // no CTA leaves while another reads its shared memory
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                       : "memory");
  }

  // A float of CTA `rank` of the cluster at this CTA's address `x`.
  __device__ __forceinline__ float remote(const float *x, int rank) const {
    float r;
    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                 : "=f"(r)
                 : "r"(cluster_addr(smem_addr(x), (uint32_t)rank))
                 : "memory");
    return r;
  }

  __device__ __forceinline__ void store_out(long long i, float x) const {
    if (kF32)
      reinterpret_cast<float *>(p.out)[i] = x;
    else
      reinterpret_cast<unsigned short *>(p.out)[i] = (unsigned short)pack_bf16x2(x, 0.0f);
  }
};

template <int DP, bool kF32, bool kPlain>
__global__ void __launch_bounds__(kThreads) attend_stream_kernel(const AttendParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  pdl_wait();
  pdl_launch_dependents();
  using K = Kernel<DP, kF32, kPlain>;
  K k(p, *reinterpret_cast<typename K::Smem *>(raw));
  k.run();
}

// Joins the splits of one row: a warp each.
__global__ void __launch_bounds__(256) attend_join_kernel(const AttendParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, D = p.cache.D, Hkv = p.cache.Hkv;
  const long long at = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);  // (b, n, query head)
  if (at >= (long long)p.B * p.N * p.Hq) return;
  const int hq = (int)(at % p.Hq), n = (int)(at / p.Hq % p.N), h = hq / p.G;
  const long long b = at / p.Hq / p.N;
  const int row = n * p.G + hq - h * p.G;
  const size_t stride = partial_floats(D);
  const float *part = p.part + (((b * Hkv + h) * p.row_tiles + row / kRows) * p.splits) * stride;
  const int r = row % kRows;
  // lane s holds split s and s + 32
  float m[2], l[2], ko[2];
  int bad = 0;
  float all = -INFINITY, all_o = -INFINITY;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = lane + 32 * i;
    m[i] = s < p.splits ? part[s * stride + r] : -INFINITY;
    l[i] = s < p.splits ? part[s * stride + kRows + r] : 0.0f;
    ko[i] = s < p.splits ? part[s * stride + 2 * kRows + r] : 0.0f;
    if (l[i] < 0.0f) bad |= (int)-l[i];
    all = fmaxf(all, m[i]);
  }
  bad = __reduce_or_sync(kAll, bad);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) all = fmaxf(all, __shfl_xor_sync(kAll, all, d));
  // (a part under a factor of 0 takes part all the same: its sums may be NaN)
  float f[2], sum = 0.0f;
  unsigned seen[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    seen[i] = __ballot_sync(kAll, m[i] > -INFINITY);
    f[i] = m[i] - all;
    if (m[i] > -INFINITY) {
      sum += l[i] * ex2_approx(f[i]);
      f[i] += ko[i];
      all_o = fmaxf(all_o, f[i]);
    }
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) all_o = fmaxf(all_o, __shfl_xor_sync(kAll, all_o, d));
#pragma unroll
  for (int i = 0; i < 2; ++i) f[i] = m[i] > -INFINITY ? ex2_approx(f[i] - all_o) : 0.0f;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
  const bool empty = bad != 0 || all == -INFINITY;
  const float inv = empty ? 0.0f : __fdividef(1.0f, sum);
  // four splits at a time, 128 elements of each, all loads before the sums
  // (all lanes take every round, as each holds splits' factors)
#pragma unroll 1
  for (int d0 = lane; d0 - lane < D; d0 += 128) {
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int s = 0; s < p.splits; s += 4) {
      float x[4][4], w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        // (not past the last split, nor of one without tokens)
        const bool in = (s < 32 ? seen[0] : seen[1]) >> ((s + u) & 31) & 1u;
        w[u] = __shfl_sync(kAll, s < 32 ? f[0] : f[1], (s + u) & 31);
        const float *rec = part + (s + u) * stride + 3 * kRows + r * D + d0;
#pragma unroll
        for (int k = 0; k < 4; ++k) x[u][k] = in && d0 + 32 * k < D ? rec[32 * k] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] += w[u] * x[u][k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int d = d0 + 32 * k;
      if (d >= D) continue;
      const float y = empty ? 0.0f : times_pow2(acc[k] * inv, all_o);
      if (p.dtype == SPECDEC_F32)
        reinterpret_cast<float *>(p.out)[at * D + d] = y;
      else
        reinterpret_cast<unsigned short *>(p.out)[at * D + d] = (unsigned short)pack_bf16x2(y, 0.0f);
    }
  }
  if (lane == 0) {
    if (p.lse) p.lse[at] = empty ? -INFINITY : (all - kLift + log2f(sum)) * 0.6931471805599453f;
    if (n == 0 && hq == 0) p.row_status[b] = bad;
  }
}

int row_tiles_of(int N, int G) { return (N * G + kRows - 1) / kRows; }

// Splits of the tokens: as many as give the device's SMs a few CTAs each; the
// most for any length, which sizes the workspace ...
int most_splits(long long B, int N, int Hkv, int G) {
  const long long ctas = B * Hkv * row_tiles_of(N, G);
  const long long s = 608 / ctas;  // 4 for each of 152 SMs
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}
// Granules that a request can hold: of what its blocks hold, or the window leaves.
long long granules_of(const AttendParams &p) {
  long long tokens = (long long)p.cache.max_blocks * p.cache.block;
  const long long reach = (long long)p.window + kGran;
  if (p.window > 0 && tokens > reach) tokens = reach;
  return (tokens + kGran - 1) / kGran + (p.N + kGran - 1) / kGran;
}
// ... and no more than leave each warp a granule where the cache is full; up to
// eight as a power of two, which a cluster joins.  More than eight go through the
// workspace, which pays once eight leave a warp more than 32 granules: one request
// of 5 (8 heads of 128, float32) takes 26.5 us with eight and 36.4 us with 33 over
// 2048 tokens, 66.8 and 62.4 over 16384, 230 and 133 over 65536.
int splits_of(const AttendParams &p) {
  const int most = most_splits(p.B, p.N, p.cache.Hkv, p.G);
  const long long granules = granules_of(p), useful = (granules + kWarps - 1) / kWarps;
  const long long s = useful < most ? useful : most;
  if (s >= 24 && granules > 8 * kWarps * 32) return (int)s;
  return s >= 8 ? 8 : s >= 4 ? 4 : s >= 2 ? 2 : 1;
}

template <int DP, bool kF32, bool kPlain>
cudaError_t launch_stream(const AttendParams &p, cudaStream_t stream) {
  static DeviceOnce once;
  const int smem = (int)sizeof(typename Kernel<DP, kF32, kPlain>::Smem);
  const cudaError_t err = smem_opt_in_once(once, attend_stream_kernel<DP, kF32, kPlain>, smem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.splits * p.row_tiles * p.B * p.cache.Hkv));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.clustered && p.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, attend_stream_kernel<DP, kF32, kPlain>, p);
}

// bfloat16 calls that the streaming kernel takes before the tiles' kernel: as many
// CTAs as run at once, two an SM, with up to 4 granules a warp, or 16 of narrow
// heads.  (us here and there: one request of 5 over 128 tokens 18.6 and 20.5, over
// 4096 28.8 and 28.7; 4 of 1 over 777 20.7 and 20.5, over 4096 30.2 and 24.7; 16 of
// 1 over 16 18.5 and 21.5, over 128, with 384 CTAs, 32.9 and 21.7; heads of 64, 16
// requests of 5 over 2048 26.6 and 30.5, over 4096 37.2 and 35.4.)
bool stream_is_quicker(const AttendParams &p) {
  const long long ctas = (long long)p.B * p.cache.Hkv * p.row_tiles * p.splits;
  return ctas <= 304 && granules_of(p) <= (long long)p.splits * kWarps * (p.cache.D <= 64 ? 16 : 4);
}

template <bool kF32, bool kPlain>
cudaError_t launch_type(const AttendParams &p, cudaStream_t stream) {
  if (p.cache.D <= 64) return launch_stream<64, kF32, kPlain>(p, stream);
  if (p.cache.D <= 128) return launch_stream<128, kF32, kPlain>(p, stream);
  return launch_stream<256, kF32, kPlain>(p, stream);
}

}  // namespace

size_t attend_workspace_bytes(long long B, int N, int Hq, int Hkv, int D, int dtype) {
  const int G = Hq / Hkv, s = most_splits(B, N, Hkv, G);
  const size_t stream =
      s <= 8 ? 0 : (size_t)B * Hkv * row_tiles_of(N, G) * s * partial_floats(D) * sizeof(float);
  // which kernel a call takes depends on the pool too, which the sizes here do not name
  const size_t tile = dtype == SPECDEC_BF16 && D <= 128 ? attend_tile_workspace_bytes(N, G, D) : 0;
  return stream > tile ? stream : tile;
}

cudaError_t launch_attend(AttendParams p, cudaStream_t stream) {
  p.row_tiles = row_tiles_of(p.N, p.G);
  p.splits = splits_of(p);
  p.clustered = p.splits <= 8;
  p.block_shift = -1;
  for (int i = 4; i < 12; ++i)
    if (p.cache.block == 1 << i) p.block_shift = i;
  if (attend_tile_applies(p) && !stream_is_quicker(p)) return launch_attend_tile(p, stream);
  const bool plain = p.softcap == 0.0f && !p.slopes;
  cudaError_t err =
      p.dtype == SPECDEC_F32
          ? (plain ? launch_type<true, true>(p, stream) : launch_type<true, false>(p, stream))
          : (plain ? launch_type<false, true>(p, stream) : launch_type<false, false>(p, stream));
  if (err != cudaSuccess || p.clustered) return err;
  const long long rows = (long long)p.B * p.N * p.Hq;
  return launch_pdl(attend_join_kernel, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, stream, p);
}

}  // namespace specdec
