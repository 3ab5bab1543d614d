// Divergence of a draft's row from the K entries of a teacher's record, and its gradient
// (specdec_distill).  With s = softmax(x / T) over the row and p_j the teacher's share of
// entry j (token id_j):
//     L = sum_j p_j (ln p_j - ln s_id_j) + r (ln r - ln s_rest)
//     dL/dx_v = (P s_v - p_v) / T at an entry's token, (P s_v - r s_v / s_rest) / T elsewhere,
// r = max(0, 1 - sum p_j), P = r + sum p_j (1 but for records of more than 1) and s_rest = the
// mass of s outside the entries when the teacher's log-sum-exp is given; without it p = softmax
// over the entries, r = 0 and P = 1.
//
// A row is held in shared memory by a cluster of CTAs: it is read from HBM once, whatever
// is computed from it, and the gradient is written once.  While the copies land, the
// teacher's shares are made; then each CTA's maximum, and its sum of exponentials with the
// entries taken out (their logits put to -infinity in shared memory, so that s_rest is a sum
// and no difference of two near equal ones); one exchange of five words between the CTAs;
// the gradient, straight from registers to global memory, then the entries' own values.  The
// loss is sum p_j (z_j - x_j) / T + sum p_j (max / T + ln S - lse), S the row's sum against
// its maximum: parts of some units each, whose sum may be a thousandth.  The entries' terms and
// weights are pairs of float32 added in 64-bit fixed point (an SM has two lanes for 64-bit
// floating point; with them the kernel took 1790 us in place of 434), and the last few steps of
// a row are 64-bit.
//
// Measured: 4096 rows of 128256 bfloat16, 64 entries, gradient out: 449 us, 4.7 TB/s, 70 % of the
// measured copy rate, the loss alone 293; 4080 rows of 32003 bfloat16: 99 us, 70 %; 508 rows of
// 152064 float32: 144 us, 64 %; 33 rows of 32000 float32: 10.3 us.  Of a CTA's 23000 clocks (three an SM) its share's
// arrival takes 7600, the sum 3300, the exchange 3000, the loss 2200, the gradient 5000: the
// chain of those steps, which three CTAs overlap in part, is what keeps it from the copy rate.
// Records that complete on an mbarrier, in place of the cluster's barrier: 1 % less, and 1 us more for
// the smallest call.  The pairs of the loss cost 4 % (434 us with float32 terms, whose loss was off
// by 2e-7, in place of 450 at that time; with the last steps in 64-bit floating point 485).
#include "draft_common.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPerThread = SPECDEC_MAX_TOPK / kThreads;

struct DistillSmem {
  Exchange ex;
  Arrival in;
  long long terms[3][kWarps];
  float red[4][kWarps];
  int status;
  int entries;
};

constexpr float kTerm = 0x1p40f;  // units of the fixed-point sums
constexpr float kMost = 0x1p12f;  // terms that they take (1024 of them); the larger are added
                                  // in float32, where a loss with such a term ends anyway (shares
                                  // that large are refused)

// Dynamic shared memory: DistillSmem, the share, one bit for each of its elements, and a
// position, logit and teacher's share for each entry.
struct Layout {
  int share, bits, pos, total;
};

__host__ __device__ inline Layout layout_of(int vectors, int elem_bytes, int K) {
  Layout l;
  l.share = ((int)sizeof(DistillSmem) + 127) / 128 * 128;
  l.bits = l.share + vectors * 16;
  l.pos = l.bits + (vectors * (16 / elem_bytes) + 31) / 32 * 4;
  l.total = l.pos + K * 12;
  return l;
}

// ---- what the loss is made of, to about 1e-9 ------------------------------------------

// A value as the sum of two.
struct Two {
  float hi, lo;
};

// (a - b) / T
__device__ __forceinline__ Two over_t(float a, float b, float inv_t, float inv_t_low) {
  const float d = a - b, z = d - a;
  const float d_low = (a - (d - z)) - (b + z);
  const float y = d * inv_t;
  return {y, fmaf(d, inv_t, -y) + fmaf(d, inv_t_low, d_low * inv_t)};
}

// e^y for |y| < 87 (and no more than float32's beyond): y log2(e) = n + g, |g| <= 1/2, and
// 2^g = 1 + g ln 2 + r by the series, the first two terms exact.
__device__ __forceinline__ Two exp_two(Two y) {
  if (!(fabsf(y.hi) < 87.0f)) return {expf(y.hi), 0.0f};
  constexpr float kHi = kLog2e, kLo = 1.9259629e-8f, kMagic = 12582912.0f;  // 1.5 * 2^23
  constexpr float kLn2 = 0.693147181f, kLn2Low = -1.90465422e-9f;
  const float t = fmaf(y.hi, kHi, kMagic);
  const float g = fmaf(y.hi, kHi, kMagic - t) + fmaf(y.hi, kLo, y.lo * kHi);
  float r = 1.32154867e-6f;  // ln^i 2 / i!, i = 8 .. 2
  r = fmaf(g, r, 1.52527338e-5f);
  r = fmaf(g, r, 1.54035304e-4f);
  r = fmaf(g, r, 1.33335581e-3f);
  r = fmaf(g, r, 9.61812911e-3f);
  r = fmaf(g, r, 5.55041087e-2f);
  r = fmaf(g, r, 2.40226507e-1f);
  const float h = g * kLn2, one = 1.0f + h;
  const float low = (h - (one - 1.0f)) + fmaf(g, kLn2Low, fmaf(g, kLn2, -h));
  const float scale = __int_as_float((__float_as_int(t) - __float_as_int(kMagic) + 127) << 23);
  return {one * scale, fmaf(g * g, r, low) * scale};
}

__device__ __forceinline__ long long fixed_two(Two x) {
  return __float2ll_rn(x.hi * kTerm) + __float2ll_rn(x.lo * kTerm);
}

// ln(v + low) in units of 2^-40, v > 0 a normal number: v = 2^e f with f in [3/4, 3/2), ln f =
// 2 atanh u by its series, u = (f - 1) / (f + 1) as a pair, |u| <= 1/5.
__device__ __forceinline__ long long ln_fixed(float v, float low) {
  const int e = (__float_as_int(v) - 0x3F400000) >> 23;
  const float f = __int_as_float(__float_as_int(v) - (e << 23));
  const float num = f - 1.0f, den = f + 1.0f, den_low = f - (den - 1.0f);
  const float by = __fdividef(1.0f, den), u = num * by, u2 = u * u;
  const float u_low = by * (fmaf(-u, den, num) - u * den_low);
  float r = 1.0f / 15.0f;
  r = fmaf(u2, r, 1.0f / 13.0f);
  r = fmaf(u2, r, 1.0f / 11.0f);
  r = fmaf(u2, r, 1.0f / 9.0f);
  r = fmaf(u2, r, 1.0f / 7.0f);
  r = fmaf(u2, r, 1.0f / 5.0f);
  r = fmaf(u2, r, 1.0f / 3.0f);
  const float rest = 2.0f * fmaf(u * u2, r, u_low) + __fdividef(low, v);
  return (long long)e * 762123384786ll + fixed_two({2.0f * u, rest});
}

// a b of numbers in units of 2^-40
__device__ __forceinline__ long long mul_fixed(long long a, long long b) {
  return (long long)((unsigned long long)__mul64hi(a, b) << 24 | (unsigned long long)(a * b) >> 40);
}

template <int DT, bool kGrad>
__global__ void __launch_bounds__(kThreads, 3) distill_kernel(const DistillParams p, int vectors) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  constexpr int es = Elem<DT>::kBytes, kN = Elem<DT>::kN;
  DistillSmem &sm = *reinterpret_cast<DistillSmem *>(smem_raw);
  const Layout l = layout_of(vectors, es, p.K);
  uint8_t *buf = smem_raw + l.share;
  uint32_t *bits = reinterpret_cast<uint32_t *>(smem_raw + l.bits);
  int *pos = reinterpret_cast<int *>(smem_raw + l.pos);
  float *at_x = reinterpret_cast<float *>(pos + p.K);
  float *at_p = at_x + p.K;
  const int tid = threadIdx.x;
  const int rank = cluster_rank(), size = cluster_size();
  const long long n = blockIdx.x / size;  // the row
  const long long b = n / p.R;
  const int r = (int)(n - b * p.R);
  int turn = 0;

  if (tid == 0) {
    for (int i = 0; i < kChunks; ++i) mbar_init(&sm.in.full[i], 1);
    sm.in.gave_up = 0;
    sm.status = 0;
    sm.entries = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  cluster_arrive_relaxed();  // all CTAs run before one writes to another (waited for below)
  __syncthreads();

  const uint8_t *row = reinterpret_cast<const uint8_t *>(p.x) +
                       (b * p.x_at.request + r * p.x_at.row) * es;
  uint8_t *out = kGrad ? reinterpret_cast<uint8_t *>(p.grad) +
                             (b * p.grad_at.request + r * p.grad_at.row) * es
                       : nullptr;
  const Share s = share_of<DT>(row, p.V, rank, size);
  float w = p.weight ? p.weight[n] : 1.0f;
  if (p.dloss) {
    const float d = p.dloss[n];
    if (d == 1.0f) {  // the gradient that stands there is the one
      cluster_wait();
      return;
    }
    if (w != 0.0f) w *= d;
  }

  // the entries: K <= 4 a thread, their ids and logits in registers
  int id[kPerThread];
  float z[kPerThread];
  float zmax = -INFINITY, lse = 0.0f;
  int status = 0, some = 0;
  if (w != 0.0f) {
    if (tid == 0) share_copy(s, buf, sm.in);
    if (p.lse) lse = p.lse[n];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int j = tid + i * kThreads;
      id[i] = -1;
      z[i] = -INFINITY;
      if (j < p.K) {
        id[i] = p.ids[n * p.K + j];
        z[i] = p.teacher[n * p.K + j];
      }
    }
    share_edges<DT>(s, row, buf);
    for (int i = tid; i < (l.pos - l.bits) / 4; i += kThreads) bits[i] = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      if (id[i] < -1 || id[i] >= p.V) {
        status |= SPECDEC_ROW_BAD_TOKEN;
        id[i] = -1;
      }
      if (id[i] < 0) {
        z[i] = -INFINITY;
        continue;
      }
      some = 1;
      if (!(z[i] < INFINITY)) status |= SPECDEC_ROW_NONFINITE;
      zmax = fmaxf(zmax, z[i]);
    }
    if (!(fabsf(w) < INFINITY)) status |= SPECDEC_ROW_NONFINITE;
  }
  some = __syncthreads_or(some);
  const bool wrong = __syncthreads_or(status) != 0;
  cluster_wait();
  // a row without weight or entries: nothing to learn, whatever its logits hold
  const bool none = w == 0.0f || (!some && !wrong);

  const float c = temperature_scale(p.temperature);
  float m = -INFINITY;
  const unsigned long long(*got)[kWords] = nullptr;
  float coef = 0.0f, M = 0.0f, inv_s = 0.0f, left = 0.0f, inv_zs = 1.0f;
  long long mass = 0;
  int st = 0;
  if (w != 0.0f) {
    // p_j = e^y_j / zs: y_j = z_j / T - lse and zs = 1, or y_j = (z_j - zmax) / T
    if (p.lse) {
      if (!(fabsf(lse) < INFINITY)) status |= SPECDEC_ROW_NONFINITE;
      zmax = 0.0f;
    } else {
      zmax = cta_max_nan<kWarps>(zmax, sm.red[0]);
      if (some && !(zmax > -INFINITY)) status |= SPECDEC_ROW_NONFINITE;
    }
    if (!p.lse) {
      // (the loss goes by the sum of the shares that this leads to: it need not be exact)
      float zs = 0.0f;
#pragma unroll
      for (int i = 0; i < kPerThread; ++i)
        if (z[i] > -INFINITY) zs += ex2_approx((z[i] - zmax) * c);
      inv_zs = 1.0f / cta_sum<kWarps>(zs, sm.red[1]);
    }

    // the shares of this CTA's entries
    float pj[kPerThread];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      pj[i] = 0.0f;
      if (id[i] < s.begin || id[i] >= s.end) continue;
      mine = 1;
      if (!(z[i] > -INFINITY)) continue;
      Two y = over_t(z[i], zmax, p.inv_t, p.inv_t_low);
      const float l = y.hi - lse, q = l - y.hi;
      y.lo += (y.hi - (l - q)) - (lse + q);
      y.hi = l;
      const Two e = exp_two(y);
      pj[i] = (e.hi + e.lo) * inv_zs;
    }

    // the largest logit, as the copies land
    uint32_t top = no_max<DT>();
    for (int i = 0; i < kChunks; ++i) {
      share_wait(sm.in, i);
      const int v1 = 1 + chunk_begin(s, i + 1);
      for (int v = 1 + chunk_begin(s, i) + tid; v < v1; v += kThreads)
        top = vector_max<DT>(*reinterpret_cast<const uint4 *>(buf + (size_t)v * 16), top);
    }
    if (tid < 2)
      top = vector_max<DT>(
          *reinterpret_cast<const uint4 *>(buf + (size_t)(tid ? s.nvec - 1 : 0) * 16), top);
    m = cta_max_nan<kWarps>(max_of<DT>(top), sm.red[2]);
    const float ref = m > -INFINITY ? m : 0.0f;

    // this CTA's entries: noted, and taken out of the row
    float large = 0.0f;
    long long terms = 0, at_mass = 0, at_s = 0;  // sums of p_j (z_j - x_j) / T, p_j, e^((x_j - ref) / T)
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      if (id[i] < s.begin || id[i] >= s.end) continue;
      const int at = id[i] - s.first;
      if (atomicOr(&bits[at >> 5], 1u << (at & 31)) >> (at & 31) & 1u) {
        status |= SPECDEC_ROW_BAD_TOKEN;  // the same token twice
        continue;
      }
      const float x = get_elem<DT>(buf + (size_t)at * es);
      put_elem<DT>(buf + (size_t)at * es, -INFINITY);
      at_s += fixed_two(exp_two(over_t(x, ref, p.inv_t, p.inv_t_low)));
      if (pj[i] > 0.0f) {
        const Two d = over_t(z[i], x, p.inv_t, p.inv_t_low);
        const float t = pj[i] * d.hi;
        if (fabsf(t) < kMost)
          terms += fixed_two({t, fmaf(pj[i], d.hi, -t) + pj[i] * d.lo});
        else
          large += x > -INFINITY ? t : INFINITY;
        at_mass += __float2ll_rn(fminf(pj[i], kMost) * kTerm);
        if (pj[i] > kMost) status |= SPECDEC_ROW_NONFINITE;
      }
      const int k = atomicAdd(&sm.entries, 1);  // (their order decides nothing)
      pos[k] = at;
      at_x[k] = x;
      at_p[k] = pj[i];
    }
    if (__any_sync(kFull, mine)) {
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) {
        terms += __shfl_xor_sync(kFull, terms, d);
        at_mass += __shfl_xor_sync(kFull, at_mass, d);
        at_s += __shfl_xor_sync(kFull, at_s, d);
        large += __shfl_xor_sync(kFull, large, d);
      }
    }
    if ((tid & 31) == 0) {
      sm.terms[0][tid >> 5] = terms;
      sm.terms[1][tid >> 5] = at_mass;
      sm.terms[2][tid >> 5] = at_s;
      sm.red[3][tid >> 5] = large;
    }
    if (status) atomicOr(&sm.status, status);
    __syncthreads();
    float2 sum0 = both(0.0f), sum1 = both(0.0f);
    for (int v = tid; v < s.nvec; v += kThreads) {
      float2 x[kN / 2];
      widen2<DT>(*reinterpret_cast<const uint4 *>(buf + (size_t)v * 16), x);
#pragma unroll
      for (int e = 0; e < kN / 2; e += 2) {
        sum0 = __fadd2_rn(sum0, exp2_pair(x[e], ref, c));
        sum1 = __fadd2_rn(sum1, exp2_pair(x[e + 1], ref, c));
      }
    }
    sum0 = __fadd2_rn(sum0, sum1);
    float rest = sum0.x + sum0.y;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) rest += __shfl_xor_sync(kFull, rest, d);
    if ((tid & 31) == 0) sm.red[0][tid >> 5] = rest;
    __syncthreads();
    unsigned long long rec[kWords];
    if (tid < 32) {
      rest = large = 0.0f;
      terms = at_mass = at_s = 0;
      for (int k = 0; k < kWarps; ++k) {
        rest += sm.red[0][k];
        large += sm.red[3][k];
        terms += sm.terms[0][k];
        at_mass += sm.terms[1][k];
        at_s += sm.terms[2][k];
      }
      const int wrong_here = sm.status | (sm.in.gave_up ? SPECDEC_ROW_INTERNAL : 0);
      rec[0] = (unsigned long long)at_s;
      rec[1] = (unsigned long long)(uint32_t)wrong_here << 32 | __float_as_uint(m);
      rec[2] = (unsigned long long)terms;
      rec[3] = (unsigned long long)at_mass;
      rec[4] = (unsigned long long)__float_as_uint(large) << 32 | __float_as_uint(rest);
    }
    got = exchange(sm.ex, turn, rec, 5, rank, size);

    M = -INFINITY;
    for (int k = 0; k < size; ++k) {
      M = fmax_nan(M, __uint_as_float((uint32_t)got[k][1]));
      st |= (int)(got[k][1] >> 32);
      mass += (long long)got[k][3];
    }
    if (!(M > -INFINITY && M <= kMaxLogit)) st |= SPECDEC_ROW_NONFINITE;
    if (none) st = 0;
    float others = 0.0f, S = 0.0f;
    for (int k = 0; k < size; ++k) {
      const float mk = __uint_as_float((uint32_t)got[k][1]);
      const float f = mk > -INFINITY ? ex2_approx((mk - M) * c) : 0.0f;
      const float q = __uint_as_float((uint32_t)got[k][4]) * f;
      others += q;
      S += q + (float)(long long)got[k][0] * 0x1p-40f * f;
    }
    inv_s = 1.0f / S;
    const float of = others * inv_s;
    const bool some_rest = of >= 0x1p-126f;
    float whole = 1.0f, share = 1.0f;  // the shares' sum, what is left of s outside the entries
    if (p.lse) {
      // The shares of a record of all tokens add up to 1 but for its log-sum-exp's rounding, and
      // that of the logits over T before their sum (three half steps of |lse|), and for a float32
      // sum of them (exponents of some 7 units, exponentials, additions, the shares: 68 half steps
      // of 1).  So much is not asked of a row that has nothing to give.
      left = fmaxf((float)((1ll << 40) - mass) * 0x1p-40f, 0.0f);
      if (!some_rest && left < fmaf(fabsf(lse), 0x1p-22f, 0x1p-17f)) left = 0.0f;
      if (!(left > 0.0f)) whole = (float)mass * 0x1p-40f;
      share = some_rest ? whole - left / of : 0.0f;
      if (left > 0.0f && !some_rest) left = INFINITY;  // (the loss asks for no more than that)
    }
    coef = fminf(fmaxf(w * p.inv_t * share * inv_s, -3.0e38f), 3.0e38f);
    inv_s *= whole;
  }

  if (rank == 0 && tid < 32 && p.loss) {
    float L = 0.0f;
    if (w != 0.0f) {
      // The CTAs' sums against the row's maximum, one a lane; then ln S, and ln of s outside
      // the entries and of r, or of what brings the shares' sum to 1.  (Sums of float32 leave
      // 2e-7 of a loss that may be 1e-3.)
      long long S = 0, O = 0, t = 0;
      float large = 0.0f, others = 0.0f;
      if (tid < size) {
        const float mk = __uint_as_float((uint32_t)got[tid][1]);
        const float rest = __uint_as_float((uint32_t)got[tid][4]);
        const float at = (float)(long long)got[tid][0];
        const float at_low = (float)((long long)got[tid][0] - (long long)at);
        const Two f = mk > -INFINITY ? exp_two(over_t(mk, M, p.inv_t, p.inv_t_low)) : Two{0.0f, 0.0f};
        others = f.hi * rest;
        O = fixed_two({others, fmaf(f.hi, rest, -others) + f.lo * rest});
        const float q = f.hi * at;
        S = O + __float2ll_rn(q) + __float2ll_rn(fmaf(f.hi, at, -q) + f.lo * at + f.hi * at_low);
        t = (long long)got[tid][2];
        large = __uint_as_float((uint32_t)(got[tid][4] >> 32));
      }
#pragma unroll
      for (int d = 1; d < kMaxCluster; d <<= 1) {
        S += __shfl_xor_sync(kFull, S, d);
        O += __shfl_xor_sync(kFull, O, d);
        others += __shfl_xor_sync(kFull, others, d);
        t += __shfl_xor_sync(kFull, t, d);
        large += __shfl_xor_sync(kFull, large, d);
      }
      constexpr long long kOne = 1ll << 40;
      const long long r = kOne - mass;
      const long long arg = tid == 0 ? S : tid == 1 ? O : r;
      float v = (float)arg * 0x1p-40f, low = (float)(arg - (long long)(float)arg) * 0x1p-40f;
      if (tid == 1 && O < kOne >> 10) {  // (few units: as float32 has it)
        v = fmaxf(others, 0x1p-126f);
        low = 0.0f;
      } else if (tid == 2 && !p.lse) {
        v = inv_zs;
        low = 0.0f;
      }
      const long long ln = v >= 0x1p-126f ? ln_fixed(v, low) : 0;
      const long long ln1 = __shfl_sync(kFull, ln, 1), ln2 = __shfl_sync(kFull, ln, 2);
      if (tid == 0) {
        const Two a = over_t(M, zmax, p.inv_t, p.inv_t_low);
        long long q = ln;  // M / T + ln S less the teacher's normaliser
        if (p.lse) {
          if (fabsf(a.hi) < 0x1p20f && fabsf(lse) < 0x1p20f && mass < 2 * kOne) {
            q += fixed_two(a) - __float2ll_rn(lse * kTerm);
            t += mul_fixed(mass, q);
          } else {
            large += (float)mass * 0x1p-40f * ((a.hi - lse) + (a.lo + (float)ln * 0x1p-40f));
          }
          if (left > 0.0f) {
            if (left < INFINITY) t += mul_fixed(r, ln2 - ln1 + ln);
            else large = INFINITY;
          }
        } else {
          // (the shares add up to 1 - r, r next to nothing)
          t += mul_fixed(t, r);
          q += ln2 + r;
          if (fabsf(a.hi) < 0x1p20f) t += q + fixed_two(a);
          else large += a.hi + (a.lo + (float)q * 0x1p-40f);
        }
        L = large + (float)t * 0x1p-40f;
      }
    }
    if (tid == 0) {
      p.loss[n] = st ? __int_as_float(0x7fc00000) : none ? 0.0f : L;
      p.row_status[n] = st;
    }
  }
  if (kGrad) {
    const float fill = st ? __int_as_float(0x7fc00000) : 0.0f;
    const bool plain = st != 0 || none;
    const bool like =
        ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    for (int v = tid; v < s.nvec; v += kThreads) {
      float2 x[kN / 2];
      if (plain) {
#pragma unroll
        for (int e = 0; e < kN / 2; ++e) x[e] = both(fill);
      } else {
        widen2<DT>(*reinterpret_cast<const uint4 *>(buf + (size_t)v * 16), x);
#pragma unroll
        for (int e = 0; e < kN / 2; ++e) x[e] = __fmul2_rn(both(coef), exp2_pair(x[e], M, c));
      }
      const uint4 y = narrow2<DT>(x);
      if (like)
        store_like<DT>(s, out, v, y);
      else
        *reinterpret_cast<uint4 *>(buf + (size_t)v * 16) = y;
    }
    __syncthreads();
    if (!plain) {
      const float k = w * p.inv_t;
      for (int j = tid; j < sm.entries; j += kThreads) {
        const float y = k * (ex2_approx((at_x[j] - M) * c) * inv_s - at_p[j]);
        put_elem<DT>(like ? out + (ptrdiff_t)(s.first + pos[j]) * es : buf + (size_t)pos[j] * es, y);
      }
    }
    if (!like) {
      __syncthreads();
      store_unlike<DT, kThreads>(s, buf, out);
    }
  }
  if (w != 0.0f && sm.in.gave_up && tid == 0) share_drain(sm.in);
}

template <int DT, bool kGrad>
cudaError_t launch_dt(const DistillParams &p, cudaStream_t stream) {
  static DeviceOnce once;
  const cudaError_t err = cluster_opt_in_once(once, distill_kernel<DT, kGrad>, 227 * 1024);
  if (err != cudaSuccess) return err;
  constexpr int es = Elem<DT>::kBytes;
  const long long rows = (long long)p.B * p.R;
  const int size = cluster_for(rows, p.V, es, 68 * 1024, 3);
  const int vectors = share_vectors(p.V, es, size);
  return launch_clusters(distill_kernel<DT, kGrad>, rows, size, kThreads,
                         layout_of(vectors, es, p.K).total, stream, p, vectors);
}

}  // namespace

cudaError_t launch_distill(const DistillParams &p, cudaStream_t stream) {
  if (p.dtype == SPECDEC_F32)
    return p.grad ? launch_dt<SPECDEC_F32, true>(p, stream) : launch_dt<SPECDEC_F32, false>(p, stream);
  return p.grad ? launch_dt<SPECDEC_BF16, true>(p, stream) : launch_dt<SPECDEC_BF16, false>(p, stream);
}

}  // namespace specdec
