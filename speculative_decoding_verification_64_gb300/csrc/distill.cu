// Divergence of a draft's row from the K entries of a teacher's record, and its gradient
// (specdec_distill).  With s = softmax(x / T) over the row and p_j the teacher's share of
// entry j (token id_j):
//     L = sum_j p_j (ln p_j - ln s_id_j) + r (ln r - ln s_rest)
//     dL/dx_v = (s_v - p_v) / T at an entry's token, (s_v - r s_v / s_rest) / T elsewhere,
// r = 1 - sum p_j and s_rest = the mass of s outside the entries when the teacher's
// log-sum-exp is given; without it p = softmax over the entries and r = 0.
//
// A row is held in shared memory by a cluster of CTAs: it is read from HBM once, whatever
// is computed from it, and the gradient is written once.  While the copies land, the
// teacher's shares are made; then each CTA's maximum, and its sum of exponentials with the
// entries taken out (their logits put to -infinity in shared memory, so that s_rest is a sum
// and no difference of two near equal ones); one exchange of five words between the CTAs;
// the gradient, straight from registers to global memory, then the entries' own values.  The
// loss is sum p_j (z_j - x_j) / T + sum p_j (max / T + ln S - lse), S the row's sum against
// its maximum: its terms are float32, added in 64-bit fixed point (an SM has two lanes for
// 64-bit floating point; with them the kernel took 1790 us in place of 434).
//
// Measured: 4096 rows of 128256 bfloat16, 64 entries, gradient out: 434 us, 4.8 TB/s, 72 % of the
// measured copy rate; 4080 rows of 32003 bfloat16: 101 us, 68 %; 508 rows of 152064 float32: 138 us,
// 66 %; 33 rows of 32000 float32: 8.5 us.  Of a CTA's 23000 clocks (three an SM) its share's
// arrival takes 7600, the sum 3300, the exchange 3000, the loss 2200, the gradient 5000: the
// chain of those steps, which three CTAs overlap in part, is what keeps it from the copy rate.
// Records that complete on an mbarrier, in place of the cluster's barrier: 430 us, and 9.2 us for
// the smallest call.
#include "draft_common.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPerThread = SPECDEC_MAX_TOPK / kThreads;

struct DistillSmem {
  Exchange ex;
  Arrival in;
  long long terms[2][kWarps];
  float red[5][kWarps];
  int status;
  int entries;
};

constexpr float kTerm = 0x1p40f;  // units of the fixed-point sums
constexpr float kMost = 0x1p12f;  // terms that they take (1024 of them); the larger are added
                                  // in float32, where a loss with such a term ends anyway

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
  cluster_arrive();  // all CTAs run before one writes to another (waited for below)
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
  float coef = 0.0f, M = 0.0f, inv_s = 0.0f, S = 0.0f, left = 0.0f, of = 0.0f, zs = 1.0f;
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
    // (1 / T in two parts, so that z / T is rounded once)
    auto y_of = [&](float zj) {
      const float dz = zj - zmax;
      return fmaf(dz, p.inv_t, -lse) + dz * p.inv_t_low;
    };
    if (!p.lse) {
      zs = 0.0f;
#pragma unroll
      for (int i = 0; i < kPerThread; ++i)
        if (z[i] > -INFINITY) zs += expf(y_of(z[i]));
      zs = cta_sum<kWarps>(zs, sm.red[1]);
    }
    const float inv_zs = 1.0f / zs;

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
    float at_s = 0.0f, large = 0.0f;
    long long terms = 0, at_mass = 0;  // sum p_j (z_j - x_j) / T, and of p_j
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      if (id[i] < s.begin || id[i] >= s.end) continue;
      mine = 1;
      const int at = id[i] - s.first;
      if (atomicOr(&bits[at >> 5], 1u << (at & 31)) >> (at & 31) & 1u) {
        status |= SPECDEC_ROW_BAD_TOKEN;  // the same token twice
        continue;
      }
      const float y = z[i] > -INFINITY ? y_of(z[i]) : -INFINITY;
      const float pj = expf(y) * inv_zs;
      const float x = get_elem<DT>(buf + (size_t)at * es);
      put_elem<DT>(buf + (size_t)at * es, -INFINITY);
      at_s += ex2_approx((x - ref) * c);
      if (pj > 0.0f) {
        const float dx = z[i] - x;
        const float t = pj * fmaf(dx, p.inv_t, dx * p.inv_t_low);
        if (fabsf(t) < kMost)
          terms += __float2ll_rn(t * kTerm);
        else
          large += x > -INFINITY ? t : INFINITY;
        at_mass += __float2ll_rn(fminf(pj, kMost) * kTerm);
      }
      const int k = atomicAdd(&sm.entries, 1);  // (their order decides nothing)
      pos[k] = at;
      at_x[k] = x;
      at_p[k] = pj;
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
      sm.red[3][tid >> 5] = at_s;
      sm.red[4][tid >> 5] = large;
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
      rest = at_s = large = 0.0f;
      terms = at_mass = 0;
      for (int k = 0; k < kWarps; ++k) {
        rest += sm.red[0][k];
        at_s += sm.red[3][k];
        large += sm.red[4][k];
        terms += sm.terms[0][k];
        at_mass += sm.terms[1][k];
      }
      const int wrong_here = sm.status | (sm.in.gave_up ? SPECDEC_ROW_INTERNAL : 0);
      rec[0] = (unsigned long long)__float_as_uint(at_s) << 32 | __float_as_uint(rest);
      rec[1] = (unsigned long long)(uint32_t)wrong_here << 32 | __float_as_uint(m);
      rec[2] = (unsigned long long)terms;
      rec[3] = (unsigned long long)at_mass;
      rec[4] = __float_as_uint(large);
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
    float others = 0.0f;
    for (int k = 0; k < size; ++k) {
      const float mk = __uint_as_float((uint32_t)got[k][1]);
      const float f = mk > -INFINITY ? ex2_approx((mk - M) * c) : 0.0f;
      const float q = __uint_as_float((uint32_t)got[k][0]) * f;
      others += q;
      S += q + __uint_as_float((uint32_t)(got[k][0] >> 32)) * f;
    }
    inv_s = 1.0f / S;
    of = others * inv_s;
    float share = 1.0f;  // what is left of s outside the entries
    if (p.lse) {
      // a log-sum-exp in float32 leaves about 2^-21 of the mass unsure: nothing is asked
      // of a row that has nothing to give
      left = fmaxf((float)((1ll << 40) - mass) * 0x1p-40f, 0.0f);
      if (!(of > 0.0f) && left < 0x1p-20f) left = 0.0f;
      share = of > 0.0f ? 1.0f - left / of : 0.0f;
    }
    coef = fminf(fmaxf(w * p.inv_t * share * inv_s, -3.0e38f), 3.0e38f);
  }

  if (rank == 0 && tid == 0 && p.loss) {
    float L = 0.0f;
    if (w != 0.0f) {
      // q = max / T + ln S - lse in units of 2^-40, 2^40 / T and ln S in parts that are rounded
      // far below float32's half step of the whole
      int e;
      const float f = frexpf(S, &e);
      float zt = 0.0f;  // without a log-sum-exp: zmax / T + ln zs is the entries' own
      int ez = 0;
      const float fz = frexpf(zs, &ez);
      if (!p.lse) zt = zmax;
      const float dm = M - zt, a = dm * p.inv_t;
      const float low = fmaf(dm, p.inv_t, -a) + dm * p.inv_t_low;
      long long t = 0;
      for (int k = 0; k < size; ++k) {
        t += (long long)got[k][2];
        L += __uint_as_float((uint32_t)got[k][4]);
      }
      float q;
      if (fabsf(a) < 0x1p21f && fabsf(lse) < 0x1p21f) {
        const long long kLn2 = 762123384786ll;  // ln 2 in units of 2^-40
        const long long qf = __float2ll_rn(a * kTerm) + __float2ll_rn((low + logf(f) - logf(fz)) * kTerm) -
                             __float2ll_rn(lse * kTerm) + (long long)(e - ez) * kLn2;
        q = (float)qf * 0x1p-40f;
        t += qf;
      } else {
        q = (a - lse) + (low + logf(S) - logf(zs));
        L += q;
      }
      // sum p_j is 1 without a log-sum-exp (by definition) and 1 - r with one
      if (p.lse) L -= q * ((float)((1ll << 40) - mass) * 0x1p-40f);
      if (left > 0.0f) L += left * logf(left / of);
      L += (float)t * 0x1p-40f;
    }
    p.loss[n] = st ? __int_as_float(0x7fc00000) : none ? 0.0f : L;
    p.row_status[n] = st;
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
