// The K largest logits of every row, largest first (equal ones by index), and the row's
// log-sum-exp (specdec_top_logits): what a verify step leaves of its target to train a
// draft with.
//
// First kernel, one pass over HBM, structured like the row statistics: a CTA an SM, 16 KB
// bulk copies into a ring, a warp reduces an 8 KB stage held in registers.  Beside the
// stage's maximum and sum it leaves the maximum of each lane's elements (16 vectors, 512
// bytes apart): groups of 64 or 128 tokens.
//
// Second kernel, a CTA a row: the K-th largest of the groups' maxima (its top 16 bits) bounds
// the K-th largest logit from below, since K groups hold one at least that large; only
// groups whose maximum reaches the bound are read again (K of some thousand), and their
// few elements that reach it, K and some, are sorted in shared memory.  Where they are too
// many for the list (long runs of equal logits), a radix selection over (value, index)
// finds the K-th place first.
#include "draft_common.cuh"
#include "stats_stage.cuh"

namespace specdec {
namespace {

using namespace stage;

struct ScanSmem {
  alignas(128) uint8_t stage[kSlots][kUnitBytes];
  alignas(8) uint64_t full[kSlots];
  alignas(8) uint64_t empty[kSlots];
  volatile long long issued;
  volatile int abort_flag;
};

// unit_geometry of a row that stands anywhere
__device__ __forceinline__ UnitGeom geometry(const uint8_t *row, int V, int spr, int ju, int es) {
  return unit_geometry(row, V, spr, 0, ju, es);
}

constexpr float kGaveUp = -2.0f;  // a stage's sum, where its copy was not waited for

template <int DT>
__global__ void __launch_bounds__(kThreads, 1) top_scan_kernel(const TopParams p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  ScanSmem &sm = *reinterpret_cast<ScanSmem *>(smem_raw);
  constexpr int es = Elem<DT>::kBytes;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int upr = (p.spr + kUnit - 1) / kUnit;
  const long long first = blockIdx.x, stride = gridDim.x;
  const long long units = (long long)p.B * p.R * upr;
  const long long n_local = units > first ? (units - first + stride - 1) / stride : 0;
  auto row_at = [&](int row) {
    const int b = row / p.R, r = row - b * p.R;
    return reinterpret_cast<const uint8_t *>(p.x) +
           ((long long)b * p.x_at.request + r * p.x_at.row) * es;
  };
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kUnit);
    }
    sm.abort_flag = 0;
    sm.issued = -1;
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == kConsumerWarps) {
    if (lane == 0) {
      UnitCursor cur;
      cur.init(first, stride, upr);
      uint32_t slot = 0, use = 0;
      long long i = 0;
      for (; i < n_local; ++i) {
        if (use > 0 && !mbar_wait_bounded(&sm.empty[slot], (use - 1) & 1)) {
          sm.abort_flag = 1;
          break;
        }
        if (sm.abort_flag) break;
        const UnitGeom g = geometry(row_at(cur.row), p.V, p.spr, cur.ju, es);
        cur.advance(upr);
        if (g.bytes > 0) {
          mbar_arrive_expect_tx(&sm.full[slot], (uint32_t)g.bytes);
          bulk_copy_g2s(sm.stage[slot], g.src, (uint32_t)g.bytes, &sm.full[slot]);
        } else {
          mbar_arrive(&sm.full[slot]);
        }
        if (++slot == kSlots) {
          slot = 0;
          ++use;
        }
      }
      sm.issued = i;
      if (sm.abort_flag) drain_ring(sm.full, kSlots, i);
    }
    return;
  }

  const float c = temperature_scale(p.temperature);
  for (long long q = warp; q < n_local * kUnit; q += kConsumerWarps) {
    const long long i = q / kUnit;
    const int t = (int)(q - i * kUnit);
    const long long g = first + i * stride;
    const int row = (int)(g / upr);
    const uint8_t *at = row_at(row);
    const UnitGeom u = geometry(at, p.V, p.spr, (int)(g - (long long)row * upr), es);
    const uint32_t slot = (uint32_t)(i % kSlots), use = (uint32_t)(i / kSlots);
    const bool real = t < u.nst;
    LaneData<DT> d;
    d.edge = -INFINITY;
    d.edge_idx = 0x7FFFFFFF;
    if (real && u.j0 + t == 0) {
      const int n_head = u.head_end, n_tail = p.V - u.tail_begin;
      int e = -1;
      if (lane < n_head) e = lane;
      else if (lane < n_head + n_tail) e = u.tail_begin + (lane - n_head);
      if (e >= 0) d.edge = load_elem(at, DT, e);
    }
    // (the slot's previous use first: a parity tells two phases apart only)
    const bool ok =
        __all_sync(kFull, !sm.abort_flag &&
                              (use == 0 || mbar_wait_bounded(&sm.empty[slot], (use - 1) & 1,
                                                             kConsumerWaitNs)) &&
                              mbar_wait_bounded(&sm.full[slot], use & 1, kConsumerWaitNs));
    if (!ok) sm.abort_flag = 1;
    const int sbytes = max(0, min(kStageBytes, u.bytes - t * kStageBytes));
    if (ok && real) load_lane<DT>(d, sm.stage[slot] + t * kStageBytes, sbytes / 16, lane);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.empty[slot]);
    if (!real) continue;
    float lm = -INFINITY, wm = -INFINITY, sum = kGaveUp;
    if (ok) {
      lm = lane_max<DT>(d);  // (with the row's edge elements, in stage 0)
      wm = warp_max_nan(lm);
      sum = wm > -INFINITY ? warp_sum(lane_sum<DT>(d, c, wm)) : 0.0f;
    }
    const long long at_part = (long long)row * p.spr + u.j0 + t;
    if (lane == 0) p.part[at_part] = make_float2(wm, sum);
    p.group[at_part * 32 + lane] = lm;
  }
  if (sm.abort_flag && lane == 0) {
    const unsigned long long t0 = global_timer_ns();
    while (sm.issued < 0 && global_timer_ns() - t0 < kWaitLimitNs) {
    }
    if (sm.issued >= 0) drain_ring(sm.full, kSlots, sm.issued);
  }
}

// ---------------------------------------------------------------------------------------

constexpr int kPickThreads = 256;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kKeys = 4096;  // maxima that the bound is found among
constexpr int kList = 2048;  // tokens that reach it and can be sorted
constexpr int kDigit = 11;   // bits of a digit of the radix selection

struct PickSmem {
  union {
    uint32_t key[kKeys];
    uint32_t count[1 << kDigit];
  } u;
  unsigned long long list[kList];
  float red[kPickWarps];
  float redf[kPickWarps];
  unsigned int total[16];
  int n, digit, need;
};

// Every element of the groups whose maximum reaches `from`, and the row's edges, that
// reaches it too: f(x, index).  Two groups a warp at a time, a lane a vector of each.
template <int DT, typename F>
__device__ __forceinline__ void candidates(const TopParams &p, const uint8_t *row,
                                           const float *group, float from, F &&f) {
  constexpr int es = Elem<DT>::kBytes, kN = Elem<DT>::kN;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const UnitGeom g0 = geometry(row, p.V, p.spr, 0, es);
  const int tail_begin = min(g0.tail_begin, p.V);   // (past it for rows that end before a boundary)
  const int inside = (tail_begin - g0.head_end) / kN;  // vectors of the row's inside
  const uint4 *base = reinterpret_cast<const uint4 *>(row + (size_t)g0.head_end * es);
  for (int st = warp; st < p.spr; st += kPickWarps) {
    unsigned hit = __ballot_sync(kFull, __ldg(group + st * 32 + lane) >= from);
    while (hit) {
      const int a = __ffs(hit) - 1;
      hit &= hit - 1;
      const int b = hit ? __ffs(hit) - 1 : -1;
      hit = hit ? hit & (hit - 1) : 0;
      const int mine = lane < 16 ? a : b;
      const int v = st * (kStageBytes / 16) + mine + 32 * (lane & 15);
      if (mine >= 0 && v < inside) {
        float x[kN];
        widen<DT>(__ldg(base + v), x);
#pragma unroll
        for (int e = 0; e < kN; ++e)
          if (x[e] >= from) f(x[e], g0.head_end + v * kN + e);
      }
    }
  }
  const int n_head = g0.head_end, n_edge = n_head + p.V - tail_begin;
  if ((int)threadIdx.x < n_edge) {
    const int e = (int)threadIdx.x < n_head ? (int)threadIdx.x
                                            : tail_begin + ((int)threadIdx.x - n_head);
    const float x = load_elem(row, DT, e);
    if (x >= from) f(x, e);
  }
}

template <int DT>
__global__ void __launch_bounds__(kPickThreads) top_pick_kernel(const TopParams p) {
  __shared__ PickSmem sm;
  static_assert(kStageBytes == 16 * 32 * 16, "16 vectors a lane");
  constexpr int es = Elem<DT>::kBytes;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  const long long n = blockIdx.x;
  const long long b = n / p.R;
  const uint8_t *row = reinterpret_cast<const uint8_t *>(p.x) +
                       (b * p.x_at.request + (n - b * p.R) * p.x_at.row) * es;
  const float *group = p.group + n * p.spr * 32;
  const float2 *part = p.part + n * p.spr;
  const float c = temperature_scale(p.temperature);

  // maximum, sum, and whether the row can be used
  float M = -INFINITY;
  int lost = 0;
  for (int i = tid; i < p.spr; i += kPickThreads) {
    const float2 q = __ldg(part + i);
    M = fmax_nan(M, q.x);
    lost |= q.y == kGaveUp;
  }
  M = cta_max_nan<kPickWarps>(M, sm.redf);
  int st = __syncthreads_or(lost) ? SPECDEC_ROW_INTERNAL : 0;
  if (!st && !(M > -INFINITY && M <= kMaxLogit)) st = SPECDEC_ROW_NONFINITE;
  if (st) {
    for (int i = tid; i < p.K; i += kPickThreads) {
      p.values[n * p.K + i] = __int_as_float(0x7fc00000);
      p.ids[n * p.K + i] = -1;
    }
    if (tid == 0) {
      p.lse[n] = __int_as_float(0x7fc00000);
      p.row_status[n] = st;
    }
    return;
  }
  float S = 0.0f;
  for (int i = tid; i < p.spr; i += kPickThreads) {
    const float2 q = __ldg(part + i);
    if (q.x > -INFINITY) S += q.y * ex2_approx((q.x - M) * c);
  }
  S = cta_sum<kPickWarps>(S, sm.red);

  // a bound that K groups reach: bit by bit, the top 16 bits of the K-th largest maximum
  const int groups = p.spr * 32, per = (groups + kKeys - 1) / kKeys;
  const int keys = (groups + per - 1) / per;
  for (int i = tid; i < keys; i += kPickThreads) {
    float m = -INFINITY;
    for (int j = i * per; j < min(groups, (i + 1) * per); ++j) m = fmaxf(m, __ldg(group + j));
    sm.u.key[i] = order_key(m) >> 16;
  }
  if (tid < 16) sm.total[tid] = 0;
  if (tid == 0) sm.n = 0;
  __syncthreads();
  uint32_t bound = 0;
  for (int bit = 15; bit >= 0; --bit) {
    const uint32_t t = bound | 1u << bit;
    unsigned m = 0;
    for (int i = tid; i < keys; i += kPickThreads) m += sm.u.key[i] >= t;
    m = __reduce_add_sync(kFull, m);
    if ((tid & 31) == 0 && m) atomicAdd(&sm.total[bit], m);
    __syncthreads();
    if (sm.total[bit] >= (unsigned)p.K) bound = t;
  }
  // (no bound above -infinity's key: fewer than K groups hold more, and every element counts)
  const float from = bound << 16 >= kLeastKey ? key_float(bound << 16) : -INFINITY;

  candidates<DT>(p, row, group, from, [&](float x, int at) {
    const int i = atomicAdd(&sm.n, 1);  // (sorted below: their order decides nothing)
    if (i < kList) sm.list[i] = place_of(x, at);
  });
  __syncthreads();
  if (sm.n > kList) {
    // radix selection of the K-th place, 11 bits at a time
    unsigned long long prefix = 0;
    int need = p.K;
    for (int above = 64; above > 0;) {
      const int lo = max(above - kDigit, 0), width = above - lo;
      __syncthreads();
      for (int i = tid; i < 1 << kDigit; i += kPickThreads) sm.u.count[i] = 0;
      __syncthreads();
      candidates<DT>(p, row, group, from, [&](float x, int at) {
        const unsigned long long q = place_of(x, at);
        if (above == 64 || q >> above == prefix >> above)
          atomicAdd(&sm.u.count[(q >> lo) & ((1u << width) - 1)], 1u);
      });
      __syncthreads();
      if (tid == 0) {
        int d = (1 << width) - 1, left = need;
        while (d > 0 && (unsigned)left > sm.u.count[d]) left -= (int)sm.u.count[d--];
        sm.digit = d;
        sm.need = left;
        sm.n = 0;
      }
      __syncthreads();
      prefix |= (unsigned long long)sm.digit << lo;
      need = sm.need;
      above = lo;
    }
    candidates<DT>(p, row, group, from, [&](float x, int at) {
      const unsigned long long q = place_of(x, at);
      if (q >= prefix) sm.list[atomicAdd(&sm.n, 1)] = q;  // (K of them)
    });
    __syncthreads();
  }
  sort_down<kPickThreads>(sm.list, sm.n);
  for (int i = tid; i < p.K; i += kPickThreads) {
    const unsigned long long q = sm.list[i];
    p.values[n * p.K + i] = place_value(q);
    p.ids[n * p.K + i] = place_index(q);
  }
  if (tid == 0) {
    p.lse[n] = (float)((double)M / (double)p.temperature + log((double)S));
    p.row_status[n] = 0;
  }
}

template <int DT>
cudaError_t launch_dt(const TopParams &p, cudaStream_t stream) {
  static DeviceOnce once;
  const int smem = (int)sizeof(ScanSmem);
  cudaError_t err = smem_opt_in_once(once, top_scan_kernel<DT>, smem);
  if (err != cudaSuccess) return err;
  const long long rows = (long long)p.B * p.R;
  const long long units = rows * ((p.spr + kUnit - 1) / kUnit);
  long long grid = device_sm_count();
  if (grid > units) grid = units;
  err = launch_pdl(top_scan_kernel<DT>, dim3((unsigned)grid), dim3(kThreads), (size_t)smem, stream, p);
  if (err != cudaSuccess) return err;
  return launch_pdl(top_pick_kernel<DT>, dim3((unsigned)rows), dim3(kPickThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_top_logits(const TopParams &p, cudaStream_t stream) {
  return p.dtype == SPECDEC_F32 ? launch_dt<SPECDEC_F32>(p, stream) : launch_dt<SPECDEC_BF16>(p, stream);
}

}  // namespace specdec
