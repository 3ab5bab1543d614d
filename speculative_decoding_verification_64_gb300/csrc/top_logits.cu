// The K largest logits of every row, largest first (equal ones by index), and the row's
// log-sum-exp (specdec_top_logits): what a verify step leaves of its target to train a
// draft with.
//
// First kernel, one pass over HBM, structured like the row statistics: a CTA an SM, 16 KB
// bulk copies into a ring, a warp reduces an 8 KB stage held in registers.  Beside the
// stage's maximum and sum it leaves the maximum of every 512 bytes (one vector of each lane):
// groups of 128 or 256 tokens.
//
// Second kernel, a CTA a row: the K-th largest of the groups' maxima (its top 16 bits) bounds
// the K-th largest logit from below, since K groups hold one at least that large; only
// groups whose maximum reaches the bound are read again (K of some hundred), and their
// few elements that reach it, K and some, are sorted in shared memory.  Where they are too
// many for the list (long runs of equal logits), a radix selection over (value, index)
// finds the K-th place first.
//
// The scan is bound by HBM, the pick by its chain of loads, one row after another in a CTA.
// 2304 rows of 128256 bfloat16, 64 entries: 132 us for both, 66 % of the measured copy rate
// over the whole call.
// 384 rows of 32003 19 us, 5 rows of 32000 float32 11 us (two launches and the chain).  For
// the 2304 rows, in the place of 159 at that time: a warp a row in the pick 212, its loads
// eight ahead in place of four 187, 512 threads 234.
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

constexpr int kGroups = kTopGroups;
static_assert(kGroups == kVecPerLane, "a group is one vector of each lane");

// Integers that order like the values (their own inverse), -0 just below +0.
__device__ __forceinline__ int signed_key(float x) {
  const int b = __float_as_int(x);
  return b ^ (b >> 31 & 0x7FFFFFFF);
}
__device__ __forceinline__ float signed_float(int k) {
  return __int_as_float(k ^ (k >> 31 & 0x7FFFFFFF));
}

// The maxima over a warp of each of a stage's groups (the row's edge elements are in the first
// group of stage 0): the lane's `group` is that of group `of`, where that is one.  Returns the
// maximum of all.  A NaN comes out as the positive one, whose key is the largest.
template <int DT>
__device__ __forceinline__ float group_maxima(const LaneData<DT> &d, int lane, float &group, int &of) {
  if (DT == SPECDEC_F32) {
    int mine = signed_key(-INFINITY), all = mine;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      float f = max_of<DT>(vector_max<DT>(d.v[k], no_max<DT>()));
      if (k == 0) f = fmax_nan(f, d.edge);
      const int m = __reduce_max_sync(kFull, signed_key(f));
      if (lane == k) mine = m;
      all = max(all, m);
    }
    group = signed_float(mine);
    of = lane;
    return signed_float(all);
  }
  // bfloat16: groups k and k + 8 in one word; each step halves a lane's words and joins two
  // lanes' (16 integer maxima over the warp in their place: 20 us for
  // 384 rows of 32003, 19 with this)
  auto max2 = [](uint32_t a, uint32_t b) {
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return a;
  };
  uint32_t w[kGroups / 2];
#pragma unroll
  for (int k = 0; k < kGroups / 2; ++k) {
    const uint32_t edge = 0xFF800000u | __float_as_uint(d.edge) >> 16;
    const uint32_t a = vector_max<DT>(d.v[k], k == 0 ? edge : no_max<DT>());
    const uint32_t b = vector_max<DT>(d.v[k + kGroups / 2], no_max<DT>());
    w[k] = max2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
  }
#pragma unroll
  for (int half = kGroups / 4; half >= 1; half /= 2) {
    const bool upper = lane & (4 * half);
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const uint32_t keep = upper ? w[i + half] : w[i], send = upper ? w[i] : w[i + half];
      w[i] = max2(keep, __shfl_xor_sync(kFull, send, 4 * half));
    }
  }
  uint32_t m = max2(w[0], __shfl_xor_sync(kFull, w[0], 2));
  m = max2(m, __shfl_xor_sync(kFull, m, 1));
  group = lane & 1 ? bf16_hi(m) : bf16_lo(m);
  of = lane & 2 ? kGroups : (lane >> 2) + (lane & 1) * (kGroups / 2);
  return signed_float(__reduce_max_sync(kFull, signed_key(max_of<DT>(m))));
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
  // The CTA's stages in turn among its warps: stage t of unit i, kConsumerWarps further each
  // time.  (Quotients by additions: four divisions of 64 bits were 300 of a stage's 1000
  // instructions.)
  constexpr int kWhole = kConsumerWarps / kUnit, kPart = kConsumerWarps % kUnit;
  static_assert(kWhole < kSlots, "a warp's next stage is in the ring's next round at most");
  UnitCursor cur, unit;
  cur.init(first + warp / kUnit * stride, kWhole * stride, upr);
  unit.init(0, stride, upr);
  int next = warp % kUnit;
  uint32_t slot_next = warp / kUnit, use_next = 0;
  for (long long i = warp / kUnit; i < n_local;) {
    const int t = next, row = cur.row;
    const uint8_t *at = row_at(row);
    const UnitGeom u = geometry(at, p.V, p.spr, cur.ju, es);
    const uint32_t slot = slot_next, use = use_next;
    i += kWhole;
    slot_next += kWhole;
    next += kPart;
    cur.advance(upr);
    if (next >= kUnit) {
      next -= kUnit;
      ++i;
      ++slot_next;
      cur.row += unit.drow;
      cur.ju += unit.dj;
      if (cur.ju >= upr) {
        cur.ju -= upr;
        ++cur.row;
      }
    }
    if (slot_next >= kSlots) {
      slot_next -= kSlots;
      ++use_next;
    }
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
    float wm = -INFINITY, sum = kGaveUp, group = -INFINITY;
    int of = lane;  // the group whose maximum this lane has
    if (ok) {
      wm = group_maxima<DT>(d, lane, group, of);
      sum = wm > -INFINITY ? warp_sum(lane_sum<DT>(d, c, wm)) : 0.0f;
    }
    const long long at_part = (long long)row * p.spr + u.j0 + t;
    if (lane == 0) p.part[at_part] = make_float2(wm, sum);
    if (of < kGroups) p.group[at_part * kGroups + of] = group;
  }
  if (sm.abort_flag && lane == 0) {
    const unsigned long long t0 = global_timer_ns();
    while (sm.issued < 0 && global_timer_ns() - t0 < kWaitLimitNs) {
    }
    if (sm.issued >= 0) drain_ring(sm.full, kSlots, sm.issued);
  }
}

// ---------------------------------------------------------------------------------------

// Threads of a row's CTA: 256, or 128 for more rows than the SMs hold CTAs of 256 of
// (2304 rows of 128256 tokens, 64 entries: 146 us in both kernels against 159 with 256;
// 384 rows of 32003: 30.7 us against 24.6; both before the vectors were noted, which gave 135
// and 20).  The smaller ones get 64 registers, eight to an SM: 135 us, with 72 registers and
// seven 141, with 48 and ten 141, with 40 and twelve 154; the larger ones 80 registers and
// three to an SM: 20 us for the 384 rows, with 94 and two 25, with 64 and four 21.
constexpr int kFewThreads = 128, kManyThreads = 256;
constexpr int kFewFrom = 8;   // CTAs an SM from which a row gets the fewer
constexpr int kKeys = 2048;   // maxima that the bound is found among
// Tokens that reach it and can be sorted.  Of G maxima the K-th largest lets some -G ln(1 - K / G)
// tokens through: more than this from K = 800 for G = 2048, where seven passes of the radix
// selection follow (2304 rows of 128256 bfloat16, K = 64, 256, 500, 640, 800 and 1000: 133, 207,
// 412, 453, 943 and 1268 us).
constexpr int kList = 1024;
constexpr int kBatch = 1024;  // groups looked at together
// Vectors of a row, an entry, below which they name the bound, in place of groups of 32 (2000
// rows of 17000 tokens, 64 entries: 55 us against 66; of 20000: 61 against 53)
constexpr int kFineBelow = 36;
constexpr int kAhead = 4;     // loads of a thread under way together
constexpr int kVecs = 256;    // vectors with such tokens that a warp notes
constexpr int kDigit = 10;    // bits of a digit of the radix selection

template <int kPickThreads>
struct PickSmem {
  union {
    uint16_t key[kKeys];
    uint32_t count[1 << kDigit];
  } u;
  unsigned long long list[kList];
  uint16_t hit[kBatch];
  uint16_t vec[kPickThreads / 32][kVecs];
  float red[2][kPickThreads / 32];
  int n, hits, digit, need;
};

// What is done with the elements that reach the bound: they go on the list (those whose
// place is at or above `prefix`), or one digit of the places that share the prefix's bits
// from `above` up is counted.
struct Take {
  float from;
  unsigned long long prefix;
  int above, lo;  // above = 0: the list
};

// Every element of the groups whose maximum reaches take.from, and the row's edges, that
// reaches it too.  The groups of a batch are named first, then their vectors are loaded,
// several a thread on their way together, and those with such an element noted; a warp
// looks at the noted ones' elements together (one vector of 25 holds one: looked at as they came,
// nearly every step of a warp went through that).
template <int DT, int kPickThreads>
__device__ __noinline__ void candidates(const uint8_t *row, int V, int spr, const float *group,
                                        Take take, PickSmem<kPickThreads> &sm) {
  constexpr int es = Elem<DT>::kBytes, kN = Elem<DT>::kN;
  const int t = threadIdx.x, lane = t & 31;
  const unsigned below = (1u << lane) - 1;
  uint16_t *vec = sm.vec[t >> 5];
  const UnitGeom g0 = geometry(row, V, spr, 0, es);
  const int tail_begin = min(g0.tail_begin, V);        // (past it for rows that end before a boundary)
  const int inside = (tail_begin - g0.head_end) / kN;  // vectors of the row's inside
  const uint4 *base = reinterpret_cast<const uint4 *>(row + (size_t)g0.head_end * es);
  const int groups = spr * kGroups;
  auto found = [&](float x, int at) {
    const unsigned long long q = place_of(x, at);
    if (take.above == 0) {
      if (q < take.prefix) return;
      const int i = atomicAdd(&sm.n, 1);  // (sorted later: their order decides nothing)
      if (i < kList) sm.list[i] = q;
    } else if (take.above == 64 || q >> take.above == take.prefix >> take.above) {
      atomicAdd(&sm.u.count[(q >> take.lo) & ((1u << (take.above - take.lo)) - 1)], 1u);
    }
  };
#pragma unroll 1
  for (int g = 0; g < groups; g += kBatch) {
    __syncthreads();  // (the last batch's readers)
    if (t == 0) sm.hits = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kBatch / kPickThreads; ++i) {
      const int at = g + i * kPickThreads + t;
      const bool hit = at < groups && __ldg(group + at) >= take.from;
      const unsigned all = __ballot_sync(kFull, hit);
      int base_hit = 0;
      if (all && lane == 0) base_hit = atomicAdd(&sm.hits, __popc(all));
      base_hit = __shfl_sync(kFull, base_hit, 0);
      if (hit) sm.hit[base_hit + __popc(all & below)] = (uint16_t)(i * kPickThreads + t);
    }
    __syncthreads();
    const int n = sm.hits * 32;  // vectors: 32 a group
    int noted = 0;
#pragma unroll 1
    for (int i0 = t; i0 - lane < n; i0 += kAhead * kPickThreads) {
      uint4 w[kAhead];
      int v[kAhead];  // of the batch
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int q = i0 + i * kPickThreads;
        v[i] = q < n ? sm.hit[q >> 5] * 32 + (q & 31) : inside;
        if (v[i] < inside - 32 * g) w[i] = __ldg(base + 32 * g + v[i]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const bool some = v[i] < inside - 32 * g &&
                          max_of<DT>(vector_max<DT>(w[i], no_max<DT>())) >= take.from;
        const unsigned all = __ballot_sync(kFull, some);
        if (some) vec[noted + __popc(all & below)] = (uint16_t)v[i];
        noted += __popc(all);
      }
      // the noted ones, before there are too many or no more come
      if (noted <= kVecs - 32 * kAhead && i0 - lane + kAhead * kPickThreads < n) continue;
      __syncwarp();
#pragma unroll 1
      for (int k = lane; k < noted; k += 32) {
        const int at = 32 * g + vec[k];
        float x[kN];
        widen<DT>(__ldg(base + at), x);
        unsigned reach = 0;
#pragma unroll
        for (int e = 0; e < kN; ++e) reach |= x[e] >= take.from ? 1u << e : 0u;
        while (reach) {
          const int e = __ffs(reach) - 1;
          reach &= reach - 1;
          float y = x[0];
#pragma unroll
          for (int q = 1; q < kN; ++q) y = e == q ? x[q] : y;
          found(y, g0.head_end + at * kN + e);
        }
      }
      noted = 0;
      __syncwarp();
    }
  }
  const int n_head = g0.head_end, n_edge = n_head + V - tail_begin;
  if (t < n_edge) {
    const int e = t < n_head ? t : tail_begin + (t - n_head);
    const float x = load_elem(row, DT, e);
    if (x >= take.from) found(x, e);
  }
  __syncthreads();
}

template <int DT, int kPickThreads>
__global__ void __launch_bounds__(kPickThreads, kPickThreads == kFewThreads ? 8 : 3)
    top_pick_kernel(const TopParams p) {
  __shared__ PickSmem<kPickThreads> sm;
  static_assert(kStageBytes == 16 * 32 * 16, "16 vectors a lane");
  constexpr int kPickWarps = kPickThreads / 32;
  constexpr int es = Elem<DT>::kBytes;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long n = blockIdx.x;
  const long long b = n / p.R;
  const uint8_t *row = reinterpret_cast<const uint8_t *>(p.x) +
                       (b * p.x_at.request + (n - b * p.R) * p.x_at.row) * es;
  const float *group = p.group + n * p.spr * kGroups;
  const float2 *part = p.part + n * p.spr;
  const float c = temperature_scale(p.temperature);

  // the groups' maxima, and the row's
  // (where they are few for K, runs of the row's vectors in their place: with 64 entries 4000 rows
  // of 12000 take 113 us, and took 946 when nearly all tokens were candidates)
  const UnitGeom g0 = geometry(row, p.V, p.spr, 0, es);
  const int groups = p.spr * kGroups;
  const int vectors = (min(g0.tail_begin, p.V) - g0.head_end) / Elem<DT>::kN;
  const bool fine = vectors < kFineBelow * p.K;
  const int parts = fine ? vectors : groups, per = max((parts + kKeys - 1) / kKeys, 1);
  const int keys = (parts + per - 1) / per;
  float M = -INFINITY;
  int lost = 0;
  for (int i = tid; i < p.spr; i += kPickThreads) {
    const float2 q = __ldg(part + i);
    M = fmax_nan(M, q.x);
    lost |= q.y == kGaveUp;
  }
  if (fine) {
    const uint4 *base = reinterpret_cast<const uint4 *>(row + (size_t)g0.head_end * es);
#pragma unroll 4
    for (int i = tid; i < keys; i += kPickThreads) {
      uint32_t m = vector_max<DT>(__ldg(base + i * per), no_max<DT>());
      for (int j = i * per + 1; j < min(vectors, (i + 1) * per); ++j)
        m = vector_max<DT>(__ldg(base + j), m);
      sm.u.key[i] = (uint16_t)(order_key(max_of<DT>(m)) >> 16);
    }
  }
#pragma unroll 4
  for (int i = fine ? keys : tid; i < keys; i += kPickThreads) {
    float m = __ldg(group + i * per);
    for (int j = i * per + 1; j < min(groups, (i + 1) * per); ++j) m = fmaxf(m, __ldg(group + j));
    sm.u.key[i] = (uint16_t)(order_key(m) >> 16);
  }
  if (tid == 0) {
    sm.n = 0;
    if (keys & 1) sm.u.key[keys < kKeys ? keys : 0] = 0;  // (keys are read in pairs; 0 is no key)
  }
  M = cta_max_nan<kPickWarps>(M, sm.red[0]);
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

  // a bound that K groups reach: the top 16 bits of the K-th largest maximum, bit by bit, by
  // one warp (a barrier of the CTA for every bit takes eight times as long)
  if (warp == 0) {
    constexpr int kHeld = 8;  // pairs of keys that a lane holds
    const uint32_t *pairs = reinterpret_cast<const uint32_t *>(sm.u.key);
    const int n_pairs = (keys + 1) / 2;
    uint32_t held[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) held[i] = lane + 32 * i < n_pairs ? pairs[lane + 32 * i] : 0;
    const uint32_t most = order_key(M) >> 16;
    uint32_t bound = 0;
#pragma unroll 1
    for (int bit = 15; bit >= 0; --bit) {
      const uint32_t t = bound | 1u << bit;
      if (t > most) continue;
      unsigned part[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kHeld; ++i) part[i & 3] += ((held[i] & 0xFFFFu) >= t) + ((held[i] >> 16) >= t);
      unsigned m = (part[0] + part[1]) + (part[2] + part[3]);
      for (int i = lane + 32 * kHeld; i < n_pairs; i += 32)
        m += ((pairs[i] & 0xFFFFu) >= t) + ((pairs[i] >> 16) >= t);
      if (__reduce_add_sync(kFull, m) >= (unsigned)p.K) bound = t;
    }
    if (lane == 0) sm.digit = (int)bound;
  }
  __syncthreads();
  const uint32_t bound = (uint32_t)sm.digit;
  // (no bound above -infinity's key: fewer than K groups hold more, and every element counts)
  const float from = bound << 16 >= kLeastKey ? key_float(bound << 16) : -INFINITY;

  candidates<DT, kPickThreads>(row, p.V, p.spr, group, {from, 0ull, 0, 0}, sm);
  // the sum, while the list is completed
  float S = 0.0f;
  for (int i = tid; i < p.spr; i += kPickThreads) {
    const float2 q = __ldg(part + i);
    if (q.x > -INFINITY) S += q.y * ex2_approx((q.x - M) * c);
  }
  S = cta_sum<kPickWarps>(S, sm.red[1]);
  if (sm.n > kList) {
    // radix selection of the K-th place, a digit at a time
    unsigned long long prefix = 0;
    int need = p.K;
#pragma unroll 1
    for (int above = 64; above > 0;) {
      const int lo = max(above - kDigit, 0);
      __syncthreads();
      for (int i = tid; i < 1 << kDigit; i += kPickThreads) sm.u.count[i] = 0;
      candidates<DT, kPickThreads>(row, p.V, p.spr, group, {from, prefix, above, lo}, sm);
      if (warp == 0) {
        // 32 digits a lane, from the largest down, then the one's own
        constexpr int kLane = (1 << kDigit) / 32;
        const int top = (1 << kDigit) - 1 - lane * kLane;
        int mine = 0;
        for (int i = 0; i < kLane; ++i) mine += (int)sm.u.count[top - i];
        int inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(kFull, inc, d);
          if (lane >= d) inc += y;
        }
        if (inc - mine < need && need <= inc) {
          int left = need - (inc - mine), d = top;
          while (left > (int)sm.u.count[d]) left -= (int)sm.u.count[d--];
          sm.digit = d;
          sm.need = left;
        }
        if (lane == 0) sm.n = 0;
      }
      __syncthreads();
      prefix |= (unsigned long long)sm.digit << lo;
      need = sm.need;
      above = lo;
    }
    candidates<DT, kPickThreads>(row, p.V, p.spr, group, {from, prefix, 0, 0}, sm);  // (K of them)
  }
  sort_down<kPickThreads>(sm.list, sm.n);
  for (int i = tid; i < p.K; i += kPickThreads) {
    const unsigned long long q = sm.list[i];
    p.values[n * p.K + i] = place_value(q);
    p.ids[n * p.K + i] = place_index(q);
  }
  if (tid == 0) {
    p.lse[n] = log_sum(M, p.inv_t, p.inv_t_low, S);
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
  if (rows > (long long)kFewFrom * device_sm_count())
    return launch_pdl(top_pick_kernel<DT, kFewThreads>, dim3((unsigned)rows), dim3(kFewThreads), 0,
                      stream, p);
  return launch_pdl(top_pick_kernel<DT, kManyThreads>, dim3((unsigned)rows), dim3(kManyThreads), 0,
                    stream, p);
}

}  // namespace

cudaError_t launch_top_logits(const TopParams &p, cudaStream_t stream) {
  return p.dtype == SPECDEC_F32 ? launch_dt<SPECDEC_F32>(p, stream) : launch_dt<SPECDEC_BF16>(p, stream);
}

}  // namespace specdec
