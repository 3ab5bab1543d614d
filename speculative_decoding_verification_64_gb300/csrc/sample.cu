// Tokens drawn from rows of logits under temperature, top-k, top-p and min-p, and the
// rows' distributions or what the filters leave of their logits (specdec_sample).
//
// With w_v = exp((l_v - max) / T), tokens in the order of their place (larger first, equal
// ones by index): top-k keeps the first k, top-p the shortest run of those whose mass is
// at least p of theirs, min-p those with w >= min_p.  What is kept is a run of places again,
// so that one cut (value, index) says it all.  A draw is the first kept token, by index,
// whose cumulative mass exceeds u times the kept mass.
//
// A row is held in shared memory by a cluster of CTAs and read from HBM once.
//   * With top-k: the k-th largest of the maxima of some hundred groups of tokens (its top 16
//     bits) bounds the k-th logit from below, the few tokens that reach it are gathered by
//     rank 0, sorted, weighed, cut and drawn from.
//   * With top-p alone, bfloat16: the tokens of every value are counted (a row has some
//     thousand values), each value is weighed once, and sums over the values name the one that
//     top-p cuts, and how many of its tokens stay.
//   * Float32, and bfloat16 rows of other magnitudes: a histogram of the logits, 1/64 octave of
//     weight a bin, says about where the cut is.  A pass adds the weights of all places above a
//     bracket around it, and in it; when the cut is inside and the bracket's tokens fit a list,
//     they are sorted and the cut is found among them.  A bracket that missed is placed anew by
//     what the pass found, and where that fails, between the places known to hold the cut, halves
//     of them.
//   * The draws of such rows: the passes leave the kept mass of every run of 32 to 128 vectors;
//     a draw looks its run up, and a warp weighs that run once more.
// Which token is cut last, or drawn, turns on sums over the vocabulary: weights and sums are
// those of draft_weight.cuh, in integers that no order of additions changes.  The cluster's
// CTAs exchange a record of a few words at each step.
//
// What bounds it: the chain of passes over the share and of exchanges, two CTAs an SM, and
// where all tokens are weighed some 23 instructions an element (rows of 128256 bfloat16, a read
// and a write of HBM):
//   2304 flat rows, top-p 0.95 and min-p, logits out: 560 us, 2.1 TB/s of reads and writes.  Of a
//     CTA's 38000 clocks arrival and maximum take 11000, counting 9000, summing the counts 9000,
//     the rows 6000.  By the histogram and exact weights of all tokens: 797.
//   672 rows, no filter, 3 draws and probabilities: 206 us.  Of 41000 clocks arrival and
//     maximum 9000, weights 17000, draws 2700, probabilities 9300.
//   256 rows, top-p 0.9, a draw and probabilities: 122 us (four waves of CTAs, the last a third
//     full; by the histogram 131).  One row of 32000 float32 under top-k 40 and top-p: 14 us, a
//     chain of exchanges and barriers (and of instructions that are not cached yet).
// With 512 threads a CTA 654, 226 and 133 us in their place: 64 registers a thread, some of them
// spilled, and the kernel's code is larger than the instruction cache's near levels, so that more
// warps in different places cost more than they hide.
#include "draft_weight.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Tokens that rank 0 can sort.  Of G groups' maxima the k-th largest lets some -G ln(1 - k / G)
// tokens through: more than this from k = 650 for G = 1024, from 800 for 2048, and a cluster of 3
// has 768 groups, which bound no larger k.  Halving passes follow there (top-k 500, 640, 768, 800 and
// 1000: 64 rows of 102400 bfloat16, three CTAs each, 56, 80, 105, 335 and 568 us; 256 rows of 128256,
// four CTAs, 180, 221, 257, 321 and 796).
constexpr int kList = 1024;
constexpr int kMine = 1024;   // tokens that a CTA can bring
constexpr int kFewK = 128;    // top-k up to which some 500 groups name the bound
constexpr int kKeys = 4096;   // groups' maxima (256 of each of 16 CTAs)
// The histogram's bins of a factor of two in weight, and its 24 octaves: a row's tail below
// 2^-24 of its largest weight is 3 % of the mass at most for 2^19 tokens, and the exact pass
// corrects the guess by what it found.  Float32 rows of 128256 under top-p, of few large tokens
// (256, top-p 0.9), flat (576, 0.95 and min-p at T = 0.7) and flatter (256, 0.9 at T = 1): 218, 378 and
// 1051 us; with 32 bins an octave 206, 351 and 1060, with 128 260, 468 (twice the bins to read
// from the other CTAs) and 382 (the flattest rows' brackets fit the list then, where halving passes
// follow with fewer).  With 16 octaves 320, 358 and 1020: tails' mass is missed, and a second
// bracket placed.
constexpr float kOctave = 64.0f;
constexpr int kBins = 24 * 64;
// A bracket reaches to either side of the place that the histogram names by this share of
// the mass (bins hold their mass to 0.54 %, the sum of many to 0.04 %), or this many tokens
// where that is less (a value of bfloat16 rows holds some 200 of a flat row), or 32 bins.
constexpr float kMargin = 0.0025f;
constexpr int kBudget = 256;
constexpr int kTries = 2;     // brackets placed by the histogram
// Halves of 2^64 places, and the brackets before them: no search is longer, and what would
// be (sums that changed between two passes) ends as SPECDEC_ROW_INTERNAL.
constexpr int kLimit = 80;
constexpr int kAll = 0x7FFFFFFF;
constexpr float kLeast = -3.402823466e38f;

using u64 = unsigned long long;

__device__ const WeightTable g_table = make_table();

// Values of bfloat16 rows that are counted one by one: magnitudes from 2^-14 up to 64, by
// exponent, sign and mantissa (neighbouring values of one sign in different banks).
constexpr int kMags = 20 * 128;
constexpr uint32_t kFirstMag = 0x3880;  // the bits of 2^-14
constexpr float kLeastMag = 0x1p-14f, kMostMag = 64.0f;
// Tokens of a row whose values are counted; shorter ones take the histogram (rows of 12000 that
// draw under top-p: 358 us by counts, 323 by the histogram; of 20000: 267 against 275, of
// 32000 220 against 265).
constexpr int kCountFrom = 16384;

struct SampleSmem {
  Exchange ex;
  Arrival in;
  alignas(8) uint64_t tabled;
  alignas(16) float2 table[kTable];
  union {
    u64 list[kList];
    uint16_t key[kKeys];
    uint32_t bin[kBins + 32];
    alignas(8) uint32_t val[2 * kMags + 32];
  };
  u64 mine[kMine];
  u64 red[2][kWarps];
  u64 sums[kWarps][7];
  float redf[2][kWarps];
  double drop;         // T ln(min_p)
  float piece[64], whole;   // of the histogram's mass
  int bracket_bin, bracket_first, bracket_last;
  float bracket_before;
  unsigned bound;      // of the k-th largest key
  int count[kWarps];
  int listed[kMaxCluster];  // tokens on each CTA's list
  int n_mine, n_kept;
  u64 cut[3];
};

struct Layout {
  int share, steps, total;
};

__host__ __device__ inline Layout layout_of(int vectors) {
  Layout l;
  l.share = ((int)sizeof(SampleSmem) + 127) / 128 * 128;
  l.steps = l.share + vectors * 16;
  l.total = l.steps + (vectors + 31) / 32 * 8;
  return l;
}

// A run of places down to one: x above the value, or equal to it with an index up to the
// bound.
struct Cut {
  float value;
  int index;
  __device__ __forceinline__ bool holds(float x, int at) const {
    return x > value || (x == value && at <= index);
  }
};

// Places >= q; q's lower half is 2^32 - 1 - index.
__device__ __forceinline__ Cut cut_at(u64 q) {
  const uint32_t low = (uint32_t)q;
  Cut c;
  c.value = place_value(q);
  c.index = (int)min(0xFFFFFFFFu - low, (uint32_t)kAll);
  if (q >> 32 == 0x7FFFFFFFu) {  // the key that -0 would have: no token's, but equal to 0
    c.value = 0.0f;
    c.index = kAll;
  }
  return c;
}

__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += shfl_xor_u64(v, d);
  return v;
}

// Inclusive sums over the lanes of a warp.
__device__ __forceinline__ u64 warp_incscan(u64 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const u64 y = shfl_up_u64(v, d);
    if (lane >= d) v += y;
  }
  return v;
}

__device__ __forceinline__ u64 shfl_u64(u64 v, int from) {
  return (u64)__shfl_sync(kFull, (uint32_t)v, from) |
         (u64)__shfl_sync(kFull, (uint32_t)(v >> 32), from) << 32;
}

// Exclusive sums over the CTA's threads in thread order, and the total.
__device__ __forceinline__ u64 cta_exscan(u64 v, u64 *red, u64 &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const u64 inc = warp_incscan(v);
  __syncthreads();
  if (lane == 31) red[warp] = inc;
  __syncthreads();
  u64 pre = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) pre += red[w];
    total += red[w];
  }
  return pre + inc - v;
}

// What a pass over the CTA's share found: mass down to the cut, and of everything; tokens
// down to the cut.
struct Found {
  u64 above, all;
  int n_above;
};

// The vectors of a run: 32 steps of a warp at most, so that a lane's sums fit 32 bits.
__device__ __forceinline__ int run_steps(const Share &s) {
  return s.nvec > 1024 ? 4 : s.nvec > 512 ? 2 : 1;
}

// Sums over a warp of lanes' sums of bits (at most 32 weights each).
__device__ __forceinline__ u64 warp_fixed(uint32_t a, uint32_t b, int n) {
  a -= (uint32_t)n * kBits6;
  const int32_t d = (int32_t)(b - (uint32_t)n * kBitsB);
  const u64 low = __reduce_add_sync(kFull, (uint32_t)d & 0xFFFFu);
  const int high = __reduce_add_sync(kFull, d >> 16);
  return ((u64)__reduce_add_sync(kFull, a) << 21) + low + (u64)((long long)high << 16);
}

// The next float that orders below x (-infinity below the least finite one).
__device__ __forceinline__ float just_below(float x) {
  const uint32_t k = order_key(x) - 1;
  return key_float(k == 0x7FFFFFFFu ? k - 1 : k);  // (past -0, which orders with 0)
}

enum Pass {
  kWhole,   // a cut that takes all tokens of its value
  kBracket  // two cuts of any kind: the tokens between them go on the list
};

// One pass over the share's runs: steps[i] gets run i's mass of the places down to `hi`.
// Sums of each warp.  Tokens of the bounds' values and those between are few where it
// counts, and looked at one by one.
template <int DT, Pass kPass>
__device__ __forceinline__ Found weigh(const Share &s, const uint8_t *buf, const WeightOf &w,
                                       const Cut &hi, const Cut &lo, u64 *steps, SampleSmem &sm) {
  constexpr int kN = Elem<DT>::kN;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = run_steps(s);
  Found f = {0, 0, 0};
  int n_above = 0;
  const float top = hi.index == kAll ? just_below(hi.value) : hi.value;
  const float low = kPass == kBracket ? lo.value : hi.value;
  for (int i = warp; 32 * per * i < s.nvec; i += kWarps) {
    uint32_t a_sum = 0, b_sum = 0, az_sum = 0, bz_sum = 0;
    u64 one_by_one = 0;
    int n = 0, more = 0;
#pragma unroll 1
    for (int q = 0; q < per; ++q) {
      const int v = 32 * (per * i + q) + lane;
      float2 x[kN / 2];
      if (v < s.nvec) {
        widen2<DT>(*reinterpret_cast<const uint4 *>(buf + (size_t)v * 16), x);
      } else {
#pragma unroll
        for (int e = 0; e < kN / 2; ++e) x[e] = both(-INFINITY);
      }
      unsigned near = 0;
#pragma unroll
      for (int e = 0; e < kN / 2; ++e) {
        uint32_t a[2], b[2];
        weight2(x[e], w, sm.table, a, b);
        if (kPass == kBracket) {
          az_sum += a[0] + a[1];
          bz_sum += b[0] + b[1];
        }
        const bool k0 = x[e].x > top, k1 = x[e].y > top;
        if (k0) {
          a_sum += a[0];
          b_sum += b[0];
          ++n;
        }
        if (k1) {
          a_sum += a[1];
          b_sum += b[1];
          ++n;
        }
        if (kPass != kWhole) {
          if (x[e].x >= low && !k0) near |= 1u << (2 * e);
          if (x[e].y >= low && !k1) near |= 2u << (2 * e);
        }
      }
      if (kPass != kWhole) {
        while (near) {
          const int e = __ffs(near) - 1;
          near &= near - 1;
          const float y = get_elem<DT>(buf + (size_t)v * 16 + e * Elem<DT>::kBytes);
          const int at = s.first + v * kN + e;
          if (hi.holds(y, at)) {
            one_by_one += weight_fixed(y, w, sm.table);
            ++more;
          } else if (kPass == kBracket && lo.holds(y, at)) {
            const int k = atomicAdd(&sm.n_mine, 1);  // (sorted later)
            if (k < kMine) sm.mine[k] = place_of(y, at);
          }
        }
      }
    }
    n_above += n + more;
    u64 t = warp_fixed(a_sum, b_sum, n);
    if (kPass != kWhole && __any_sync(kFull, more)) t += warp_sum_u64(one_by_one);
    if (lane == 0) steps[i] = t;
    f.above += t;
    if (kPass == kBracket) f.all += warp_fixed(az_sum, bz_sum, per * kN);
  }
  f.n_above = __reduce_add_sync(kFull, n_above);
  return f;
}

// The same, and the sums of the cluster: `mine` gets this CTA's mass, sm.n_mine of `n_in`
// tokens between the cuts are on its list, and `fits` says that all CTAs' are on theirs.
template <int DT, Pass kPass>
__device__ __forceinline__ Found weigh_row(const Share &s, const uint8_t *buf, const WeightOf &w,
                                           const Cut &hi, const Cut &lo, u64 *steps, int rank,
                                           int size, int &turn, u64 &mine, u64 &before, int &n_in,
                                           bool &fits, SampleSmem &sm) {
  const Found m = weigh<DT, kPass>(s, buf, w, hi, lo, steps, sm);
  const int warp = threadIdx.x >> 5;
  __syncthreads();  // (the sums' last readers)
  if ((threadIdx.x & 31) == 0) {
    sm.red[0][warp] = m.above;
    sm.red[1][warp] = m.all;
    sm.count[warp] = m.n_above;
  }
  __syncthreads();
  u64 rec[kWords] = {0, 0, 0};
#pragma unroll
  for (int q = 0; q < kWarps; ++q) {
    rec[0] += sm.red[0][q];
    rec[1] += sm.red[1][q];
    rec[2] += (u64)sm.count[q] << 32;
  }
  rec[2] |= (uint32_t)sm.n_mine;
  mine = rec[0];
  const u64(*got)[kWords] = exchange(sm.ex, turn, rec, 3, rank, size);
  Found f = {0, 0, 0};
  before = 0;
  n_in = 0;
  fits = true;
#pragma unroll 1
  for (int q = 0; q < size; ++q) {
    if (q < rank) before += got[q][0];
    f.above += got[q][0];
    f.all += got[q][1];
    f.n_above += (int)(got[q][2] >> 32);
    const int here = (int)(uint32_t)got[q][2];
    if (threadIdx.x == 0) sm.listed[q] = here;
    n_in += here;
    fits = fits && here <= kMine;
  }
  fits = fits && n_in <= kList;
  return f;
}

__device__ __forceinline__ void count_bin(uint32_t at) {
  asm volatile("red.shared::cta.add.u32 [%0], 1;" ::"r"(at) : "memory");
}

// A histogram of the CTA's tokens: bin j counts those whose weight is within half a bin of
// 2^(-j / 64).  The lighter ones go to places of their own, one a lane (there most tokens
// of a row of text stand, many of one value).  The bin's number is read off the bits of
// 2^23 + j.  Ends with the cluster's barrier.
template <int DT>
__device__ __forceinline__ void histogram(const Share &s, const uint8_t *buf, float M, float ch,
                                          int size, SampleSmem &sm) {
  constexpr int kN = Elem<DT>::kN;
  for (int i = threadIdx.x; i < kBins; i += kThreads) sm.bin[i] = 0;
  __syncthreads();
  const float2 c = both(-ch * kOctave), one = both(8388608.0f);
  const uint32_t base = smem_addr(sm.bin);
  const uint32_t rest = kBins + (threadIdx.x & 31);
  for (int v = threadIdx.x; v < s.nvec; v += kThreads) {
    float2 x[kN / 2];
    widen2<DT>(*reinterpret_cast<const uint4 *>(buf + (size_t)v * 16), x);
#pragma unroll
    for (int e = 0; e < kN / 2; ++e) {
      const float2 y = __ffma2_rn(__fadd2_rn(x[e], both(-M)), c, one);
      count_bin(base + 4 * min(__float_as_uint(y.x) - 0x4B000000u, rest));
      count_bin(base + 4 * min(__float_as_uint(y.y) - 0x4B000000u, rest));
    }
  }
  __syncthreads();
  cluster_sync(size);
}

// Where the mass of the cluster's histograms reaches `want` in their first bins (of weights
// as they stand there; a share of all of it where `share` is set): the bins of a bracket
// around that place, and the mass before them.  The same in every CTA.
__device__ __forceinline__ void place_bracket(float want, bool share, int size, SampleSmem &sm,
                                              int &first, int &last, float &before) {
  // pairs of bins a thread, those of a warp's threads next to one another
  constexpr int kEach = (kBins / 2 + kThreads - 1) / kThreads;
  static_assert(kBins % 64 == 0, "whole warps of pairs");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t bins = smem_addr(sm.bin);
  // weight of bin j
  auto weight = [](int j) { return ex2_approx((float)j * (-1.0f / kOctave)); };
  u64 n[kEach];  // (counts of a row fit half of a word)
#pragma unroll
  for (int i = 0; i < kEach; ++i) n[i] = 0;
#pragma unroll 2
  for (int q = 0; q < size; ++q) {
    const uint32_t at = cluster_addr(bins, q);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int j = i * kThreads + tid;
      if (j < kBins / 2) n[i] += remote_get_weak(at + 8u * j);
    }
  }
  __syncthreads();  // (the last readers of what follows)
  float inc[kEach];  // mass of the warp's bins up to this thread's
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int j = 2 * (i * kThreads + tid);
    inc[i] = (float)(uint32_t)n[i] * weight(j) + (float)(uint32_t)(n[i] >> 32) * weight(j + 1);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float y = __shfl_up_sync(kFull, inc[i], d);
      if (lane >= d) inc[i] += y;
    }
    if (lane == 31) sm.piece[i * kWarps + warp] = inc[i];
  }
  if (tid == 0) sm.bracket_bin = kBins;
  __syncthreads();
  if (warp == 0) {
    // the pieces' sums, two a lane
    static_assert(kEach * kWarps <= 64, "two pieces a lane");
    const float p0 = 2 * lane < kEach * kWarps ? sm.piece[2 * lane] : 0.0f;
    const float p1 = 2 * lane + 1 < kEach * kWarps ? sm.piece[2 * lane + 1] : 0.0f;
    float sum = p0 + p1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float y = __shfl_up_sync(kFull, sum, d);
      if (lane >= d) sum += y;
    }
    sm.piece[2 * lane] = sum - p1 - p0;
    sm.piece[2 * lane + 1] = sum - p1;
    if (lane == 31) sm.whole = sum;
  }
  __syncthreads();
  const float whole = sm.whole;
  if (share) want *= whole;
  // the first bin whose mass reaches it (rounded sums of neighbours may both, or overlap:
  // the first one, the same in every CTA)
  int at = kBins;
  float b = 0.0f;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int j = 2 * (i * kThreads + tid);
    const float m0 = (float)(uint32_t)n[i] * weight(j), m1 = (float)(uint32_t)(n[i] >> 32) * weight(j + 1);
    const float to = sm.piece[i * kWarps + warp] + inc[i];
    if (at == kBins && m0 + m1 > 0.0f && to >= want) {
      const bool second = m0 == 0.0f || (m1 > 0.0f && to - m1 < want);
      at = second ? j + 1 : j;
      b = second ? to - m1 : to - m1 - m0;
    }
  }
  if (at < kBins) atomicMin(&sm.bracket_bin, at);
  __syncthreads();
  if (at == sm.bracket_bin && at < kBins) sm.bracket_before = b;
  __syncthreads();
  if (warp == 0) {
    at = sm.bracket_bin;
    b = sm.bracket_before;
    if (at == kBins) {  // (beyond what rounded sums reach)
      at = kBins - 1;
      b = whole;
    }
    const int j_up = at - 1 - lane, j_down = at + 1 + lane;
    uint32_t up = 0, down = 0;
#pragma unroll 1
    for (int q = 0; q < size; ++q) {
      const uint32_t from = cluster_addr(bins, q);
      if (j_up >= 0) up += remote_get32(from + 4u * j_up);
      if (j_down < kBins) down += remote_get32(from + 4u * j_down);
    }
    const float m_up = (float)up * weight(j_up);
    float to_up = m_up, to_down = (float)down * weight(j_down);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(kFull, up, d), z = __shfl_up_sync(kFull, down, d);
      const float f = __shfl_up_sync(kFull, to_up, d), g = __shfl_up_sync(kFull, to_down, d);
      if (lane >= d) {
        up += y;
        down += z;
        to_up += f;
        to_down += g;
      }
    }
    // as many bins as stay below both, and the one that passes the margin
    const float margin = kMargin * whole;
    const int n_up = min(min(at, 32), 1 + __popc(__ballot_sync(kFull, up <= kBudget && to_up < margin)));
    const int n_down = min(min(kBins - 1 - at, 32),
                           1 + __popc(__ballot_sync(kFull, down <= kBudget && to_down < margin)));
    float m = lane < n_up ? m_up : 0.0f;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m += __shfl_xor_sync(kFull, m, d);
    if (lane == 0) {
      sm.bracket_before = b - m;
      sm.bracket_first = at - n_up;
      sm.bracket_last = at + n_down;
    }
  }
  __syncthreads();
  before = sm.bracket_before;
  first = sm.bracket_first;
  last = sm.bracket_last;
}

// Counts of the CTA's tokens by value (bfloat16); tokens of other magnitudes are counted in
// places that nobody reads (no branch a token: 556 us for the 2304 rows, with one 648), and those
// that weigh anything go on the list.  Those are looked at one by one, -infinity among them: 576 flat
// rows of 128256 under top-p 0.95 take 228 us, half masked 460, masked but for 1000 tokens 336, and
// rows of nothing but zeros, all of which are noted by one counter before the histogram has its
// turn, 10.9 ms.
__device__ __forceinline__ void count_values(const Share &s, const uint8_t *buf, float least,
                                             SampleSmem &sm) {
  for (int i = threadIdx.x; i < 2 * kMags; i += kThreads) sm.val[i] = 0;
  __syncthreads();
  const uint32_t base = smem_addr(sm.val), rest = 2u * kMags + (threadIdx.x & 31);
#pragma unroll 2
  for (int v = threadIdx.x; v < s.nvec; v += kThreads) {
    const uint4 q = *reinterpret_cast<const uint4 *>(buf + (size_t)v * 16);
    const uint32_t a[4] = {q.x, q.y, q.z, q.w};
    unsigned odd = 0;  // pairs with such a token
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // both halves as exponent, sign, mantissa
      const uint32_t r = ((a[i] << 1) & 0xFF00FF00u) | ((a[i] >> 8) & 0x00800080u) | (a[i] & 0x007F007Fu);
      const uint32_t j0 = (r & 0xFFFFu) - 2 * kFirstMag, j1 = (r >> 16) - 2 * kFirstMag;
      count_bin(base + 4 * min(j0, rest));
      count_bin(base + 4 * min(j1, rest));
      odd |= max(j0, j1) >= 2u * kMags ? 1u << i : 0u;
    }
    while (odd) {
      const int e0 = 2 * (__ffs(odd) - 1);
      odd &= odd - 1;
      for (int e = e0; e < e0 + 2; ++e) {
        const float y = get_elem<SPECDEC_BF16>(buf + (size_t)v * 16 + 2 * e);
        if (!(y >= least) || (fabsf(y) >= kLeastMag && fabsf(y) < kMostMag)) continue;
        const int k = atomicAdd(&sm.n_mine, 1);
        if (k < kMine) sm.mine[k] = place_of(y, s.first + v * 8 + e);
      }
    }
  }
}

// top-p's cut of a bfloat16 row below 64 from counts of its values: a sum over the values in
// place of one over the tokens.  Each CTA adds up the counts of all for its share of the
// magnitudes, weighs them, and one exchange says whose share holds the cut; that CTA finds
// the value and how many of its tokens are kept, and where that is not all, the CTA that
// holds the last of them finds its index.  The least of top-p's and min-p's cut comes out, with the
// kept mass and count.  False, and nothing found, where the cut is among tokens that are not
// counted (near 0, below -64), or too many of those or of one value would have to be listed.
// The same in every CTA.
__device__ __noinline__ bool cut_by_values(const Share &s, const uint8_t *buf, const WeightOf &w,
                                           float M, float top_p, float floor_value, int rank, int size,
                                           int &turn, Cut &cut, u64 &Z, int &kept, SampleSmem &sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  count_values(s, buf, M - 60.0f / w.ch, sm);
  __syncthreads();
  cluster_sync(size);
  const uint32_t vals = smem_addr(sm.val);
  const int per = (kMags + size - 1) / size;
  const int m0 = min(rank * per, kMags), m1 = min(m0 + per, kMags);
  auto place = [&](int m) { return vals + 4u * (uint32_t)(m + (m & ~127)); };  // of +v; -v 128 further
  auto counts = [&](int m) {  // of +v in the lower half, of -v in the upper
    uint32_t p = 0, n = 0;
#pragma unroll 4
    for (int q = 0; q < size; ++q) {
      const uint32_t at = cluster_addr(place(m), q);
      p += remote_get32(at);
      n += remote_get32(at + 512u);
    }
    return (u64)n << 32 | p;
  };
  auto magnitude = [](int m) { return __uint_as_float((kFirstMag + (uint32_t)m) << 16); };

  // mass: of the positive values, the negative ones, tokens near 0, tokens below -64, and of
  // all down to min-p's cut
  u64 mass[5] = {0, 0, 0, 0, 0};
  unsigned n[4] = {0, 0, 0, 0};  // tokens: positive, negative, near 0, down to min-p's cut
#pragma unroll 1
  for (int m = m0 + tid; m < m1; m += kThreads) {
    const u64 c = counts(m);
    if (!c) continue;
    const float v = magnitude(m);
    uint32_t a[2], b[2];
    weight2(make_float2(v, -v), w, sm.table, a, b);
    const uint32_t up = (uint32_t)c, down = (uint32_t)(c >> 32);
    const u64 of_up = up * fixed_sum(a[0], b[0], 1), of_down = down * fixed_sum(a[1], b[1], 1);
    mass[0] += of_up;
    mass[1] += of_down;
    n[0] += up;
    n[1] += down;
    if (v >= floor_value) {
      mass[4] += of_up;
      n[3] += up;
    }
    if (-v >= floor_value) {
      mass[4] += of_down;
      n[3] += down;
    }
  }
#pragma unroll 1
  for (int i = tid; i < min(sm.n_mine, kMine); i += kThreads) {
    const float x = place_value(sm.mine[i]);
    const u64 t = weight_fixed(x, w, sm.table);
    const bool near = fabsf(x) < kLeastMag;
    mass[2] += near ? t : 0;
    mass[3] += near ? 0 : t;
    n[2] += near;
    if (x >= floor_value) {
      mass[4] += t;
      ++n[3];
    }
  }
#pragma unroll
  for (int i = 0; i < 5; ++i) mass[i] = warp_sum_u64(mass[i]);
#pragma unroll
  for (int i = 0; i < 4; ++i) n[i] = __reduce_add_sync(kFull, n[i]);
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < 5; ++i) sm.sums[warp][i] = mass[i];
    sm.sums[warp][5] = (u64)n[0] << 32 | n[1];
    sm.sums[warp][6] = (u64)n[2] << 32 | n[3];
  }
  __syncthreads();
  u64 rec[kWords];
  if (warp == 0) {
#pragma unroll
    for (int i = 0; i < 7; ++i) {
      rec[i] = 0;
#pragma unroll
      for (int q = 0; q < kWarps; ++q) rec[i] += sm.sums[q][i];
    }
    rec[7] = (u64)(uint32_t)sm.n_mine;
  }
  const u64(*got)[kWords] = exchange(sm.ex, turn, rec, 8, rank, size);
  u64 all[5] = {0, 0, 0, 0, 0};
  int n_up = 0, n_near = 0, n_floor = 0;
  bool fits = true;
#pragma unroll 1
  for (int q = 0; q < size; ++q) {
#pragma unroll
    for (int i = 0; i < 5; ++i) all[i] += got[q][i];
    n_up += (int)(got[q][5] >> 32);
    n_near += (int)(got[q][6] >> 32);
    n_floor += (int)(uint32_t)got[q][6];
    fits = fits && got[q][7] <= kMine;
  }
  if (!fits) return false;
  const u64 want = max(share_at_least(top_p, all[0] + all[1] + all[2] + all[3]), 1ull);
  if (want > all[4]) {  // min-p's cut comes first
    cut = {floor_value, kAll};
    Z = all[4];
    kept = n_floor;
    return true;
  }
  const bool up = want <= all[0];
  u64 above = up ? 0 : all[0] + all[2];
  int n_above = up ? 0 : n_up + n_near;
  if (!up && (want <= above || want > above + all[1])) return false;
  int owner = -1;
#pragma unroll 1
  for (int i = 0; i < size; ++i) {
    const int q = up ? size - 1 - i : i;
    const u64 here = got[q][up ? 0 : 1];
    if (want <= above + here) {
      owner = q;
      break;
    }
    above += here;
    n_above += (int)(up ? got[q][5] >> 32 : (uint32_t)got[q][5]);
  }
  if (rank == owner) {
    bool found = false;
    if (tid == 0) sm.cut[2] = 0;
#pragma unroll 1
    for (int i = 0; i < per && !found; i += kThreads) {
      const int m = up ? m1 - 1 - i - tid : m0 + i + tid;
      const bool mine = m >= m0 && m < m1;
      const u64 c = mine ? counts(m) : 0;
      const uint32_t here = up ? (uint32_t)c : (uint32_t)(c >> 32);
      const float v = up ? magnitude(m) : -magnitude(m);
      const u64 t = here ? weight_fixed(v, w, sm.table) : 0;
      u64 whole, tokens;
      const u64 before = above + cta_exscan(here * t, sm.red[0], whole);
      const int n_before = n_above + (int)cta_exscan((u64)here, sm.red[1], tokens);
      const bool hit = before < want && want <= before + here * t;
      if (hit) {
        const uint32_t keep = (uint32_t)((want - before + t - 1) / t);
        sm.cut[0] = (u64)__float_as_uint(v) << 32 | (uint32_t)(n_before + (int)keep);
        sm.cut[1] = before + keep * t;
        sm.cut[2] = (u64)keep << 32 | here;
      }
      found = __syncthreads_or(hit);
      above += whole;
      n_above += (int)tokens;
    }
  }
  __syncthreads();
  rec[0] = sm.cut[0];
  rec[1] = sm.cut[1];
  rec[2] = sm.cut[2];
  got = exchange(sm.ex, turn, rec, 3, rank, size);
  const float value = __uint_as_float((uint32_t)(got[owner][0] >> 32));
  const int count = (int)(uint32_t)got[owner][0];
  const u64 sum = got[owner][1];
  int keep = (int)(got[owner][2] >> 32);
  cut = {value, kAll};
  if (keep < (int)(uint32_t)got[owner][2]) {
    // the last of `keep` tokens of this value, by index
    const uint32_t at =
        place((int)((__float_as_uint(value) >> 16 & 0x7FFFu) - kFirstMag)) + (up ? 0u : 512u);
    int here = lane < size ? (int)remote_get32(cluster_addr(at, lane)) : 0, upto = here;
#pragma unroll
    for (int d = 1; d < kMaxCluster; d <<= 1) {
      const int y = __shfl_up_sync(kFull, upto, d);
      if (lane >= d) upto += y;
    }
    // (the last CTA's sum is all of them: one lane reaches it)
    const int of = __ffs(__ballot_sync(kFull, upto >= keep)) - 1;
    keep -= __shfl_sync(kFull, upto - here, of);
    here = __shfl_sync(kFull, here, of);
    __syncthreads();  // (the list's last readers)
    if (tid == 0) sm.n_mine = 0;
    __syncthreads();
    if (here > kMine) {
      cluster_sync(size);  // (the counts' last readers)
      return false;
    }
    if (rank == of) {
      const uint32_t both_bits = (__float_as_uint(value) >> 16) * 0x10001u;
      for (int v = tid; v < s.nvec; v += kThreads) {
        const uint4 q = *reinterpret_cast<const uint4 *>(buf + (size_t)v * 16);
        const uint32_t a[4] = {q.x ^ both_bits, q.y ^ both_bits, q.z ^ both_bits, q.w ^ both_bits};
        unsigned same = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          same |= (e & 1 ? a[e >> 1] >> 16 : a[e >> 1] & 0xFFFFu) == 0 ? 1u << e : 0u;
        while (same) {
          const int e = __ffs(same) - 1;
          same &= same - 1;
          sm.mine[atomicAdd(&sm.n_mine, 1)] = place_of(value, s.first + v * 8 + e);
        }
      }
      __syncthreads();
      sort_down<kThreads>(sm.mine, here);
    }
    __syncthreads();
    rec[0] = (u64)(uint32_t)place_index(sm.mine[keep - 1]);
    got = exchange(sm.ex, turn, rec, 1, rank, size);
    cut.index = (int)got[of][0];
  }
  Z = sum;
  kept = count;
  return true;
}

// The tokens from `lo` up, on the list.
template <int DT>
__device__ __forceinline__ void gather(const Share &s, const uint8_t *buf, const Cut &lo,
                                       SampleSmem &sm) {
  constexpr int kN = Elem<DT>::kN;
  for (int v = threadIdx.x; v < s.nvec; v += kThreads) {
    const uint8_t *from = buf + (size_t)v * 16;
    if (!(max_of<DT>(vector_max<DT>(*reinterpret_cast<const uint4 *>(from), no_max<DT>())) >= lo.value))
      continue;
    unsigned reach = 0;
    float x[kN];
    widen<DT>(*reinterpret_cast<const uint4 *>(from), x);
#pragma unroll
    for (int e = 0; e < kN; ++e) reach |= x[e] >= lo.value ? 1u << e : 0u;
    while (reach) {
      const int e = __ffs(reach) - 1;
      reach &= reach - 1;
      const float y = get_elem<DT>(from + e * Elem<DT>::kBytes);
      const int at = s.first + v * kN + e;
      if (!lo.holds(y, at)) continue;
      const int k = atomicAdd(&sm.n_mine, 1);
      if (k < kMine) sm.mine[k] = place_of(y, at);
    }
  }
}

// The kept tokens' mass of each run, where they fit the list; the CTA's mass.
template <int DT>
__device__ __forceinline__ u64 weigh_few(const Share &s, const uint8_t *buf, const WeightOf &w,
                                         const Cut &cut, u64 *steps, SampleSmem &sm) {
  const int per = 32 * run_steps(s);
  for (int i = threadIdx.x; i * per < s.nvec; i += kThreads) steps[i] = 0;
  gather<DT>(s, buf, cut, sm);
  __syncthreads();
  u64 add = 0, mass;
  for (int i = threadIdx.x; i < sm.n_mine; i += kThreads) {
    const u64 q = sm.mine[i];
    const u64 t = weight_fixed(place_value(q), w, sm.table);
    atomicAdd(&steps[(place_index(q) - s.first) / Elem<DT>::kN / per], t);
    add += t;
  }
  (void)cta_exscan(add, sm.red[0], mass);
  return mass;
}

// All CTAs' lists, by rank 0, sorted.
__device__ __forceinline__ int collect(int size, SampleSmem &sm) {
  __syncthreads();  // (their numbers)
  int all = 0;
#pragma unroll 1
  for (int q = 0; q < size; ++q) all += sm.listed[q];
  for (int i = threadIdx.x; i < all; i += kThreads) {
    int q = 0, at = i;
    while (at >= sm.listed[q]) at -= sm.listed[q++];
    sm.list[i] = remote_get(cluster_addr(smem_addr(&sm.mine[at]), q));
  }
  __syncthreads();
  sort_down<kThreads>(sm.list, all);
  return all;
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p, int vectors) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  constexpr int es = Elem<DT>::kBytes, kN = Elem<DT>::kN;
  SampleSmem &sm = *reinterpret_cast<SampleSmem *>(smem_raw);
  const Layout l = layout_of(vectors);
  uint8_t *buf = smem_raw + l.share;
  u64 *steps = reinterpret_cast<u64 *>(smem_raw + l.steps);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster_rank(), size = cluster_size();
  const long long n = blockIdx.x / size;  // the row
  const long long b = n / p.R;
  const int r = (int)(n - b * p.R);
  int turn = 0;

  const uint8_t *row = reinterpret_cast<const uint8_t *>(p.x) +
                       (b * p.x_at.request + r * p.x_at.row) * es;
  const Share s = share_of<DT>(row, p.V, rank, size);
  if (tid == 0) {
    for (int i = 0; i < kChunks; ++i) mbar_init(&sm.in.full[i], 1);
    mbar_init(&sm.tabled, 1);
    sm.in.gave_up = 0;
    sm.n_mine = 0;
    fence_mbar_init();
    // (the table is no kernel's output)
    mbar_arrive_expect_tx(&sm.tabled, (uint32_t)sizeof(sm.table));
    bulk_copy_g2s(sm.table, &g_table, (uint32_t)sizeof(sm.table), &sm.tabled);
  }
  pdl_wait();
  pdl_launch_dependents();
  if (tid == 0) share_copy(s, buf, sm.in);
  // the request's filters
  float T = p.temperature[b];
  int k = p.top_k ? p.top_k[b] : 0;
  float top_p = p.top_p ? p.top_p[b] : 1.0f;
  float min_p = p.min_p ? p.min_p[b] : 0.0f;
  cluster_arrive_relaxed();  // (all CTAs run before one writes to another)
  __syncthreads();
  share_edges<DT>(s, row, buf);

  int st = 0;
  if (!temperature_valid(T)) st |= SPECDEC_ROW_BAD_TEMP;
  if (k < 0 || k > SPECDEC_MAX_TOPK || !(top_p >= 0.0f && top_p <= 1.0f) ||
      !(min_p >= 0.0f && min_p <= 1.0f))
    st |= SPECDEC_ROW_BAD_FILTER;
  if (T == 0.0f || st) {  // greedy: the first of the largest
    T = 1.0f;
    k = 1;
    top_p = 1.0f;
    min_p = 0.0f;
  }
  if (warp == 1 && min_p > 0.0f) {
    const double drop = (double)T * log((double)min_p);
    if (lane == 0) sm.drop = drop;
  }
  // log2(e) / T in two parts: the quotient, and what is left of it
  const float ch = __fdiv_rn(kLog2e, T);
  const float cl = __fdiv_rn(fmaf(-ch, T, kLog2e) + 1.9259629e-8f, T);

  // the largest logit, and the largest of each thread's part of every copy
  uint32_t top[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    top[i] = no_max<DT>();
    share_wait(sm.in, i);
    const int v1 = 1 + chunk_begin(s, i + 1);
    for (int v = 1 + chunk_begin(s, i) + tid; v < v1; v += kThreads)
      top[i] = vector_max<DT>(*reinterpret_cast<const uint4 *>(buf + (size_t)v * 16), top[i]);
  }
  if (!mbar_wait_bounded(&sm.tabled, 0, kConsumerWaitNs)) sm.in.gave_up = 1;
  __syncthreads();
  if (tid < 2)
    top[0] = vector_max<DT>(
        *reinterpret_cast<const uint4 *>(buf + (size_t)(tid ? s.nvec - 1 : 0) * 16), top[0]);
  float gm[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) gm[i] = max_of<DT>(top[i]);
  float M = fmax_nan(fmax_nan(gm[0], gm[1]), fmax_nan(gm[2], gm[3]));
  // top-k's groups: for small k a warp's lanes share some, 256 to 896 in all; else, and where
  // too few of those would hold tokens, each thread has one to four
  const int lanes = size < 4 ? 1 : size < 8 ? 2 : size < 16 ? 4 : 8;
  const int holding = min(kThreads, (int)((long long)p.V / kN / size / kChunks)) / lanes * size;
  const bool few = k <= kFewK && holding >= 4 * k;
  const int sub = few || size > 4 || size == 3 ? 1 : size == 4 ? 2 : 4;
  const int fold = few ? lanes : 1;
  const int own = kThreads * sub / fold, groups = own * size;
  cluster_wait();
  if (k > 0) {
    if (sub == 2) {
      gm[0] = fmax_nan(gm[0], gm[2]);
      gm[1] = fmax_nan(gm[1], gm[3]);
    } else if (sub == 1) {
      gm[0] = M;
    }
#pragma unroll 1
    for (int d = 1; d < fold; d *= 2) gm[0] = fmax_nan(gm[0], __shfl_xor_sync(kFull, gm[0], d));
    if (tid % fold == 0) {
#pragma unroll 1
      for (int q = 0; q < size; ++q) {
        const uint32_t to = cluster_addr(smem_addr(&sm.key[rank * own + tid / fold * sub]), q);
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
          if (i < sub) remote_put16(to + 2u * i, order_key(gm[i]) >> 16);
      }
    }
  }
  M = cta_max_nan<kWarps>(M, sm.redf[0]);
  u64 rec[kWords];
  rec[0] = (u64)(sm.in.gave_up ? SPECDEC_ROW_INTERNAL : 0) << 32 | __float_as_uint(M);
  const u64(*got)[kWords] = exchange(sm.ex, turn, rec, 1, rank, size);
  M = -INFINITY;
#pragma unroll 1
  for (int q = 0; q < size; ++q) {
    M = fmax_nan(M, __uint_as_float((uint32_t)got[q][0]));
    st |= (int)(got[q][0] >> 32);
  }
  if (!(st & SPECDEC_ROW_INTERNAL) && !(M > -INFINITY && M <= kMaxLogit)) st |= SPECDEC_ROW_NONFINITE;

  // (from here every CTA of the cluster takes the same branches: they turn on the
  // request's filters and on exchanged records)
  const WeightOf w = weight_of(M, ch, cl);
  Cut cut = {kLeast, kAll};  // everything but -infinity
  u64 Z = 0;                 // the kept mass
  int kept = 0;
  const float floor_value =
      min_p > 0.0f ? __double2float_ru((double)M + sm.drop) : kLeast;
  const u64 over = ((u64)order_key(M) + 1) << 32;  // above every place
  const float *u = p.uniforms + n * p.S;
  int32_t *tokens = p.tokens + n * p.S;

  if (!st && k > 0) {
    // ---- top-k: the few largest, by rank 0 --------------------------------------------
    // (bit by bit, by one warp: with a barrier of the CTA for every bit this took 8000 to 9500
    // of a small row's 30000 clocks)
    if (warp == 0) {
      constexpr int kHeld = 8;  // pairs of keys that a lane holds
      const uint32_t *pairs = reinterpret_cast<const uint32_t *>(sm.key);
      uint32_t held[kHeld], found = 0;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) held[i] = lane + 32 * i < groups / 2 ? pairs[lane + 32 * i] : 0;
      const uint32_t most = order_key(M) >> 16;
#pragma unroll 1
      for (int bit = 15; bit >= 0; --bit) {
        const uint32_t t = found | 1u << bit;
        if (t > most) continue;
        unsigned m0 = 0, m1 = 0;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          m0 += (held[i] & 0xFFFFu) >= t;
          m1 += (held[i] >> 16) >= t;
        }
#pragma unroll 4
        for (int i = lane + 32 * kHeld; i < groups / 2; i += 32) {
          m0 += (pairs[i] & 0xFFFFu) >= t;
          m1 += (pairs[i] >> 16) >= t;
        }
        if (__reduce_add_sync(kFull, m0 + m1) >= (unsigned)k) found = t;
      }
      if (lane == 0) sm.bound = found;
    }
    __syncthreads();
    const uint32_t bound = sm.bound;
    // At least k tokens (or all that are finite) stand at places >= from, fewer than k at
    // places >= H.  Where those at `from` are too many to list, halves of what is between:
    // at the end exactly k.
    u64 from = (u64)max(bound << 16, kLeastKey) << 32, H = over, probe = from;
    for (int i = 0;; ++i) {
      gather<DT>(s, buf, cut_at(probe), sm);
      __syncthreads();
      rec[0] = (u64)(uint32_t)sm.n_mine;
      got = exchange(sm.ex, turn, rec, 1, rank, size);
      int all = 0;
      bool fits = true;
#pragma unroll 1
      for (int q = 0; q < size; ++q) {
        if (tid == 0) sm.listed[q] = (int)got[q][0];
        all += (int)got[q][0];
        fits = fits && got[q][0] <= kMine;
      }
      const bool enough = probe == from || all >= k;
      if (enough && fits && all <= kList) break;
      if (i == kLimit) {
        st = SPECDEC_ROW_INTERNAL;
        break;
      }
      if (enough) from = probe;
      else H = probe;
      probe = from + (H - from) / 2;
      __syncthreads();
      if (tid == 0) sm.n_mine = 0;
      __syncthreads();
    }
    if (rank == 0 && !st) {
      const int m = min(k, collect(size, sm));
      // weights of the first k, four a thread, and their sums
      constexpr int kEach = SPECDEC_MAX_TOPK / kThreads;
      const int each = (m + kThreads - 1) / kThreads;  // of neighbours, a thread
      u64 wt[kEach], mine = 0, whole;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int j = tid * each + i;
        wt[i] = i < each && j < m ? weight_fixed(place_value(sm.list[j]), w, sm.table) : 0;
        mine += wt[i];
      }
      u64 before = cta_exscan(mine, sm.red[0], whole);
      const u64 want = top_p < 1.0f ? share_at_least(top_p, whole) : ~0ull;
      // kept: places before which less than the wanted mass stands
      int c = 0;
      u64 sum = before;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int j = tid * each + i;
        c += i < each && j < m && (sum < want || j == 0) && place_value(sm.list[j]) >= floor_value;
        sum += wt[i];
      }
      if (tid == 0) sm.n_kept = 0;
      __syncthreads();
      c = __reduce_add_sync(kFull, c);
      if (lane == 0) atomicAdd(&sm.n_kept, c);
      __syncthreads();
      const int nk = sm.n_kept;
      // (sm.mine's own tokens are on the list by now: it holds weights)
      sum = before;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int j = tid * each + i;
        sum += wt[i];
        if (i < each && j == nk - 1) {
          sm.cut[0] = sm.list[j];
          sm.cut[1] = sum;
        }
        if (i < each && j < nk) sm.mine[j] = wt[i];
      }
      __syncthreads();
      Z = sm.cut[1];
      rec[0] = sm.cut[0];
      rec[1] = Z;
      rec[2] = (u64)nk;
      if (p.S > 0) {
        // the kept by index, and the draws
        for (int i = tid; i < nk; i += kThreads)
          sm.list[i] = (u64)(uint32_t)sm.list[i] << 32 | (uint32_t)i;
        __syncthreads();
        sort_down<kThreads>(sm.list, nk);
        int token[kEach];
        mine = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int j = tid * each + i;
          const u64 q = i < each && j < nk ? sm.list[j] : 0;
          token[i] = (int)(0xFFFFFFFFu - (uint32_t)(q >> 32));
          wt[i] = i < each && j < nk ? sm.mine[(uint32_t)q] : 0;
          mine += wt[i];
        }
        before = cta_exscan(mine, sm.red[1], whole);
        for (int d = 0; d < p.S; ++d) {
          const u64 target = uniform_target(u[d], Z);
          sum = before;
#pragma unroll
          for (int i = 0; i < kEach; ++i) {
            if (sum <= target && target < sum + wt[i]) tokens[d] = token[i];
            sum += wt[i];
          }
        }
      }
    }
    __syncthreads();
    got = exchange(sm.ex, turn, rec, 3, rank, size);
    cut = cut_at(got[0][0]);
    Z = got[0][1];
    kept = (int)got[0][2];
  } else if (!st) {
    // ---- the whole vocabulary ----------------------------------------------------------
    bool weighed = false;    // steps[] holds the kept mass
    u64 mass = 0, before = 0;  // kept in this CTA, and in those before it
    int n_in;
    bool fits;
    if (floor_value > kLeast) cut = {floor_value, kAll};
    bool found = false;
    if (DT == SPECDEC_BF16 && p.V >= kCountFrom && top_p < 1.0f && M < kMostMag) {
      found = cut_by_values(s, buf, w, M, top_p, floor_value, rank, size, turn, cut, Z, kept, sm);
      __syncthreads();
      if (tid == 0) sm.n_mine = 0;
      __syncthreads();
      if (found && p.S == 0) {
        weighed = true;
      } else if (found && kept <= kMine) {
        mass = weigh_few<DT>(s, buf, w, cut, steps, sm);
        rec[0] = mass;
        got = exchange(sm.ex, turn, rec, 1, rank, size);
#pragma unroll 1
        for (int q = 0; q < rank; ++q) before += got[q][0];
        weighed = true;
      } else if (found && cut.index != kAll) {
        weigh_row<DT, kBracket>(s, buf, w, cut, cut, steps, rank, size, turn, mass, before, n_in, fits, sm);
        weighed = true;
      }
    }
    if (top_p < 1.0f && !found) {
      // less than the wanted mass stands above H, all of it down to L: sums are exact, so that
      // this holds throughout, and halves end
      u64 L = (u64)max(order_key(M - 45.0f / ch), kLeastKey) << 32, H = over, lo, hi;
      const u64 least = (u64)order_key(cut.value) << 32;  // min_p's cut
      int n_low = kAll, n_high = 0;                       // tokens down to L and to H
      float guess = top_p, hist_before;
      Found f;  // of the whole row
      u64 want;
      histogram<DT>(s, buf, M, ch, size, sm);
      for (int tries = 0;; ++tries) {
        if (tries == kLimit) {
          st = SPECDEC_ROW_INTERNAL;
          break;
        }
        if (tries < kTries) {
          int first, last;
          place_bracket(guess, tries == 0, size, sm, first, last, hist_before);
          const float bin = 1.0f / (ch * kOctave);
          const u64 from = (u64)max(order_key(M - ((float)last + 0.5f) * bin), kLeastKey) << 32;
          const u64 to = first > 0 ? (u64)order_key(M - ((float)first - 0.5f) * bin) << 32 : over;
          lo = max(from, L);
          hi = min(to, H);
          if (lo >= hi && tries == 0) {  // (bins finer than the logits: what they weigh, first)
            lo = L;
            hi = H;
          } else if (lo >= hi) {  // (the bins point beyond what is known)
            tries = kTries - 1;
            continue;
          }
        } else if (n_low - n_high <= kMine || H - L <= 1) {
          lo = L;
          hi = H;
        } else {
          hi = L + (H - L) / 2;
          f = weigh_row<DT, kBracket>(s, buf, w, cut_at(hi), cut_at(hi), steps, rank, size, turn, mass,
                                   before, n_in, fits, sm);
          if (want <= f.above) {
            L = hi;
            n_low = f.n_above;
          } else {
            H = hi;
            n_high = f.n_above;
          }
          continue;
        }
        // a bracket below min_p's cut: all that can be asked is what stands down to that
        const bool floored = hi <= least;
        if (floored) lo = hi = min(least, over);
        f = weigh_row<DT, kBracket>(s, buf, w, cut_at(hi), cut_at(lo), steps, rank, size, turn, mass,
                                    before, n_in, fits, sm);
        want = max(share_at_least(top_p, f.all), 1ull);
        if (want > f.above && floored) {
          weighed = true;
          break;
        }
        u64 in = 0;
        if (want > f.above && fits && !floored) {
          // the list: in place order, up to the one that reaches the mass
          u64 rec2[kWords];  // (rank 0's counts)
          if (rank == 0) {
            const int all = collect(size, sm);
            constexpr int kEach = kList / kThreads;
            const int each = (all + kThreads - 1) / kThreads;  // of neighbours, a thread
            u64 wt[kEach], mine = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
              const int j = tid * each + i;
              wt[i] = i < each && j < all ? weight_fixed(place_value(sm.list[j]), w, sm.table) : 0;
              mine += wt[i];
            }
            u64 sum = f.above + cta_exscan(mine, sm.red[1], in);
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
              const int j = tid * each + i;
              if (sum < want && sum + wt[i] >= want) {
                sm.cut[0] = sm.list[j];
                sm.cut[1] = (u64)(f.n_above + j + 1);
                sm.cut[2] = sum + wt[i];
              }
              sum += wt[i];
            }
          }
          __syncthreads();
          rec2[0] = sm.cut[0];
          rec2[1] = sm.cut[1];
          rec2[2] = sm.cut[2];
          rec2[3] = in;
          got = exchange(sm.ex, turn, rec2, 4, rank, size);
          in = got[0][3];
          if (want <= f.above + in) {
            cut = cut_at(got[0][0]);
            kept = (int)got[0][1];
            Z = got[0][2];
            break;
          }
          H = lo;
          n_high = f.n_above + n_in;
        } else if (want > f.above) {
          H = hi;
          n_high = f.n_above;
          tries = kTries;  // (too many for the list)
        } else {
          L = hi;
          n_low = f.n_above;
        }
        // the histogram's mass is off by what the pass shows at the bracket's upper end
        const float unit = ex2_approx(-w.rest) / kFixed;
        guess = hist_before + ((float)want - (float)f.above) * unit;
        // (rank 0's list stands where its histogram was: it is made again)
        if (tries < kTries - 1) histogram<DT>(s, buf, M, ch, size, sm);
        __syncthreads();
        if (tid == 0) sm.n_mine = 0;
        __syncthreads();
      }
      if (st) {
        weighed = true;
      } else if (weighed) {
        kept = f.n_above;
        Z = f.above;
      } else if (floor_value > cut.value) {
        cut = {floor_value, kAll};
      } else if (p.S == 0) {
        weighed = true;
      } else {
        // the list's kept tokens join their runs
        u64 add = 0, more;
        for (int i = tid; i < sm.n_mine; i += kThreads) {
          const u64 q = sm.mine[i];
          if (!cut.holds(place_value(q), place_index(q))) continue;
          const u64 t = weight_fixed(place_value(q), w, sm.table);
          atomicAdd(&steps[(place_index(q) - s.first) / kN / (32 * run_steps(s))], t);
          add += t;
        }
        (void)cta_exscan(add, sm.red[0], more);
        mass += more;
        rec[0] = mass;
        got = exchange(sm.ex, turn, rec, 1, rank, size);
        before = 0;
#pragma unroll 1
        for (int q = 0; q < rank; ++q) before += got[q][0];
        weighed = true;
      }
    }
    if (!weighed) {
      const Found f = weigh_row<DT, kWhole>(s, buf, w, cut, cut, steps, rank, size, turn, mass, before,
                                            n_in, fits, sm);
      Z = f.above;
      kept = f.n_above;
    }

    // the draws that fall into this CTA's mass
    for (int d = warp; d < p.S && !st; d += kWarps) {
      const u64 target = uniform_target(u[d], Z);
      if (target < before || target - before >= mass) continue;
      u64 left = target - before;
      // the run: 32 at a time
      int at = -1;
      const int per = run_steps(s), runs = (s.nvec + 32 * per - 1) / (32 * per);
      for (int i0 = 0; i0 < runs && at < 0; i0 += 32) {
        const u64 t = i0 + lane < runs ? steps[i0 + lane] : 0;
        const u64 inc = warp_incscan(t);
        const unsigned hit = __ballot_sync(kFull, inc > left);
        if (hit) at = i0 + __ffs(hit) - 1;
        left -= hit ? shfl_u64(inc - t, __ffs(hit) - 1) : shfl_u64(inc, 31);
      }
      // the token: the run's weights once more
      for (int q = 0; q < per; ++q) {
        const int v = 32 * (per * at + q) + lane;
        const int first = s.first + v * kN;
        uint32_t a_sum = 0, b_sum = 0;
        int n = 0;
        if (v < s.nvec) {
          float2 x[kN / 2];
          widen2<DT>(*reinterpret_cast<const uint4 *>(buf + (size_t)v * 16), x);
#pragma unroll
          for (int e = 0; e < kN / 2; ++e) {
            uint32_t a[2], c[2];
            weight2(x[e], w, sm.table, a, c);
            if (cut.holds(x[e].x, first + 2 * e)) {
              a_sum += a[0];
              b_sum += c[0];
              ++n;
            }
            if (cut.holds(x[e].y, first + 2 * e + 1)) {
              a_sum += a[1];
              b_sum += c[1];
              ++n;
            }
          }
        }
        const u64 t = fixed_sum(a_sum, b_sum, n);
        const u64 inc = warp_incscan(t), whole = shfl_u64(inc, 31);
        if (left >= whole) {
          left -= whole;
          continue;
        }
        u64 sum = inc - t;
        if (sum <= left && left < inc) {
          int e = 0;
          for (; e < kN - 1; ++e) {
            const float y = get_elem<DT>(buf + (size_t)v * 16 + e * es);
            if (cut.holds(y, first + e)) sum += weight_fixed(y, w, sm.table);
            if (left < sum) break;
          }
          tokens[d] = first + e;
        }
        break;
      }
    }
  }

  if (st) {
    if (rank == 0)
      for (int d = tid; d < p.S; d += kThreads) tokens[d] = -1;
    kept = 0;
  }
  if (rank == 0 && tid == 0) {
    p.kept[n] = kept;
    p.row_status[n] = st;
  }
  if (p.rows) {
    uint8_t *out = reinterpret_cast<uint8_t *>(p.rows) +
                   (b * p.rows_at.request + r * p.rows_at.row) * es;
    const bool like =
        ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    // 2^rest 2^42 / Z, rounded about once: 1 / Z's error and 2^rest - 1 are small terms
    const float zf = __ull2float_rn(Z), q0 = __fdiv_rn(kFixed, zf);
    const float off = fmaf(-q0, zf, kFixed) / zf - (float)(long long)(Z - __float2ull_rn(zf)) * (q0 / zf);
    const float up = w.rest * fmaf(w.rest, fmaf(w.rest, 0.0555041087f, 0.240226507f), 0.693147181f);
    const float g = q0 + fmaf(q0, up, off);
    const bool ties = cut.index != kAll;
    // kept: above this, and what of the cut's own value the index lets through
    const float under = ties ? cut.value : just_below(cut.value);
    __syncthreads();  // (draws read the share)
    for (int v = tid; v < s.nvec; v += kThreads) {
      const uint4 in = *reinterpret_cast<const uint4 *>(buf + (size_t)v * 16);
      float2 x[kN / 2];
      widen2<DT>(in, x);
      uint4 y;
      if (st) {
#pragma unroll
        for (int e = 0; e < kN / 2; ++e) x[e] = both(__int_as_float(0x7fc00000));
      } else if (p.logits) {
#pragma unroll
        for (int e = 0; e < kN / 2; ++e)
          x[e] = make_float2(x[e].x > under ? x[e].x : -INFINITY, x[e].y > under ? x[e].y : -INFINITY);
      } else {
        // (most vectors of a row under a filter keep nothing)
        if (max_of<DT>(vector_max<DT>(in, no_max<DT>())) > under) {
#pragma unroll
          for (int e = 0; e < kN / 2; ++e) {
            const float2 q = __fmul2_rn(both(g), exp2_pair(x[e], M, ch));
            x[e] = make_float2(x[e].x > under ? q.x : 0.0f, x[e].y > under ? q.y : 0.0f);
          }
        } else {
#pragma unroll
          for (int e = 0; e < kN / 2; ++e) x[e] = both(0.0f);
        }
      }
      y = narrow2<DT>(x);
      if (ties && !st) {
        // tokens of the cut's value
        const int at = s.first + v * kN;
        const float same = p.logits ? cut.value : g * exp2_pair(both(cut.value), M, ch).x;
        const uint32_t a[4] = {in.x, in.y, in.z, in.w};
        uint32_t o[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const float z = DT == SPECDEC_F32 ? __uint_as_float(a[e & 3])
                                            : e & 1 ? bf16_hi(a[e >> 1]) : bf16_lo(a[e >> 1]);
          if (z != cut.value || at + e > cut.index) continue;
          if (DT == SPECDEC_F32)
            o[e & 3] = p.logits ? a[e & 3] : __float_as_uint(same);
          else if (e & 1)
            o[e >> 1] = (o[e >> 1] & 0xFFFFu) | two_bf16(0.0f, same);
          else
            o[e >> 1] = (o[e >> 1] & 0xFFFF0000u) | two_bf16(same, 0.0f);
        }
        y = make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (like)
        store_like<DT>(s, out, v, y);
      else
        *reinterpret_cast<uint4 *>(buf + (size_t)v * 16) = y;
    }
    if (!like) {
      __syncthreads();
      store_unlike<DT, kThreads>(s, buf, out);
    }
  }
  if (sm.in.gave_up && tid == 0) {
    share_drain(sm.in);
    mbar_wait_bounded(&sm.tabled, 0);
  }
}

template <int DT>
cudaError_t launch_dt(const SampleParams &p, cudaStream_t stream) {
  static DeviceOnce once;
  const cudaError_t err = cluster_opt_in_once(once, sample_kernel<DT>, 227 * 1024);
  if (err != cudaSuccess) return err;
  constexpr int es = Elem<DT>::kBytes;
  const long long rows = (long long)p.B * p.R;
  const int size = cluster_for(rows, p.V, es, 68 * 1024, 2);
  const int vectors = share_vectors(p.V, es, size);
  return launch_clusters(sample_kernel<DT>, rows, size, kThreads, layout_of(vectors).total, stream, p,
                         vectors);
}

}  // namespace

cudaError_t launch_sample(const SampleParams &p, cudaStream_t stream) {
  return p.dtype == SPECDEC_F32 ? launch_dt<SPECDEC_F32>(p, stream) : launch_dt<SPECDEC_BF16>(p, stream);
}

}  // namespace specdec
