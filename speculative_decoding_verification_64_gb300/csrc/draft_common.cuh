// Shared pieces of the draft side of the step (specdec_sample, specdec_top_logits,
// specdec_distill): parameters, rows of logits held by a cluster of CTAs in shared
// memory, and the exchange of a few words between those CTAs.
#pragma once

#include "common.cuh"

namespace specdec {

// Rows (b, r) of V elements at base + b * request + r * row elements.
struct RowsAt {
  long long request, row;
};

struct SampleParams {
  const void *x;
  RowsAt x_at;
  const float *temperature;  // [B]
  const int32_t *top_k;      // [B] or NULL
  const float *top_p;        // [B] or NULL
  const float *min_p;        // [B] or NULL
  const float *uniforms;     // [B, R, S]
  int dtype, B, R, V, S;
  int32_t *tokens;           // [B, R, S]
  void *rows;                // or NULL
  RowsAt rows_at;
  int logits;                // rows holds logits, not probabilities
  int32_t *kept;             // [B, R]
  int32_t *row_status;       // [B, R]
};

constexpr int kTopGroups = 16;  // of a stage's 8 KB

struct TopParams {
  const void *x;
  RowsAt x_at;
  float temperature;
  float inv_t, inv_t_low;  // 1 / temperature, in two parts
  int dtype, B, R, V, K;
  int spr;               // stages a row (as in the row statistics)
  float2 *part;          // [rows, spr]: each stage's maximum and sum, in the workspace
  float *group;          // [rows, spr, kTopGroups]: the maximum of each 512 bytes
  float *values;         // [B, R, K]
  int32_t *ids;          // [B, R, K]
  float *lse;            // [B, R]
  int32_t *row_status;   // [B, R]
};

struct DistillParams {
  const void *x;
  RowsAt x_at;
  const int32_t *ids;    // [B, R, K]
  const float *teacher;  // [B, R, K]
  const float *lse;      // [B, R] or NULL
  const float *weight;   // [B, R] or NULL
  const float *dloss;    // [B, R]: the backward call; NULL otherwise
  float temperature;
  float inv_t, inv_t_low;  // 1 / temperature, in two parts
  int dtype, B, R, V, K;
  float *loss;           // [B, R]; NULL in the backward call, as row_status
  void *grad;            // or NULL
  RowsAt grad_at;
  int32_t *row_status;   // [B, R]
};

cudaError_t launch_sample(const SampleParams &p, cudaStream_t stream);
cudaError_t launch_top_logits(const TopParams &p, cudaStream_t stream);
cudaError_t launch_distill(const DistillParams &p, cudaStream_t stream);

constexpr int kMaxCluster = 16;

#ifdef __CUDACC__

constexpr unsigned kFull = 0xffffffffu;

// ---- elements -------------------------------------------------------------------------

template <int DT>
struct Elem {
  static constexpr int kBytes = DT == SPECDEC_F32 ? 4 : 2;
  static constexpr int kN = 16 / kBytes;  // elements of a 16-byte vector
};

template <int DT>
__device__ __forceinline__ void widen(const uint4 &w, float *x) {
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (DT == SPECDEC_F32) {
      x[i] = __uint_as_float(a[i]);
    } else {
      x[2 * i] = bf16_lo(a[i]);
      x[2 * i + 1] = bf16_hi(a[i]);
    }
  }
}

__device__ __forceinline__ uint32_t two_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int DT>
__device__ __forceinline__ uint4 narrow(const float *x) {
  if (DT == SPECDEC_F32)
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  return make_uint4(two_bf16(x[0], x[1]), two_bf16(x[2], x[3]), two_bf16(x[4], x[5]),
                    two_bf16(x[6], x[7]));
}

// The same as pairs of neighbours, for packed arithmetic.
template <int DT>
__device__ __forceinline__ void widen2(const uint4 &w, float2 *x) {
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
  if (DT == SPECDEC_F32) {
    x[0] = make_float2(__uint_as_float(a[0]), __uint_as_float(a[1]));
    x[1] = make_float2(__uint_as_float(a[2]), __uint_as_float(a[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(bf16_lo(a[i]), bf16_hi(a[i]));
  }
}

template <int DT>
__device__ __forceinline__ uint4 narrow2(const float2 *x) {
  if (DT == SPECDEC_F32)
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                      __float_as_uint(x[1].y));
  return make_uint4(two_bf16(x[0].x, x[0].y), two_bf16(x[1].x, x[1].y), two_bf16(x[2].x, x[2].y),
                    two_bf16(x[3].x, x[3].y));
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// 2^((x - m) c) of a pair
__device__ __forceinline__ float2 exp2_pair(float2 x, float m, float c) {
  x = __fmul2_rn(__fadd2_rn(x, both(-m)), both(c));
  return make_float2(ex2_approx(x.x), ex2_approx(x.y));
}

// The larger of a vector's elements and `m` (NaN where one is), held as 16 bytes' own types:
// two bfloat16 or one float32 in a word.
template <int DT>
__device__ __forceinline__ uint32_t vector_max(const uint4 &w, uint32_t m) {
  uint32_t r = m;
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (DT == SPECDEC_F32)
      r = __float_as_uint(fmax_nan(__uint_as_float(r), __uint_as_float(a[i])));
    else
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(a[i]));
  }
  return r;
}
template <int DT>
__device__ __forceinline__ uint32_t no_max() {
  return DT == SPECDEC_F32 ? 0xFF800000u : 0xFF80FF80u;
}
template <int DT>
__device__ __forceinline__ float max_of(uint32_t m) {
  return DT == SPECDEC_F32 ? __uint_as_float(m) : fmax_nan(bf16_lo(m), bf16_hi(m));
}

template <int DT>
__device__ __forceinline__ float get_elem(const uint8_t *p) {
  if (DT == SPECDEC_F32) return *reinterpret_cast<const float *>(p);
  return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(p) << 16);
}

template <int DT>
__device__ __forceinline__ void put_elem(uint8_t *p, float x) {
  if (DT == SPECDEC_F32)
    *reinterpret_cast<float *>(p) = x;
  else
    *reinterpret_cast<uint16_t *>(p) = (uint16_t)two_bf16(x, 0.0f);
}

// ---- places ---------------------------------------------------------------------------

// Keys that order like the values, -0 like +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float key_float(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

constexpr uint32_t kLeastKey = 0x00800000u;  // of the least finite value

// A token among others of its row: the larger first, equal ones by index.
__device__ __forceinline__ unsigned long long place_of(float x, int index) {
  return (unsigned long long)order_key(x) << 32 | (0xFFFFFFFFu - (uint32_t)index);
}
__device__ __forceinline__ float place_value(unsigned long long p) {
  return key_float((uint32_t)(p >> 32));
}
__device__ __forceinline__ int place_index(unsigned long long p) {
  return (int)(0xFFFFFFFFu - (uint32_t)p);
}

// Sorts list[0, n) in kE chunks of one token a thread each: a token's rank in its own chunk is
// counted, its rank in the others, once they are sorted, found by halves.
template <int kThreads, int kE>
__device__ __forceinline__ void sort_by_rank(unsigned long long *list, int n) {
  const int tid = threadIdx.x;
  unsigned long long v[kE];
  int rank[kE];
#pragma unroll
  for (int i = 0; i < kE; ++i) {
    const int at = tid + i * kThreads, len = min(n - i * kThreads, kThreads);
    v[i] = at < n ? list[at] : 0ull;
    rank[i] = 0;
#pragma unroll 4
    for (int j = 0; j < len; ++j) rank[i] += list[i * kThreads + j] > v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kE; ++i)
    if (tid + i * kThreads < n) list[i * kThreads + rank[i]] = v[i];
  __syncthreads();
  if constexpr (kE > 1) {
#pragma unroll 1
    for (int c = 0; c * kThreads < n; ++c) {
      const int len = min(n - c * kThreads, kThreads);
      int above[kE];  // tokens of the chunk that are larger
#pragma unroll
      for (int i = 0; i < kE; ++i) above[i] = 0;
#pragma unroll 1
      for (int step = kThreads; step > 0; step /= 2) {
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          const int at = above[i] + step;
          if (at <= len && list[c * kThreads + at - 1] > v[i]) above[i] = at;
        }
      }
#pragma unroll
      for (int i = 0; i < kE; ++i) rank[i] += i == c ? 0 : above[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kE; ++i)
      if (tid + i * kThreads < n) list[rank[i]] = v[i];
    __syncthreads();
  }
}

// Sorts the CTA's list[0, n) downwards, n <= 1024, all tokens of it different and none 0
// (17 tokens: 800 clocks, 70 to 95 tokens: 2000 to 3000 beside another working CTA, where a
// bitonic network took 6700; records of 512 entries of 1500 rows of 32000 128 us, each token
// compared with all others 144).
template <int kThreads>
__device__ __noinline__ void sort_down(unsigned long long *list, int n) {
  if (n <= kThreads)
    sort_by_rank<kThreads, 1>(list, n);
  else
    sort_by_rank<kThreads, 1024 / kThreads>(list, n);
}

// m / T + ln s for s > 0, rounded about once: in units of 2^-40, where its parts are not
// beyond them.  inv_t + inv_t_low is 1 / T.
__device__ __forceinline__ float log_sum(float m, float inv_t, float inv_t_low, float s) {
  int e;
  const float f = frexpf(s, &e);
  const float a = m * inv_t, low = fmaf(m, inv_t, -a) + m * inv_t_low;
  if (!(fabsf(a) < 0x1p21f)) return a + (low + logf(s));
  const long long t = __float2ll_rn(a * 0x1p40f) + __float2ll_rn((low + logf(f)) * 0x1p40f) +
                      (long long)e * 762123384786ll;  // ln 2
  return (float)t * 0x1p-40f;
}

// ---- clusters -------------------------------------------------------------------------

__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}

__device__ __forceinline__ int cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return (int)r;
}

// Every thread of every CTA of the cluster arrives, then waits.  (A barrier of the
// hardware between CTAs that run together; no thread leaves a kernel below before its
// last one.)
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
// The same where this thread has nothing to show the other CTAs.
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The cluster's barrier for what stands before a barrier of the CTA (or was written by the
// first warp): the first warp alone releases it, as that waits for all stores in flight (3 to
// 8 % of the kernels' time with all warps).  A CTA alone has its own barrier (4 to 10 % for
// rows that one CTA holds).
__device__ __forceinline__ void cluster_sync(int size) {
  if (size == 1) {
    __syncthreads();
    return;
  }
  if (threadIdx.x < 32) cluster_arrive();
  else cluster_arrive_relaxed();
  cluster_wait();
}

__device__ __forceinline__ void remote_put(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void remote_put16(uint32_t addr, uint32_t v) {
  asm volatile("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tst.shared::cluster.u16 [%0], h;\n\t}" ::"r"(addr),
               "r"(v)
               : "memory");
}
__device__ __forceinline__ unsigned long long remote_get(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// (one of many that may be under way together, between two barriers of the cluster)
__device__ __forceinline__ unsigned long long remote_get_weak(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t remote_get32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

constexpr int kWords = 8;  // of one CTA's record in an exchange

// What the CTAs of a cluster tell one another: two buffers used in turn, so that a CTA
// may write its next record while others still read the last one.
struct Exchange {
  unsigned long long rec[2][kMaxCluster][kWords];
};

// Thread c of the CTA writes the record to CTA c of the cluster; behind the barrier every
// CTA reads all records from its own shared memory.  `rec` is valid in the first `size`
// threads.  Called by all threads, behind a barrier of the CTA.
__device__ __forceinline__ const unsigned long long (*exchange(Exchange &ex, int &turn,
                                                               const unsigned long long *rec,
                                                               int words, int rank,
                                                               int size))[kWords] {
  const int t = turn & 1;
  turn ^= 1;
  if ((int)threadIdx.x < size) {
    const uint32_t at = cluster_addr(smem_addr(&ex.rec[t][rank][0]), threadIdx.x);
    for (int i = 0; i < words; ++i) remote_put(at + 8u * i, rec[i]);
  }
  __syncwarp();
  cluster_sync(size);
  return ex.rec[t];
}

// ---- sums over a CTA ------------------------------------------------------------------

// Sum of v over the CTA in a fixed order; `red` holds one value a warp.  Every thread
// gets it.  A barrier before `red` is used again.
template <int kWarps>
__device__ __forceinline__ float cta_sum(float v, float *red) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += red[w];
  return s;
}

template <int kWarps>
__device__ __forceinline__ float cta_max_nan(float v, float *red) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v = fmax_nan(v, __shfl_xor_sync(kFull, v, d));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float m = red[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) m = fmax_nan(m, red[w]);
  return m;
}

// ---- a CTA's share of a row -----------------------------------------------------------

// A row's 16-byte aligned inside is cut into equal runs of vectors, one for each CTA of
// the cluster in rank order.  The elements before it belong to rank 0, those behind it to
// the last rank.  In shared memory a share is vectors 0 .. nvec-1: vector 0 ends with the
// elements before the inside, vectors 1 .. body are the run, the last one begins with the
// elements behind; what is left of those two is -infinity.
struct Share {
  const uint8_t *src;  // the run in global memory, 16-byte aligned
  int body;            // its vectors
  int nvec;            // body + 2
  int first;           // the row's index of vector 0's first element (may be negative)
  int begin, end;      // the row's elements of this CTA
};

template <int DT>
__device__ __forceinline__ Share share_of(const uint8_t *row, int V, int rank, int size) {
  constexpr int es = Elem<DT>::kBytes, kN = Elem<DT>::kN;
  const int mis = (int)(reinterpret_cast<uintptr_t>(row) & 15);
  const int head = min(V, mis ? (16 - mis) / es : 0);
  const int inside = (V - head) / kN;
  const int per = (inside + size - 1) / size;
  const int v0 = min(rank * per, inside), v1 = min(v0 + per, inside);
  Share s;
  s.src = row + (size_t)head * es + (size_t)v0 * 16;
  s.body = v1 - v0;
  s.nvec = s.body + 2;
  s.first = head + (v0 - 1) * kN;
  s.begin = rank == 0 ? 0 : head + v0 * kN;
  s.end = rank == size - 1 ? V : head + v1 * kN;
  return s;
}

// Vectors that the largest share of a row takes in shared memory, whatever its alignment.
inline int share_vectors(int V, int elem_bytes, int size) {
  const int inside = (int)(((long long)V * elem_bytes) / 16);
  return (inside + size - 1) / size + 2;
}

constexpr int kChunks = 4;  // copies that bring a share, each with its own barrier

struct Arrival {
  alignas(8) uint64_t full[kChunks];
  int gave_up;
};

// The first vector of copy i of a share's run, and one past the last copy's.
__device__ __forceinline__ int chunk_begin(const Share &s, int i) {
  const int per = (s.body + kChunks - 1) / kChunks;
  return min(i * per, s.body);
}

// One thread, after the barriers were made (and everybody knows): the copies.
__device__ __forceinline__ void share_copy(const Share &s, uint8_t *buf, Arrival &in) {
  for (int i = 0; i < kChunks; ++i) {
    const int v0 = chunk_begin(s, i), n = chunk_begin(s, i + 1) - v0;
    if (n > 0) {
      mbar_arrive_expect_tx(&in.full[i], (uint32_t)n * 16);
      bulk_copy_g2s(buf + (size_t)(1 + v0) * 16, s.src + (size_t)v0 * 16, (uint32_t)n * 16,
                    &in.full[i]);
    } else {
      mbar_arrive(&in.full[i]);
    }
  }
}

// The two edge vectors, by the CTA's first 2 kN threads.  A barrier before they are read.
template <int DT>
__device__ __forceinline__ void share_edges(const Share &s, const uint8_t *row, uint8_t *buf) {
  constexpr int es = Elem<DT>::kBytes, kN = Elem<DT>::kN;
  const int t = threadIdx.x;
  if (t < 2 * kN) {
    const int v = t < kN ? 0 : s.nvec - 1, e = t < kN ? t : t - kN;
    const int at = s.first + v * kN + e;
    const bool mine = at >= s.begin && at < s.end;
    uint8_t *to = buf + (size_t)v * 16 + e * es;
    if (DT == SPECDEC_F32)
      *reinterpret_cast<uint32_t *>(to) =
          mine ? reinterpret_cast<const uint32_t *>(row)[at] : 0xFF800000u;
    else
      *reinterpret_cast<uint16_t *>(to) =
          mine ? reinterpret_cast<const uint16_t *>(row)[at] : (uint16_t)0xFF80u;
  }
}

// Waits for copy i; a wait that gives up is noted.  Called by whole warps.
__device__ __forceinline__ void share_wait(Arrival &in, int i) {
  if (!mbar_wait_bounded(&in.full[i], 0, kConsumerWaitNs)) in.gave_up = 1;
}

// After a wait gave up: no copy may land in a CTA that has left.
__device__ __forceinline__ void share_drain(Arrival &in) {
  for (int i = 0; i < kChunks; ++i) mbar_wait_bounded(&in.full[i], 0);
}

// Writes a share held in shared memory (elements [begin, end) of the row, in the layout
// above) to a row whose alignment differs from the one it came from.
template <int DT, int kThreads>
__device__ __forceinline__ void store_unlike(const Share &s, const uint8_t *buf, uint8_t *row) {
  constexpr int es = Elem<DT>::kBytes, kN = Elem<DT>::kN;
  const int mis = (int)(reinterpret_cast<uintptr_t>(row) & 15);
  const int head = mis ? (16 - mis) / es : 0;
  // whole vectors of the row inside [begin, end): elements head + kN i
  const int i0 = s.begin <= head ? 0 : (s.begin - head + kN - 1) / kN;
  const int i1 = s.end <= head ? 0 : (s.end - head) / kN;
  const uint8_t *b = buf - (ptrdiff_t)s.first * es;
  for (int i = i0 + threadIdx.x; i < i1; i += kThreads) {
    const uint8_t *from = b + (ptrdiff_t)(head + kN * i) * es;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (DT == SPECDEC_F32)
        w[k] = reinterpret_cast<const uint32_t *>(from)[k];
      else
        w[k] = reinterpret_cast<const uint16_t *>(from)[2 * k] |
               (uint32_t)reinterpret_cast<const uint16_t *>(from)[2 * k + 1] << 16;
    }
    *reinterpret_cast<uint4 *>(row + (ptrdiff_t)(head + kN * i) * es) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
  // what is left at both ends (all of a share that holds no whole vector)
  const int a1 = i1 > i0 ? head + kN * i0 : s.end, b0 = i1 > i0 ? head + kN * i1 : s.end;
  const int na = a1 - s.begin, n = na + (s.end - b0);
  for (int t = threadIdx.x; t < n; t += kThreads) {
    const int at = t < na ? s.begin + t : b0 + (t - na);
    if (DT == SPECDEC_F32)
      reinterpret_cast<uint32_t *>(row)[at] =
          *reinterpret_cast<const uint32_t *>(b + (ptrdiff_t)at * es);
    else
      reinterpret_cast<uint16_t *>(row)[at] =
          *reinterpret_cast<const uint16_t *>(b + (ptrdiff_t)at * es);
  }
}

// Vector v of a share to a row aligned like the one that it came from: whole, or the
// elements of it that are the share's.
template <int DT>
__device__ __forceinline__ void store_like(const Share &s, uint8_t *row, int v, const uint4 &w) {
  constexpr int es = Elem<DT>::kBytes, kN = Elem<DT>::kN;
  const int at = s.first + v * kN;
  if (v > 0 && v <= s.body) {
    *reinterpret_cast<uint4 *>(row + (ptrdiff_t)at * es) = w;
    return;
  }
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < kN; ++e) {
    if (at + e < s.begin || at + e >= s.end) continue;
    if (DT == SPECDEC_F32)
      reinterpret_cast<uint32_t *>(row)[at + e] = a[e];
    else
      reinterpret_cast<uint16_t *>(row)[at + e] = (uint16_t)(a[e >> 1] >> (16 * (e & 1)));
  }
}

// How many CTAs hold a row: the fewest whose shares are small enough for several of them
// an SM (`per_sm`, which hides one CTA's waits behind another's work), more where the rows
// leave SMs idle, none with less than 4 KB to do.  Measured with shares other than the
// callers' (rows of 128256 bfloat16, us):
//   sampling, 4 CTAs a row and 2 an SM: 122 / 207 / 560 for 256 rows under top-p, 672 rows
//     without a filter, 2304 flat rows under top-p; 6 and 3: 163 / 252 / 821; 8 and 3: 151 /
//     240 / 819 (every CTA of a row has the same exchanges to wait for, and fewer registers).
//     float32, 256 rows under top-p and without a filter, 8 and 2: 218 / 115; 12 and 3: 340 /
//     142; 16 and 3: 440 / 149
//   distillation (before its loss was held in pairs), 4 a row and 3 an SM: 434 for 4096 rows;
//     5, 6 and 8 a row with 4 to 5 an SM: 463 to 500.  508 rows of 152064 float32: 138 with 10 a
//     row and 3 an SM, 154 with 8 and 2, 152 with 12 and 4, 208 with 16 and 5
inline int cluster_for(long long rows, int V, int elem_bytes, int share_bytes, int per_sm) {
  int c = 1;
  while (c < kMaxCluster && (long long)V * elem_bytes > (long long)c * share_bytes)
    c += c < 8 ? 1 : 2;
  const long long slots = (long long)device_sm_count() * per_sm;
  while (c * 2 <= kMaxCluster && rows * c * 2 <= slots && (long long)V * elem_bytes > c * 8192ll) c *= 2;
  return c;
}

// A launch of `rows` clusters of `size` CTAs, after the kernel before it on the stream.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_clusters(void (*kernel)(KArgs...), long long rows, int size, int threads,
                                   int smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * size));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)size;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The opt-in to clusters of 16 and to shared memory, once per device.
template <typename K>
inline cudaError_t cluster_opt_in_once(DeviceOnce &o, K kernel, int bytes) {
  return device_once(o, [&](int) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e != cudaSuccess
               ? e
               : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
}

#endif  // __CUDACC__

}  // namespace specdec
