// Attention of drafted tokens over the 8-bit cache on the tensor cores
// (specdec_attend, bfloat16 activations, heads of at most 128 elements).
//
// Per request, k/v head and up to RN rows (node n, query head g of the group),
// tiles of 128 tokens go through
//     S^T = K Q^T          [128 tokens, rows]     tcgen05.mma, e4m3
//     P^T = 2^(S^T - m)    by one thread per token and group of rows
//     O^T += V^T P^T       [128 elements, rows]   tcgen05.mma, fp16
// with m a running maximum per row.  Tokens stand on the 128 lanes of the
// accumulators and rows on their columns, so that a product costs what its
// rows need, and the same tile serves one token of G = 4 heads and a tree's 64
// nodes.
//
//   * K goes from the cache into the products as it is, e4m3.  A bfloat16 q has
//     8 significant bits: scaled by a power of two per row it is the sum of two
//     e4m3 values of 4 bits each, exactly for elements above 2^-9 of the row's largest;
//     below, to 2^-17 of that, half of e4m3's smallest step: less than what a bfloat16 q
//     has lost at its larger elements already.  Two products with K give q k^T.
//   * V widens to fp16 exactly, in shared memory, four warps' work; P is fp16
//     around 2^6 (11 bits, down to 2^-20 of the largest).  P in e4m3 would lose
//     the many small weights under one large one.
//   * the drafted tokens' own k and v are one more kind of tile: k in two e4m3
//     terms as q, v in fp16, each scaled by a power of two per node.
//   * m moves only when a score passes it by 2^8: weights are made under m as it
//     is and looked at on the way; in the rare case they are taken back from the
//     sums, m moves, and they are made again before the products read them.
//   * scores and each thread's sums stay in tensor memory, and all loops over rows
//     are rolled, 8 at a time: all roles share an SM's instruction cache, and what
//     does not fit it costs most.  Unrolled, with both in registers, 256 requests
//     of 9 nodes over 4096 tokens took 583 us, rolled 473; loops over 16 rows in
//     place of 8 cost 11 % more.
//   * V's units (block scales, or a drafted token's power of two), u = 2^k f with f in
//     [1, 2), ride on P.  P's fp16 range has to fit what a row sees and nothing else, so
//     the running maximum m of a row is that of s' + k, of what its tokens put into the
//     outputs: a token that a row does not see, or sees with next to no weight, leaves
//     the row alone whatever its size.  The sum of the weights under such an m is far
//     from 1, which float32 has room for: units from 2^-58 up (v from about 2^-48) keep
//     all bits, smaller ones (as after scores whose v is 0, weights below 2^-80 of
//     theirs) fewer in a row that sees nothing larger.
//
// A persistent grid.  All tiles of all requests, heads and row tiles form one
// line that is cut into equal parts, one per CTA, from the lengths on the device:
// any mix of lengths keeps all SMs busy to the end.  What a cut divides is joined
// by a second kernel, in order.  Up to 64 rows an SM holds two CTAs: one's
// beginnings and ends of requests, which are chains of short steps, overlap the
// other's tiles.  With 128 rows one CTA takes the whole SM, and four groups of
// warps a quarter of the rows each (two groups took 9 % more for 32 trees of 64
// nodes over 4096 tokens with a cap).
// Roles: warp 0 copies (TMA), warp 1 issues products, warps 4-7 widen V, stage q
// and build drafted tiles, the others take the softmax and write results.  A
// request's drafted tiles come first: they are built while the results of the
// request before are written.  Every wait is bounded in time.
//
// Measured (128 elements a head, 8 heads of k and v, G = 4): 256 requests of 9
// nodes over 4096 tokens 379 us, 3.0 TB/s; 64 of 6 95 us, 2.9 TB/s; one of 5 over
// 131071 81 us, 3.3 TB/s; 32 trees of 64 over 4096 with a cap 297 us.  Neither HBM
// (44 %) nor the tensor cores (busy 26 % of the time) bound it but the steps
// between: a tile's scores, softmax and products are a chain of about 3300 clocks, of
// which an SM holds two.
#include <cstddef>

#include <cuda.h>

#include "attention_common.cuh"

namespace specdec {
namespace {

constexpr int kTok = 128;
constexpr int kRow = 128;              // bytes of a shared-memory row: one swizzle span
constexpr int kTileBytes = kTok * kRow;
constexpr int kMaxSms = 160;
constexpr uint32_t kWaitClocks = 2000000000u;
constexpr float kRaise = 8.0f;
constexpr float kLift = 6.0f;
constexpr float kMost = 15.0f;  // P's exponent is cut off there, until the maxima move
constexpr float kUnit = 0x1p30f;       // of the outputs
// Least exponent of a token's unit in those, for the maxima: weights of up to 2^(15 + 88),
// and the sum of 2^24 of them inside float32.
constexpr float kLeast = -88.0f;
constexpr float kUnseen = 1e30f;       // minus the maximum of a row that has seen nothing
constexpr unsigned kAll = 0xffffffffu;

template <int RN>
struct Cfg {
  static constexpr int kCtas = RN <= 64 ? 2 : 1;       // CTAs an SM
  static constexpr int kGroups = RN <= 64 ? 1 : 4;     // softmax groups of four warps: a part of the rows each
  static constexpr int kWorkers = 4;                   // warps that widen V: one on each quarter of the SM
  static constexpr int kFirst = 8;                     // first softmax warp
  // Registers a thread: of the launch (what two CTAs, or one, leave room for), and
  // of the three kinds of warpgroup, which share out those of the launch:
  // kIssue + kWiden + kGroups kSoft = (2 + kGroups) kRegs
  static constexpr int kRegs = 80;
  static constexpr int kIssue = 64, kWiden = 64;
  static constexpr int kSoft = RN <= 64 ? 112 : 88;
  static_assert(kIssue + kWiden + kGroups * kSoft == (2 + kGroups) * kRegs, "");
  static constexpr int kThreads = 32 * (kFirst + 4 * kGroups);
  static constexpr int kCols = RN / kGroups;           // most columns of a softmax thread
  static constexpr int kK = RN <= 64 ? 1 : 2;          // stages of K codes (free once scores are made)
  static constexpr int kV = RN <= 48 ? 3 : 2;          // half tiles of V codes (free once widened)
  static constexpr int kBuf = RN <= 64 ? 1 : 2;        // buffers of widened V, and of P^T
  static constexpr int kTmem = RN == 32 ? 128 : RN <= 64 ? 256 : 512;
  static constexpr int kSpans = RN <= 64 ? 1 : 2;      // 64-row groups of P^T
};

// one CTA's part of the line of tiles
struct Plan {
  int b, off;       // first request, first tile of it
  long long count;  // the end's, b << 32 | off
};

// (Out of line: one copy of a 64-bit division.  The kernels' code has to stay
// small, as all roles' loops share an SM's instruction cache.)
__device__ __noinline__ long long divide(long long a, long long b) { return a / b; }

struct Request {
  int len, nodes, from;  // cached tokens, drafted ones, first token that the window leaves
  int drafted, tiles;    // tiles of drafted tokens, and in all
  int bad;
};

// A run of tiles of one unit (request, head, row tile).
struct Segment {
  int b, h, rt, t0, t1;  // b < 0: the end
  Request r;
  int whole;
};

template <int RN>
struct Smem {
  using C = Cfg<RN>;
  uint8_t k[C::kK][kTileBytes];           // K codes [token][128 B], 128-byte swizzle
  uint8_t v[C::kV][kTileBytes / 2];       // V codes, the same, 64 tokens each
  uint8_t vh[C::kBuf][2][kTileBytes];     // V in fp16, [64 elements][token][128 B]
  // P^T in fp16, [64 rows][token][128 B]; before a drafted tile's, the low terms of its k
  uint8_t pt[C::kBuf][C::kSpans][kTileBytes];
  uint8_t q[2][RN * kRow];                // q: high and low terms [row][128 B]
  float2 boxes[8][8];                     // k and v scales of a tile's pieces
  float2 unit[2][kTok];                   // drafted tiles: per token (k below 0: it is not finite)
  alignas(16) uint32_t see[2][4][RN];     // drafted tiles: bits of the nodes that a row sees
  // of the rows of four segments: the next one's are staged while the results of the
  // one three before may still be written
  alignas(16) float rf[4][RN];            // what turns a product into base-2 units
  float slope[4][RN], depth[4][RN];       // of the bias by distance; position from the length
  // per softmax group, by column
  alignas(16) float nm[C::kGroups][C::kCols];      // kLift - m, m of scores and units
  // the square root of l's and O's factor when m moves (at the end: addresses, 8 bytes each)
  alignas(16) float fac[C::kGroups][2][C::kCols];
  alignas(16) float red[C::kGroups][4][C::kCols];
  alignas(16) float ones[C::kCols];
  int vote[C::kGroups][4];
  uint32_t moves[C::kGroups];             // waits of the products on `again`
  Segment seg[8];
  int bad[8], dirty[8];
  uint64_t seg_full[8], box_full[8];
  uint64_t k_full[C::kK], k_empty[C::kK], v_full[C::kV], v_empty[C::kV], q_full, q_empty;
  uint64_t s_full[2], s_empty[2], p_full[C::kBuf], vh_full[C::kBuf], pv_done[C::kBuf];
  uint64_t group[C::kGroups], again[C::kGroups], both, fin;
  uint32_t tmem;
  int give_up;
  int done[C::kGroups];                   // segments that a softmax group finished
  long long scan[32];                     // of the plan: one a warp
  Plan plan;
};

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------
__device__ __forceinline__ void prefetch_l2(const void *at) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
}
__device__ __forceinline__ void tma_rows(void *dst, const CUtensorMap *map, int row, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(0), "r"(row), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}
template <bool kF8>
__device__ __forceinline__ void mma_issue(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          bool add) {
  if (kF8)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// Shared-memory operand, 128-byte swizzle.  group: bytes between groups of 8
// rows; span: bytes between 64-element groups of an operand whose rows run
// along the inner dimension.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t group, uint32_t span) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(span >> 4) << 16 |
         (uint64_t)(group >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// float32 accumulators, M = 128, N = n; `outer`: both operands have their outer
// dimension contiguous
__device__ __forceinline__ uint32_t shape(int n, bool outer) {
  return 1u << 4 | (outer ? 3u << 15 : 0u) | (uint32_t)(n >> 3) << 17 | 8u << 24;
}
__device__ __forceinline__ void tmem_load8(uint32_t at, float *x) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "r"(at));
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r[i]);
}
// The wait names the registers, so that nothing reads them before it.
__device__ __forceinline__ void tmem_wait8(float *x) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]),
                 "+f"(x[6]), "+f"(x[7]));
}
__device__ __forceinline__ void tmem_store8(uint32_t at, const float *x) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at),
               "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]),
               "f"(x[7])
               : "memory");
}
__device__ __forceinline__ void tmem_load4(uint32_t at, float *x) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ float tmem_load1(uint32_t at) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r)
               : "r"(at)
               : "memory");
  return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_store1(uint32_t at, float x) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(at), "f"(x) : "memory");
}
__device__ __forceinline__ void tmem_stored() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void store_global16(bool here, unsigned long long at, uint32_t x) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b16 t;\n\tsetp.ne.u32 p, %0, 0;\n\tcvt.u16.u32 t, %2;\n\t"
      "@p st.global.u16 [%1], t;\n\t}" ::"r"((uint32_t)here),
      "l"(at), "r"(x)
      : "memory");
}
__device__ __forceinline__ void store_global32(bool here, unsigned long long at, float x) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p st.global.f32 [%1], %2;\n\t}" ::"r"(
                   (uint32_t)here),
               "l"(at), "f"(x)
               : "memory");
}

__device__ __forceinline__ float min_nan(float a, float b) {  // NaN if one is
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

using f2 = unsigned long long;  // two float32 values in one register pair
__device__ __forceinline__ f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(f2 v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// 2^k, k in [-126, 127].
__device__ __forceinline__ float pow2i(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }
// floor(log2(u)), at least kLeast, for u >= 0.
__device__ __forceinline__ float exponent_of(float u) {
  return fmaxf((float)((int)(__float_as_uint(u) >> 23) - 127), kLeast);
}
// k with top / 2^k in [2^at, 2^(at + 1)), inside the range of pow2i(+-k)
__device__ __forceinline__ int unit_exponent(float top, int at) {
  return min(max((int)(__float_as_uint(top) >> 23) - 127 - at, -126), 126);
}

// ---------------------------------------------------------------------------
// the line of tiles
// ---------------------------------------------------------------------------
__device__ __noinline__ Request request_of(const AttendParams &p, int b, int box) {
  Request r;
  r.bad = 0;
  r.len = p.cache.length[b];
  r.nodes = p.n_nodes ? p.n_nodes[b] : p.N;
  if (r.len < 0 || (long long)r.len > (long long)p.cache.max_blocks * p.cache.block)
    r.bad = SPECDEC_ROW_BAD_CACHE;
  if (r.nodes < 0 || r.nodes > p.N) r.bad |= SPECDEC_ROW_BAD_TREE;
  if (r.bad) r.len = r.nodes = 0;
  r.from = p.window > 0 ? max(0, r.len - p.window + 1) / box * box : 0;
  // a request without tokens still has its rows to write
  r.drafted = max(1, (r.nodes + kTok - 1) / kTok);
  r.tiles = r.drafted + (r.nodes > 0 ? (r.len - r.from + kTok - 1) / kTok : 0);
  return r;
}

// What a segment costs beside its tiles, in tiles: q, the first maxima, results.
constexpr int kExtra = 4;

// The part of CTA `i` of `n`; all threads of the CTA, `scan` shared.  The line is
// measured in costs: each unit its tiles and kExtra, which stands before them.
__device__ __forceinline__ Plan make_plan(const AttendParams &p, int box, int i, int n,
                                          long long *scan, Plan *shared) {
  const int t = threadIdx.x, threads = blockDim.x;
  const int units = p.cache.Hkv * p.row_tiles;
  const int per = (p.B + threads - 1) / threads;
  long long mine = 0;
#pragma unroll 1
  for (int b = t * per; b < min(p.B, (t + 1) * per); ++b)
    mine += (long long)(request_of(p, b, box).tiles + kExtra) * units;
  long long upto = mine;  // inclusive scan
#pragma unroll 1
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(kAll, upto, d);
    if ((t & 31) >= d) upto += o;
  }
  if ((t & 31) == 31) scan[t >> 5] = upto;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll 1
  for (int w = 0; w < threads / 32; ++w) {
    if (w < (t >> 5)) before += scan[w];
    total += scan[w];
  }
  upto += before;
  // the tiles from the first cut to the second; a cut is found by the thread
  // whose requests it falls among
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const long long cut = divide(total * (i + side), n);
    if (cut >= upto - mine && (cut < upto || (cut == total && upto == total && mine > 0))) {
      long long at = upto - mine;
      int b = t * per, off = 0;
#pragma unroll 1
      for (;; ++b) {
        const int each = request_of(p, b, box).tiles + kExtra;
        const long long here = (long long)each * units;
        if (cut < at + here || b == min(p.B, (t + 1) * per) - 1) {
          const int in = (int)min(cut - at, here), unit = in / each;
          off = unit * (each - kExtra) + max(0, in - unit * each - kExtra);
          break;
        }
        at += here;
      }
      if (side == 0) {
        shared->b = b;
        shared->off = off;
      } else {
        shared->count = ((long long)b << 32) | (uint32_t)off;  // the end's place, for now
      }
    }
  }
  __syncthreads();
  return *shared;
}

// Segments of a CTA's part: runs of tiles of one unit (request, head, row tile).
// Warp 0 walks them and publishes each in shared memory for the other roles.
struct Walk {
  int b, off, end_b, end_off;
  Request r;

  __device__ Walk(const AttendParams &p, int box, const Plan &plan)
      : b(plan.b), off(plan.off), end_b((int)(plan.count >> 32)), end_off((int)plan.count) {
    r = request_of(p, b, box);
  }
  __device__ __forceinline__ bool next(const AttendParams &p, int box, Segment &s) {
    s.b = -1;
    const int units = p.cache.Hkv * p.row_tiles;
    if (off >= r.tiles * units && b < end_b) {
      ++b;
      off = 0;
      r = request_of(p, b, box);
    }
    const int last = b < end_b ? r.tiles * units : end_off;
    if (off >= last) return false;
    const int unit = off / r.tiles;
    s.b = b;
    s.t0 = off - unit * r.tiles;
    s.h = unit / p.row_tiles;
    s.rt = unit - s.h * p.row_tiles;
    s.t1 = min(r.tiles, s.t0 + last - off);
    s.r = r;
    s.whole = s.t0 == 0 && s.t1 == r.tiles;
    off += s.t1 - s.t0;
    return true;
  }
};

// What the join has to know of a CTA's part.
struct Note {
  int tiles;        // of the part
  int first, head;  // its first segment: where in its unit, and how many tiles
  int unit;         // that unit's tiles, and which it is
  int b, h, rt;
  int open;         // tiles done of a unit that was begun but not ended here, or 0
  int lost, lost_to;  // requests of the segments that were given up, or -1
};

// Waits until the phase of `parity` is complete.  Gives up after kWaitClocks, about a
// second, where no wait of a working kernel takes a tenth of that (the longest are for
// rows that see values that are not finite, `stray` below: tens of ms at 1024 nodes), and
// says so in shared memory at `give_up`.  (A 64-bit timer, or a look at `give_up` on the
// way, are more code at each wait: 7 to 10 % more time for the 256 requests above.)
__device__ __forceinline__ bool wait_lane(uint32_t bar, uint32_t parity, uint32_t give_up) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 t0, t;\n\t"
      "mov.u32 t0, %%clock;\n\t"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 2000;\n\t"
      "@p bra DONE;\n\t"
      "mov.u32 t, %%clock;\n\t"
      "sub.u32 t, t, t0;\n\t"
      "setp.lt.u32 q, t, %4;\n\t"
      "@q bra AGAIN;\n\t"
      "st.volatile.shared.u32 [%3], 1;\n\t"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(give_up), "n"(kWaitClocks)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {  // of unsigned 16-bit halves
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t half2_to_e4m3x2(uint32_t h) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f16x2 t, %1;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(r)
      : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t sub_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The largest finite size (bfloat16 bits) among the 16 lanes of a row.
__device__ __noinline__ uint32_t finite_top(uint4 w) {
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
  uint32_t m = 0;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const uint32_t x = (i < 2 ? a[0] : i < 4 ? a[1] : i < 6 ? a[2] : a[3]) >> (16 * (i & 1)) & 0x7FFFu;
    if (x < 0x7F80u) m = max(m, x);
  }
#pragma unroll 1
  for (int d = 8; d >= 1; d >>= 1) m = max(m, __shfl_xor_sync(kAll, m, d));
  return m;
}

// 8 bfloat16 values from an address that is not a multiple of 16 bytes
__device__ __noinline__ uint4 load8_narrow(const unsigned short *s) {
  uint32_t a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = (uint32_t)__ldg(s + 2 * i) | (uint32_t)__ldg(s + 2 * i + 1) << 16;
  return make_uint4(a[0], a[1], a[2], a[3]);
}

// Whether a window hides part of cached tile t from some row.
__device__ __forceinline__ bool partly_hidden(const AttendParams &p, const Request &r, int t) {
  return p.window > 0 && r.from + (t - r.drafted) * kTok <= r.len + p.N - 1 - p.window;
}

// A partial: for each row m, l, then its D elements; flags as l < 0.
__host__ __device__ inline size_t partial_floats(int RN, int D) { return (size_t)RN * (D + 2); }
// Two slots a CTA: what it did of a unit begun before, and of one that it began.
// Behind them the notes.
__device__ __forceinline__ Note *notes_of(float *part, int RN, int D) {
  return reinterpret_cast<Note *>(part + 4 * kMaxSms * partial_floats(RN, D));
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <int RN, bool kPlain>
struct Tile {
  using S = Smem<RN>;
  using C = Cfg<RN>;
  static constexpr int kK = C::kK, kV = C::kV, kBuf = C::kBuf;
  const AttendParams &p;
  S &sm;
  const CUtensorMap *k_map, *v_map;
  const int box, lane, warp;
  const int box_shift;
  const uint32_t g_magic;  // ceil(2^32 / G): row / G for rows below 2^32 / G
  int columns;  // rows of a tile, a multiple of 16

  __device__ Tile(const AttendParams &p_, S &s_, const CUtensorMap *k_, const CUtensorMap *v_,
                  int box_)
      : p(p_), sm(s_), k_map(k_), v_map(v_), box(box_), lane(threadIdx.x & 31),
        warp(threadIdx.x >> 5), box_shift(box_ == 128 ? 7 : box_ == 64 ? 6 : box_ == 32 ? 5 : 4),
        g_magic((uint32_t)(0xFFFFFFFFu / (uint32_t)p_.G) + 1u) {
    columns = (min(RN, p.N * p.G) + 15) / 16 * 16;
    if (!kPlain) {
      // (finite, so that a score of 0 stays 0 under the smallest caps)
      cap_in = p.softcap > 0.0f ? fminf(2.0f / p.softcap, 3.4e38f) : 0.0f;
      cap_at = p.softcap * kLog2e;
      cap_out = -2.0f * cap_at;
    }
  }

  // Bounded wait of a whole warp; false when it, or another, gave up.
  __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(kAll, wait_lane(smem_addr(bar), parity, smem_addr(&sm.give_up)));
  }
  // Slot and parities of tile c in a ring of n: full is waited on with the
  // first, empty (of the slot's last use) with the second.
  static __device__ __forceinline__ uint32_t full_par(uint32_t c, int n) { return (c / n) & 1; }
  static __device__ __forceinline__ uint32_t empty_par(uint32_t c, int n) { return ((c / n) & 1) ^ 1; }

  // Segment i, published by warp 0 (a ring of eight is enough, since it is at
  // most seven ahead of the softmax); false at the end or on giving up.
  __device__ __forceinline__ bool segment(uint32_t i, bool &ok) {
    ok = wait(&sm.seg_full[i & 7], (i >> 3) & 1);
    return ok && sm.seg[i & 7].b >= 0;
  }

  // ------------------------------------------------------------ warp 0: copies
  // A lane's piece of a tile: its block id in flight.
  struct Piece {
    int id, tok;
    bool mine;
  };
  __device__ __forceinline__ Piece piece_of(const Segment &w, int t) const {
    const specdec_kv_cache &kv = p.cache;
    Piece x;
    x.tok = w.r.from + (t - w.r.drafted) * kTok + lane * box;
    x.mine = t >= w.r.drafted && lane * box < kTok && x.tok < w.r.len;
    x.id = x.mine ? __ldg(kv.block_table + (long long)w.b * kv.max_blocks + x.tok / kv.block) : 0;
    return x;
  }
  Note note;
  __device__ __forceinline__ bool take(Walk &walk, Segment &w) {
    const bool more = walk.next(p, box, w);
    if (more) {
      if (note.tiles == 0) {
        note.first = w.t0;
        note.head = w.t1 - w.t0;
        note.unit = w.r.tiles;
        note.b = w.b;
        note.h = w.h;
        note.rt = w.rt;
      }
      note.tiles += w.t1 - w.t0;
      note.open = w.t0 == 0 && !w.whole ? w.t1 : 0;
    }
    return more;
  }
  // The rows that the others read next, towards the L2.
  __device__ __forceinline__ void fetch(const Segment &w) const {
    const long long first = (long long)w.b * p.N;
    const int D = p.cache.D;
#pragma unroll 1
    for (int n = lane; n < w.r.nodes; n += 32) {
      const char *q = reinterpret_cast<const char *>(p.q) + ((first + n) * p.q_stride + w.h * p.G * D) * 2;
#pragma unroll 1
      for (int i = 0; i < p.G * D * 2; i += 128) prefetch_l2(q + i);
      if (w.t0 < w.r.drafted) {
        prefetch_l2(reinterpret_cast<const char *>(p.k_new) + ((first + n) * p.k_stride + w.h * D) * 2);
        prefetch_l2(reinterpret_cast<const char *>(p.v_new) + ((first + n) * p.v_stride + w.h * D) * 2);
      }
    }
  }
  __device__ __forceinline__ bool publish(Walk &walk, uint32_t index, Segment &w) {
    const bool more = take(walk, w);
    if (more) fetch(w);
    if (lane == 0) {
      sm.seg[index & 7] = w;
      mbar_arrive(&sm.seg_full[index & 7]);
    }
    return more;
  }

  __device__ __forceinline__ void copies(const Plan &plan) {
    const specdec_kv_cache &kv = p.cache;
    uint32_t c = 0, v = 0, index = 0;  // tiles; half tiles of V
    note.tiles = note.first = note.head = note.open = 0;
    note.lost = note.lost_to = -1;
    copied = copied_v = 0;
    Walk walk(p, box, plan);
    Segment w, ahead;
    bool ok = true, more = true;
    // each segment is published one ahead, so that the others prepare it
#pragma unroll 1
    for (;; ++index) {
      w = ahead;
      const bool have = index > 0 && more;
      if (more) more = publish(walk, index, ahead);
      if (index == 0) continue;
      if (!have) break;
      Piece next = piece_of(w, w.t0);
#pragma unroll 1
      for (int t = w.t0; t < w.t1; ++t, ++c) {
        const int ks = c % kK;
        Piece x = next;
        if (t + 1 < w.t1) next = piece_of(w, t + 1);  // the next tile's ids load meanwhile
        const bool cached = t >= w.r.drafted;
        if (x.id < 0 || x.id >= kv.n_blocks) {
          x.id = 0;
          atomicOr(&sm.bad[(index - 1) & 7], SPECDEC_ROW_BAD_CACHE);  // (or BAD_TREE stands there)
        }
        const long long cell = (long long)x.id * kv.Hkv + w.h;
        const int row = (int)(cell * kv.block + x.tok % kv.block);
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(kAll, x.mine)) * box * kRow;
        float2 unit = make_float2(0.0f, 0.0f);
        if (x.mine) unit = make_float2(__ldg(kv.k_scale + cell), __ldg(kv.v_scale + cell));
        if (!(ok = wait(&sm.k_empty[ks], empty_par(c, kK)))) break;
        // Drafted tiles have nothing to copy, but their products wait for this
        // arrival: were they done before the wait above looks, it would miss their
        // phase and take the next one of the same parity for it.
        copied = c + 1;
        if (!cached) {
          if (lane == 0) mbar_arrive(&sm.k_full[ks]);
          __syncwarp();
          continue;
        }
        if (lane == 0) mbar_arrive_expect_tx(&sm.k_full[ks], bytes);
        __syncwarp();
        if (x.mine) {
          tma_rows(sm.k[ks] + lane * box * kRow, k_map, row, &sm.k_full[ks]);
          sm.boxes[c & 7][lane] = unit;
        }
        __syncwarp();
        if (lane < 4) mbar_arrive(&sm.box_full[c & 7]);
#pragma unroll
        for (int half = 0; half < 2; ++half, ++v) {
          if (!(ok = wait(&sm.v_empty[v % kV], empty_par(v, kV)))) break;
          const bool here = x.mine && (lane * box >= kTok / 2) == (half == 1);
          const uint32_t n = (uint32_t)__popc(__ballot_sync(kAll, here)) * box * kRow;
          if (lane == 0) mbar_arrive_expect_tx(&sm.v_full[v % kV], n);
          __syncwarp();
          if (here)
            tma_rows(sm.v[v % kV] + (lane * box - half * (kTok / 2)) * kRow, v_map, row,
                     &sm.v_full[v % kV]);
          copied_v = v + 1;
        }
        if (!ok) break;
      }
      if (!ok) break;
    }
    // After giving up only the notes go on: no further segment is published, as its
    // place in the ring may still be read.
    while (more) more = take(walk, ahead);
    if (lane == 0) notes_of(p.part, RN, kv.D)[blockIdx.x] = note;
  }

  // Every copy has been waited on by its reader, unless somebody gave up: then copies in
  // flight get time to land before the CTA may leave.
  uint32_t copied, copied_v;  // of K and of V: issued, on barriers of their own order
  __device__ void drain() {
    for (uint32_t i = copied > kK ? copied - kK : 0; i < copied; ++i)
      mbar_wait_bounded(&sm.k_full[i % kK], full_par(i, kK));
    for (uint32_t i = copied_v > kV ? copied_v - kV : 0; i < copied_v; ++i)
      mbar_wait_bounded(&sm.v_full[i % kV], full_par(i, kV));
  }

  // ------------------------------------------------------------ warp 1: products
  __device__ __forceinline__ void scores(uint32_t c, bool drafted, bool ends) {
    if (elected()) {
      const uint32_t d = sm_tmem + (c & 1) * RN, idesc = shape(columns, false);
      const int steps = (p.cache.D + 31) / 32;
      // 32 elements a step: 32 bytes, 2 units of the descriptor's address
      const uint64_t ka = operand(smem_addr(sm.k[c % kK]), 1024, 16);
      const uint64_t qa = operand(smem_addr(sm.q[0]), 1024, 16);
      const uint64_t qb = operand(smem_addr(sm.q[1]), 1024, 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= steps) continue;
        mma_issue<true>(d, ka + 2 * i, qa + 2 * i, idesc, i > 0);
        mma_issue<true>(d, ka + 2 * i, qb + 2 * i, idesc, true);
      }
      if (drafted) {
        const uint64_t kl = operand(smem_addr(sm.pt[c % kBuf][0]), 1024, 16);
#pragma unroll 1
        for (int i = 0; i < steps; ++i) {
          mma_issue<true>(d, kl + 2 * i, qa + 2 * i, idesc, true);
          mma_issue<true>(d, kl + 2 * i, qb + 2 * i, idesc, true);
        }
      }
      mma_commit(&sm.s_full[c & 1]);
      mma_commit(&sm.k_empty[c % kK]);
      if (ends) mma_commit(&sm.q_empty);
    }
    __syncwarp();
  }

  // The test build in which waits give up without looking (see common.cuh): here for the
  // copies of every second CTA, of all its segments or from the second one on.
  __device__ __forceinline__ bool gives_up(uint32_t index) const {
    if (kConsumerWaitNs != 0 || blockIdx.x % 2 == 0) return false;
    if (blockIdx.x % 4 == 1 && index == 0) return false;
    *(volatile int *)&sm.give_up = 1;
    return true;
  }

  // O^T += V^T P^T of tile c, as soon as both are there.  (Inline, and what runs in rare
  // cases last in this class: functions stand behind the kernel's body in this order, so
  // that the size of the rare ones does not shift what runs at every tile within the
  // instruction cache, which is worth up to 10 % either way.)
  __device__ __forceinline__ bool outputs(uint32_t c, bool first) {
    const uint32_t d = sm_tmem + 2 * RN;
    const uint32_t give_up = smem_addr(&sm.give_up);
    if (!__all_sync(kAll, wait_lane(smem_addr(&sm.vh_full[c % kBuf]), full_par(c, kBuf), give_up) &&
                              wait_lane(smem_addr(&sm.p_full[c % kBuf]), full_par(c, kBuf), give_up)))
      return false;
    // a group whose maxima move writes its weights again
#pragma unroll 1
    for (int g = 0; g < C::kGroups; ++g)
      if (*(volatile int *)&sm.vote[g][c & 3]) {
        const uint32_t parity = *(volatile uint32_t *)&sm.moves[g] & 1;
        if (!__all_sync(kAll, wait_lane(smem_addr(&sm.again[g]), parity, give_up))) return false;
        if (elected()) sm.moves[g] += 1;
        __syncwarp();
      }
    fence_after();
    if (elected()) {
      const uint32_t idesc = shape(columns, true);
      const uint64_t va = operand(smem_addr(sm.vh[c % kBuf][0]), 1024, kTileBytes);
      const uint64_t pb = operand(smem_addr(sm.pt[c % kBuf][0]), 1024, kTileBytes);
#pragma unroll
      for (int i = 0; i < kTok / 16; ++i)  // 16 tokens a step: 2048 bytes
        mma_issue<false>(d, va + 128 * i, pb + 128 * i, idesc, !first || i > 0);
      mma_commit(&sm.pv_done[c % kBuf]);
    }
    __syncwarp();
    return true;
  }

  uint32_t sm_tmem;
  __device__ __forceinline__ void products() {
    uint32_t c = 0;
    bool ok = true, pending = false, pending_first = false;  // outputs of tile c - 1
    sm_tmem = sm.tmem;
#pragma unroll 1
    for (uint32_t index = 0; segment(index, ok); ++index) {
      const int t0 = sm.seg[index & 7].t0, t1 = sm.seg[index & 7].t1;
      const int drafts = sm.seg[index & 7].r.drafted;
#pragma unroll 1
      for (int t = t0; t < t1; ++t, ++c) {
        const bool drafted = t < drafts, first = t == t0;
        // Scores run a tile ahead of outputs; but at a segment's start, and before
        // a drafted tile that needs the room which they free, outputs come first.
        const bool flush = first || (kBuf == 1 && drafted);
        if (flush && pending) {
          if (!(ok = outputs(c - 1, pending_first))) break;
          pending = false;
        }
        if (first && !(ok = wait(&sm.q_full, index & 1))) break;
        if (!(ok = wait(&sm.box_full[c & 7], (c >> 3) & 1))) break;
        if (gives_up(index)) {
          ok = false;
          break;
        }
        if (!(ok = wait(&sm.k_full[c % kK], full_par(c, kK)))) break;
        if (!(ok = wait(&sm.s_empty[c & 1], ((c >> 1) & 1) ^ 1))) break;
        fence_after();
        scores(c, drafted, t == t1 - 1);
        if (pending && !(ok = outputs(c - 1, pending_first))) break;
        pending = true;
        pending_first = first;
      }
      if (!ok) break;
    }
    if (ok && pending) outputs(c - 1, pending_first);
    // products in flight end before the CTA may leave
    if (elected()) mma_commit(&sm.fin);
    __syncwarp();
    mbar_wait_bounded(&sm.fin, 0);
  }

  // ------------------------------------------------------------ warps 2-5: operands
  __device__ __forceinline__ int node_of(int row) const {  // row / G
    return p.G == 1 ? row : (int)__umulhi((uint32_t)row, g_magic);
  }
  // The node above a, -1 above a root; `first`: the request's first node.
  __device__ __forceinline__ int above(long long first, int a) const {
    if (!p.parent || a == 0) return a - 1;
    const int up = __ldg(p.parent + first + a);
    return up < a ? max(up, -1) : -1;
  }
  __device__ __forceinline__ int depth_of(int b, int n) const {
    if (!p.parent) return n;
    int depth = 0;
#pragma unroll 1
    for (int a = above((long long)b * p.N, n); a >= 0; a = above((long long)b * p.N, a)) ++depth;
    return depth;
  }

  // Rows are staged by 16 lanes each, 8 elements a lane, two rows a warp at once.
  // The lane's elements of a row, as packed bfloat16; `wide`: 16-byte aligned.
  __device__ __forceinline__ uint4 load8(const void *base, long long at, bool wide) const {
    const unsigned short *s = reinterpret_cast<const unsigned short *>(base) + at;
    return wide ? __ldg(reinterpret_cast<const uint4 *>(s)) : load8_narrow(s);
  }

  // The row's largest finite size, and whether all are finite.
  __device__ __forceinline__ float row_top(const uint4 &w, bool &all) const {
    uint32_t m = max2(max2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                      max2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
    m = max(m >> 16, m & 0xFFFFu);
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) m = max(m, __shfl_xor_sync(kAll, m, d));
    all = m < 0x7F80u;
    if (__any_sync(kAll, !all)) m = finite_top(w);
    return __uint_as_float(m << 16);
  }

  // The row in units of 2^ex as the sum of two e4m3 terms: 8 bytes of each at
  // element e of row r.  (In fp16 between: bfloat16's bits fit, and so does what
  // the first term leaves.)
  __device__ __forceinline__ void split(uint8_t *hi, uint8_t *lo, int r, int e, const uint4 &w,
                                        int ex) const {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
    const float inv = pow2i(-ex);
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = pack_half2(bf16_lo(a[i]) * inv, bf16_hi(a[i]) * inv);
      h[i] = half2_to_e4m3x2(x);
      l[i] = half2_to_e4m3x2(sub_half2(x, e4m3x2_to_half2(h[i])));
    }
    const int at = r * kRow + ((((e >> 4) ^ (r & 7)) << 4) | (e & 8));
    *reinterpret_cast<uint2 *>(hi + at) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    *reinterpret_cast<uint2 *>(lo + at) = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
  }

  __device__ __forceinline__ void stage_q(uint32_t index, int worker) {
    const Segment &w = sm.seg[index & 7];
    const int D = p.cache.D, ring = index & 3, e = (lane & 15) * 8;
    const int nodes = w.r.nodes, row0 = w.rt * RN;
    const bool wide = ((reinterpret_cast<uintptr_t>(p.q) | (uintptr_t)(p.q_stride * 2)) & 15) == 0;
    const long long first = (long long)w.b * p.N;
    constexpr int kStep = 2 * C::kWorkers;  // rows at once
    const int r0 = worker * 2 + (lane >> 4);
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    // a row is loaded while the one before is split
#pragma unroll 1
    for (int r = r0; r - (lane >> 4) < columns + kStep; r += kStep) {
      uint4 next = make_uint4(0u, 0u, 0u, 0u);
      {
        const int row = row0 + r, n = node_of(row);
        if (r < columns && row < p.N * p.G && n < nodes && e < D)
          next = load8(p.q, (first + n) * p.q_stride + (w.h * p.G + row - n * p.G) * D + e, wide);
      }
      if (r != r0) {
        const int col = r - kStep, row = row0 + col, n = node_of(row);
        bool all;
        const int ex = unit_exponent(row_top(x, all), 7);
        split(sm.q[0], sm.q[1], col, e, x, ex);
        if ((lane & 15) == 0) {
          const bool in = row < p.N * p.G && n < nodes;
          // a q that is not finite makes its row NaN
          const float unit = all ? pow2i(ex) : __int_as_float(0x7fc00000);
          const int depth = in && (p.window > 0 || p.slopes) ? depth_of(w.b, n) : 0;
          sm.rf[ring][col] = in ? p.scale * kLog2e * unit : 0.0f;
          sm.depth[ring][col] = (float)depth;
          if (!kPlain)
            sm.slope[ring][col] = in && p.slopes ? p.slopes[w.h * p.G + row - n * p.G] * kLog2e : 0.0f;
        }
        __syncwarp();
      }
      x = next;
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_full);
  }

  // NaN codes of a tile that a window hides in part: out of the products, as
  // they must not reach rows that do not see them (the results add them).
  __device__ __noinline__ static bool sift(uint8_t *codes, int tid) {
    bool odd = false;
#pragma unroll 1
    for (int i = tid >> 4; i < kTok / 2; i += 2 * C::kWorkers) {  // the thread's own pieces
      uint32_t *w = reinterpret_cast<uint32_t *>(codes + i * kRow +
                                                 ((((tid & 15) >> 1) ^ (i & 7)) << 4) + (tid & 1) * 8);
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        uint32_t keep = 0;
        for (int s = 0; s < 32; s += 8)
          if (((w[k] >> s) & 0x7Fu) != 0x7Fu) keep |= 0xFFu << s;
        odd |= keep != kAll;
        w[k] &= keep;
      }
    }
    return odd;
  }

  // Half a tile of V codes to fp16; tokens past the length as zeros.  A thread
  // takes 8 codes at a time, 16 lanes a token: 8 bytes in, 16 out, each half-warp
  // over all banks; all loads before the first store, which the compiler cannot
  // know to be elsewhere.
  __device__ __forceinline__ void widen(uint8_t *codes, uint8_t *vh, int held, int worker) {
    constexpr int kStep = 2 * C::kWorkers, kBatch = kTok / 2 / kStep;
    const int tid = worker * 32 + lane, h = tid & 15, tok0 = tid >> 4;
    const uint8_t *src = codes + (h & 1) * 8;
    uint8_t *dst = vh + (h >> 3) * kTileBytes;
    uint2 x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int tok = tok0 + i * kStep;
      x[i] = *reinterpret_cast<const uint2 *>(src + tok * kRow + (((h >> 1) ^ (tok & 7)) << 4));
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int tok = tok0 + i * kStep;
      if (tok >= held) x[i] = make_uint2(0u, 0u);
      *reinterpret_cast<uint4 *>(dst + tok * kRow + (((h & 7) ^ (tok & 7)) << 4)) =
          make_uint4(e4m3x2_to_half2(x[i].x), e4m3x2_to_half2(x[i].x >> 16),
                     e4m3x2_to_half2(x[i].y), e4m3x2_to_half2(x[i].y >> 16));
    }
  }

  // A tile of drafted tokens: nodes [j0, j0 + 128).
  __device__ __forceinline__ void build(const Segment &w, uint32_t index, int t, uint32_t c,
                                        int worker) {
    const int D = p.cache.D, j0 = t * kTok, e = (lane & 15) * 8;
    const int nodes = w.r.nodes, held = min(nodes - j0, kTok);
    const long long first = (long long)w.b * p.N;
    const bool k_wide =
        ((reinterpret_cast<uintptr_t>(p.k_new) | (uintptr_t)(p.k_stride * 2)) & 15) == 0;
    const bool v_wide =
        ((reinterpret_cast<uintptr_t>(p.v_new) | (uintptr_t)(p.v_stride * 2)) & 15) == 0;
#pragma unroll 1
    for (int r = worker * 2 + (lane >> 4); r - (lane >> 4) < held; r += 2 * C::kWorkers) {
      const bool in = r < held && e < D;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      const uint4 x = in ? load8(p.k_new, (first + j0 + r) * p.k_stride + (long long)w.h * D + e, k_wide)
                         : zero;
      const uint4 y = in ? load8(p.v_new, (first + j0 + r) * p.v_stride + (long long)w.h * D + e, v_wide)
                         : zero;
      bool all;
      const int ek = unit_exponent(row_top(x, all), 7);
      split(sm.k[c % kK], sm.pt[c % kBuf][0], r, e, x, ek);
      const float k_unit = all ? pow2i(ek) : -1.0f;
      const int ev = unit_exponent(row_top(y, all), 10);
      const float inv = pow2i(-ev);
      if (!all) sm.dirty[index & 7] = 1;
      const uint32_t b[4] = {y.x, y.y, y.z, y.w};
      uint32_t a[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v0 = bf16_lo(b[i]), v1 = bf16_hi(b[i]);
        a[i] = pack_half2(finite(v0) ? v0 * inv : 0.0f, finite(v1) ? v1 * inv : 0.0f);
      }
      *reinterpret_cast<uint4 *>(sm.vh[c % kBuf][e >> 6] + r * kRow +
                                 ((((e & 63) >> 3) ^ (r & 7)) << 4)) =
          make_uint4(a[0], a[1], a[2], a[3]);
      if ((lane & 15) == 0) sm.unit[c & 1][r] = make_float2(k_unit, pow2i(ev));
    }
    // past the last node: weights there are 0, but V must not be NaN
    const int tid = worker * 32 + lane;
#pragma unroll 1
    for (int i = max(held, 0) * 8 + tid; i < kTok * 8; i += 32 * C::kWorkers) {
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      reinterpret_cast<uint4 *>(sm.vh[c % kBuf][0])[i] = zero;
      reinterpret_cast<uint4 *>(sm.vh[c % kBuf][1])[i] = zero;
    }
    // what each row sees of this tile: its node's ancestors, as bits
#pragma unroll 1
    for (int col = tid; col < columns; col += 32 * C::kWorkers) {
      const int n = node_of(w.rt * RN + col);
      uint32_t bits[4] = {0u, 0u, 0u, 0u};
      if (n < nodes && !p.parent) {  // a chain: nodes lo .. n
        const int lo = max(p.window > 0 ? n - p.window + 1 : 0, j0) - j0, hi = min(n - j0, kTok - 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int a = max(lo - 32 * i, 0), z = min(hi - 32 * i, 31);
          bits[i] = z < a ? 0u : (kAll >> (31 - z)) & (kAll << a);
        }
      } else if (n < nodes) {
        int a = n;
#pragma unroll 1
        for (int step = 0; a >= j0; ++step) {
          if (a < j0 + kTok && (p.window == 0 || step < p.window)) {
            const uint32_t bit = 1u << ((a - j0) & 31);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((a - j0) >> 5 == i) bits[i] |= bit;
          }
          a = above(first, a);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sm.see[c & 1][i][col] = bits[i];
    }
    if (p.parent) {
      bool wrong = false;
#pragma unroll 1
      for (int i = tid; i < nodes; i += 32 * C::kWorkers) {
        const int up = __ldg(p.parent + first + i);
        wrong |= i == 0 ? up != -1 : (up < 0 || up >= i);
      }
      if (wrong) atomicOr(&sm.bad[index & 7], SPECDEC_ROW_BAD_TREE);
    }
  }

  __device__ __forceinline__ void operands() {
    const int worker = warp - 4;
    uint32_t c = 0, v = 0;
    bool ok = true;
#pragma unroll 1
    for (uint32_t index = 0; segment(index, ok); ++index) {
      const Segment &w = sm.seg[index & 7];
      const int t0 = w.t0, t1 = w.t1, drafts = w.r.drafted;
      if (!(ok = wait(&sm.q_empty, (index & 1) ^ 1))) break;
      stage_q(index, worker);
#pragma unroll 1
      for (int t = t0; t < t1; ++t, ++c) {
        const bool drafted = t < drafts;
        // room: outputs of the tile before in this buffer are done
        if (!(ok = wait(&sm.pv_done[c % kBuf], empty_par(c, kBuf)))) break;
        if (drafted) {
          if (!(ok = wait(&sm.k_empty[c % kK], empty_par(c, kK)))) break;
          build(w, index, t, c, worker);
        } else {
          const int held = w.r.len - (w.r.from + (t - drafts) * kTok);
#pragma unroll 1
          for (int half = 0; half < 2; ++half, ++v) {
            if (!(ok = wait(&sm.v_full[v % kV], full_par(v, kV)))) break;
            uint8_t *codes = sm.v[v % kV];
            if (partly_hidden(p, w.r, t) && sift(codes, worker * 32 + lane)) sm.dirty[index & 7] = 1;
            widen(codes, sm.vh[c % kBuf][0] + half * (kTileBytes / 2), held - half * (kTok / 2), worker);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.v_empty[v % kV]);
          }
          if (!ok) break;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.vh_full[c % kBuf]);
          if (drafted) mbar_arrive(&sm.box_full[c & 7]);
        }
      }
      if (!ok) break;
    }
  }

  // ------------------------------------------------------------ the last warps: softmax
  uint32_t group_phase, both_phase;
  // The four warps of one group: a warp's arrival, and the wait for all; and all
  // softmax warps.
  __device__ __forceinline__ void arrive(int group) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.group[group]);
  }
  __device__ __forceinline__ bool join(int group) {
    const bool ok = wait(&sm.group[group], group_phase);
    group_phase ^= 1;
    return ok;
  }
  __device__ __forceinline__ bool meet(int group) {
    arrive(group);
    return join(group);
  }
  __device__ __forceinline__ bool meet_all() {
    fence_before();
    bool ok;
    if (C::kGroups == 1) {
      ok = meet(0);
    } else {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.both);
      ok = wait(&sm.both, both_phase);
      both_phase ^= 1;
    }
    fence_after();
    return ok;
  }

  // The cap: y to cap tanh(y / cap), both in base-2 units.  With u = y / cap and z =
  // 2 u log2(e): where all of a warp's scores are near 0, as most are under the caps that
  // models have, y times the series of tanh(u) / u; else 1 - 2 / (1 + 2^z) for tanh(u),
  // absolute error below 2^-22, in place of the series for those that are not near.
  float cap_in, cap_out, cap_at;  // 2 / softcap, -2 and 1 times softcap log2(e)
  __device__ __forceinline__ void cap8(float *s) const {
    constexpr double kU = 0.34657359027997264, kU2 = kU * kU;  // u = z ln(2) / 2
    constexpr float kNear = (float)(kTanhNear / kU);
    float z[8], far = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const f2 y = pair(s[k], s[k + 1]), zz = mul2(y, pair(cap_in, cap_in)), x = mul2(zz, zz);
      constexpr float c1 = (float)(kTanh1 * kU2), c2 = (float)(kTanh2 * kU2 * kU2),
                      c3 = (float)(kTanh3 * kU2 * kU2 * kU2),
                      c4 = (float)(kTanh4 * kU2 * kU2 * kU2 * kU2);
      f2 t = fma2(pair(c4, c4), x, pair(c3, c3));
      t = fma2(t, x, pair(c2, c2));
      t = fma2(t, x, pair(c1, c1));
      t = fma2(t, x, pair(1.0f, 1.0f));
      unpair(zz, z[k], z[k + 1]);
      unpair(mul2(y, t), s[k], s[k + 1]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) far = max_nan(far, fabsf(z[k]));
    if (__any_sync(kAll, !(far < kNear))) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float t = fmaf(rcp_approx(1.0f + ex2_approx(z[k])), cap_out, cap_at);
        s[k] = fabsf(z[k]) < kNear ? s[k] : t;
      }
    }
  }

  // Scores of a tile that needs more than a factor, in place: capped, biased and
  // masked, in base-2 units.  tok: the thread's token; unit: its k's.
  __device__ __forceinline__ void bend(const Segment &w, int ring, int t, uint32_t c, bool drafted,
                                       bool hidden, float unit, int tok, int c0, int mine,
                                       uint32_t s_at) {
    const int at = w.r.from + (t - w.r.drafted) * kTok + tok, j = t * kTok + tok;
    const bool exists = drafted ? j < w.r.nodes : at < w.r.len, special = drafted && unit < 0.0f;
    const int quarter = tok >> 5, window = hidden ? p.window : 0;
    const float reach = (float)(window + at - w.r.len);
    if (!__any_sync(kAll, exists)) {  // a warp past the last token
      const float none[8] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY,
                             -INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
      for (int ch = 0; ch < mine; ch += 8) tmem_store8(s_at + ch, none);
      tmem_stored();
      return;
    }
    const float position =  // of the token, from the length
        kPlain ? 0.0f : (float)(!drafted ? at - w.r.len : p.slopes && exists ? depth_of(w.b, j) : 0);
    __syncwarp();
    if (__any_sync(kAll, special)) {  // k is not finite: its products term by term
#pragma unroll 1
      for (int i = 0; i < mine; ++i) {
        float s = tmem_load1(s_at + i);
        const float rf = sm.rf[ring][c0 + i];
        // (rf is 0 under a scale of 0, and of rows that do not exist, which see nothing)
        if (special && exists)
          s = rf != 0.0f ? -plain_dot(p, w.b, w.h, w.rt * RN + c0 + i, j) * (p.scale * kLog2e / rf)
                         : __int_as_float(0x7fc00000);
        __syncwarp();
        tmem_store1(s_at + i, s);
        tmem_stored();
      }
    }
#pragma unroll 1
    for (int ch = 0; ch < mine; ch += 8) {
      float s[8];
      tmem_load8(s_at + ch, s);
      const float *rf = &sm.rf[ring][c0 + ch];
      uint32_t seen = exists ? 0xFFu : 0u;
      if (drafted) {
        uint32_t bits = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          bits |= (sm.see[c & 1][quarter][c0 + ch + k] >> lane & 1u) << k;
        seen &= bits;
      } else if (window > 0) {
        uint32_t bits = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) bits |= (uint32_t)(sm.depth[ring][c0 + ch + k] < reach) << k;
        seen &= bits;
      }
      tmem_wait8(s);
      const f2 u2 = pair(unit, unit);
#pragma unroll
      for (int k = 0; k < 8; k += 4) {
        const ulonglong2 r = *reinterpret_cast<const ulonglong2 *>(rf + k);
        unpair(mul2(pair(s[k], s[k + 1]), mul2(r.x, u2)), s[k], s[k + 1]);
        unpair(mul2(pair(s[k + 2], s[k + 3]), mul2(r.y, u2)), s[k + 2], s[k + 3]);
      }
      if (!kPlain && cap_in > 0.0f) cap8(s);
      if (!kPlain && p.slopes) {
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
          const float4 g = *reinterpret_cast<const float4 *>(&sm.slope[ring][c0 + ch + k]);
          const float4 d = *reinterpret_cast<const float4 *>(&sm.depth[ring][c0 + ch + k]);
          s[k] = fmaf(g.x, position - d.x, s[k]);  // (differences are exact)
          s[k + 1] = fmaf(g.y, position - d.y, s[k + 1]);
          s[k + 2] = fmaf(g.z, position - d.z, s[k + 2]);
          s[k + 3] = fmaf(g.w, position - d.w, s[k + 3]);
        }
      }
      if (__any_sync(kAll, seen != 0xFFu)) {
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k] = (seen >> k & 1u) ? s[k] : -INFINITY;
      }
      tmem_store8(s_at + ch, s);
    }
    tmem_stored();
  }

  // 8 scores under their columns' maxima: x = s * factor * unit + nm.
  __device__ __forceinline__ void under(float *s, const float *factor, const float *nm, f2 unit) const {
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      const ulonglong2 r = *reinterpret_cast<const ulonglong2 *>(factor + k);
      const ulonglong2 n = *reinterpret_cast<const ulonglong2 *>(nm + k);
      unpair(fma2(pair(s[k], s[k + 1]), mul2(r.x, unit), n.x), s[k], s[k + 1]);
      unpair(fma2(pair(s[k + 2], s[k + 3]), mul2(r.y, unit), n.y), s[k + 2], s[k + 3]);
    }
  }

  // Sums, or maxima, of 8 values over a warp's lanes: lane 4 i holds that of value i.
  template <bool kMax>
  __device__ __forceinline__ float over_lanes(const float *v) const {
    auto join = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
    float a[4], b[2];
    bool up = lane & 16;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      a[k] = join(up ? v[k + 4] : v[k], __shfl_xor_sync(kAll, up ? v[k] : v[k + 4], 16));
    up = lane & 8;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      b[k] = join(up ? a[k + 2] : a[k], __shfl_xor_sync(kAll, up ? a[k] : a[k + 2], 8));
    up = lane & 4;
    float x = join(up ? b[1] : b[0], __shfl_xor_sync(kAll, up ? b[0] : b[1], 4));
    x = join(x, __shfl_xor_sync(kAll, x, 2));
    return join(x, __shfl_xor_sync(kAll, x, 1));
  }

  // All loops over columns are rolled, 8 at a time, and what a thread keeps per
  // column (scores, sums) stays in tensor memory: their code, times all roles', has
  // to stay inside the instruction cache.  (Sums and scores in registers, loops
  // unrolled: 371 us for the drafted trees of 64 nodes, and 500 with the cap there.)
  __device__ __forceinline__ void softmax() {
    const int group = C::kGroups == 1 ? 0 : (warp - C::kFirst) >> 2;
    const int quarter = warp & 3, tok = quarter * 32 + lane;
    // the group's columns, in eights
    const int parts = (min(RN, p.N * p.G) + 7) / 8, each = (parts + C::kGroups - 1) / C::kGroups;
    const int c0 = group * each * 8, mine = max(min(each, parts - group * each), 0) * 8;
    const bool leader = lane == 0 && quarter == 0;
    const uint32_t lanes = sm.tmem + ((uint32_t)quarter << 21);  // TMEM lanes of this warp
    const uint32_t o_at = lanes + 2 * RN + c0, l_at = lanes + 3 * RN + c0;
    const specdec_kv_cache &kv = p.cache;
    uint32_t c = 0;  // the tile's number, of all
    group_phase = both_phase = 0;
    float *const nms = sm.nm[group];
    if (tok < mine) nms[tok] = 0.0f;
    bool ok = meet(group);
#pragma unroll 1
    for (uint32_t index = 0; ok && segment(index, ok); ++index) {
      const Segment &w = sm.seg[index & 7];
      const int ring = index & 3, t0 = w.t0, t1 = w.t1;
      bool unseen = true;  // the thread's column (tok) has seen no score yet
#pragma unroll 1
      for (int t = t0; t < t1; ++t, ++c) {
        const bool drafted = t < w.r.drafted, first = t == t0;
        const uint32_t s_at = lanes + (c & 1) * RN + c0;
        // (the scores' products have waited for the units, too)
        if (!(ok = wait(&sm.s_full[c & 1], (c >> 1) & 1))) break;
        const float2 unit = drafted ? sm.unit[c & 1][tok] : sm.boxes[c & 7][tok >> box_shift];
        fence_after();
        // a plain tile's scores are a factor away; the others are written back
        const int past = drafted ? (t + 1) * kTok - w.r.nodes
                                 : w.r.from + (t - w.r.drafted + 1) * kTok - w.r.len;
        const bool hidden = !drafted && partly_hidden(p, w.r, t);
        const bool bent = !kPlain || drafted || past > 0 || hidden;
        const float v_unit = past + tok < kTok ? unit.y : 0.0f;
        const float ratio = v_unit * (1.0f / kUnit), v_k = exponent_of(ratio);
        const float k_unit = bent ? 1.0f : unit.x;
        const f2 ks = pair(k_unit, k_unit);
        const float *factor = bent ? sm.ones : sm.rf[ring] + c0;
        if (bent) bend(w, ring, t, c, drafted, hidden, unit.x, tok, c0, mine, s_at);
        // P^T of the tile before in this buffer has been read
        if (!(ok = wait(&sm.pv_done[c % kBuf], empty_par(c, kBuf)))) break;
        if (leader) sm.vote[group][(c - kBuf) & 3] = 0;
        uint8_t *pt = sm.pt[c % kBuf][0] + tok * kRow;
        // The weights are made under the maxima as they are, which seldom move: if
        // some turn out far above a maximum, they are taken back, the maxima move, and
        // they are made again.  At a
        // segment's start the maxima are all at 0 and move from there; after the drafted
        // tokens, of which a row sees a few only, they move at once.
        const bool sure = first || t == w.r.drafted;
        int round = sure ? 2 : 0;  // 0: make, 1: take back, 2: move and make
#pragma unroll 1
        for (;; ++round) {
          if (round == 2) {
            if (!first) {
              if (!(ok = meet(group))) break;  // all have read the maxima
              if (tok < mine && unseen) nms[tok] = 0.0f;
              if (!(ok = meet(group))) break;
            }
#pragma unroll 1
            for (int ch = 0; ch < mine; ch += 8) {
              float s[8];
              tmem_load8(s_at + ch, s);
              tmem_wait8(s);
              under(s, factor + ch, nms + ch, ks);
#pragma unroll
              for (int k = 0; k < 8; ++k) s[k] += v_k;
              const float best = over_lanes<true>(s);
              if ((lane & 3) == 0) sm.red[group][quarter][ch + (lane >> 2)] = best;
              __syncwarp();
            }
            if (!(ok = meet(group))) break;
            if (tok < mine) {
              const float best = fmaxf(fmaxf(sm.red[group][0][tok], sm.red[group][1][tok]),
                                       fmaxf(sm.red[group][2][tok], sm.red[group][3][tok]));
              const float nm = nms[tok];
              float f = 1.0f;
              if (best > -INFINITY && (unseen || best > kLift)) {
                nms[tok] = kLift - (best - nm);
                f = unseen ? 0.0f : ex2_approx(0.5f * (kLift - best));
                unseen = false;
              } else if (unseen) {
                nms[tok] = kUnseen;
              }
              sm.fac[group][0][tok] = f;
            }
            if (!first && !(ok = wait(&sm.pv_done[(c - 1) % kBuf], full_par(c - 1, kBuf)))) break;
            fence_after();
            if (!(ok = meet(group))) break;
            if (!first) {  // the sums, then the outputs
#pragma unroll 1
              for (int i = 0; i < 2 * mine; i += 8) {
                const int ch = i < mine ? i : i - mine;
                const uint32_t at = i < mine ? l_at + ch : o_at + ch;
                const float *fac = sm.fac[group][0] + ch;
                float o[8];
                tmem_load8(at, o);
                tmem_wait8(o);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] = o[k] * fac[k] * fac[k];
                tmem_store8(at, o);
              }
              tmem_stored();
            }
          }
          const float cut = kMost - v_k;
          const f2 r2 = pair(ratio, ratio), sign = round == 1 ? pair(-1.0f, -1.0f) : pair(1.0f, 1.0f);
          float top = -INFINITY;
#pragma unroll 1
          for (int ch = 0; ch < mine; ch += 8) {
            float s[8], l[8];
            tmem_load8(s_at + ch, s);
            tmem_load8(l_at + ch, l);
            tmem_wait8(s);
            tmem_wait8(l);
            under(s, factor + ch, nms + ch, ks);
            uint32_t out[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              top = fmaxf(top, fmaxf(s[2 * k], s[2 * k + 1]));
              const f2 e = pair(ex2_approx(min_nan(s[2 * k], cut)), ex2_approx(min_nan(s[2 * k + 1], cut)));
              if (first) l[2 * k] = l[2 * k + 1] = 0.0f;
              unpair(fma2(e, sign, pair(l[2 * k], l[2 * k + 1])), l[2 * k], l[2 * k + 1]);
              float a, b;
              unpair(mul2(e, r2), a, b);
              out[k] = pack_half2(a, b);
            }
            tmem_store8(l_at + ch, l);
            const int col = c0 + ch;
            *reinterpret_cast<uint4 *>(pt + (col >> 6) * kTileBytes +
                                       ((((col & 63) >> 3) ^ (tok & 7)) << 4)) =
                make_uint4(out[0], out[1], out[2], out[3]);
          }
          tmem_stored();
          if (round == 1) continue;
          const bool vote = round == 0 && __any_sync(kAll, top + v_k > kRaise + kLift);
          fence_async_smem();
          fence_before();
          __syncwarp();
          if (lane == 0) {
            if (vote) sm.vote[group][c & 3] = 1;
            mbar_arrive(round == 0 || sure ? &sm.p_full[c % kBuf] : &sm.again[group]);
          }
          if (round == 2) break;
          if (!(ok = wait(&sm.p_full[c % kBuf], full_par(c, kBuf)))) break;
          if (*(volatile int *)&sm.vote[group][c & 3] == 0) break;
        }
        if (!ok) break;
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.s_empty[c & 1]);
      }
      if (!ok) break;

      // the segment's sums, by column
#pragma unroll 1
      for (int ch = 0; ch < mine; ch += 8) {
        float l[8];
        tmem_load8(l_at + ch, l);
        tmem_wait8(l);
        const float sum = over_lanes<false>(l);
        if ((lane & 3) == 0) sm.red[group][quarter][ch + (lane >> 2)] = sum;
        __syncwarp();
      }
      if (!(ok = wait(&sm.pv_done[(c - 1) % kBuf], full_par(c - 1, kBuf)))) break;
      if (!(ok = meet_all())) break;
      // all are past the segment before; nobody is seven ahead
      if (leader && group == 0) sm.bad[(index + 7) & 7] = sm.dirty[(index + 7) & 7] = 0;
      const int bad = w.r.bad | *(volatile int *)&sm.bad[index & 7];
      const bool dirty = *(volatile int *)&sm.dirty[index & 7] != 0, whole = w.whole;
      float *part = p.part + (size_t)(2 * blockIdx.x + (t0 == 0)) * partial_floats(RN, kv.D);
      // results; a thread for each row first: its statistics, the factor of its
      // outputs (in the room of a sum that only it reads) and their address (in that
      // of the factors)
      float *const out_fac = sm.red[group][0];
      unsigned long long *const out_at = reinterpret_cast<unsigned long long *>(sm.fac[group]);
      if (tok < mine) {
        const int col = c0 + tok, row = w.rt * RN + col, n = node_of(row);
        const float nm = nms[tok];
        const float sum = (sm.red[group][0][tok] + sm.red[group][1][tok]) +
                          (sm.red[group][2][tok] + sm.red[group][3][tok]);
        const bool in = row < p.N * p.G;
        const bool empty = bad || n >= w.r.nodes || sum == 0.0f;
        const int at = (w.b * p.N + n) * p.Hq + w.h * p.G + row - n * p.G;
        float *rec = part + (size_t)col * (kv.D + 2);
        out_fac[tok] = empty ? 0.0f : whole ? __fdividef(kUnit, sum) : 1.0f;
        out_at[tok] = !in     ? 0ull
                      : whole ? reinterpret_cast<unsigned long long>(p.out) + (size_t)at * kv.D * 2
                              : reinterpret_cast<unsigned long long>(rec + 2);
        if (in && whole && p.lse)
          p.lse[at] = empty ? -INFINITY : (log2f(sum) - nm) * 0.6931471805599453f;
        if (in && !whole) {
          rec[0] = empty ? -INFINITY : -nm;
          rec[1] = bad ? -(float)bad : empty ? 0.0f : sum;
        }
        nms[tok] = 0.0f;  // for the next segment
      }
      if (!(ok = meet(group))) break;
      if (dirty)  // what the products left out because it is not finite
#pragma unroll 1
        for (int i = 0; i < mine; ++i) {
          float extra = 0.0f;
          if (out_at[i] && tok < kv.D && out_fac[i] != 0.0f)
            extra = stray(p, box, w.b, w.h, t0, t1, w.rt * RN + c0 + i,
                          w.r.len + (int)sm.depth[ring][c0 + i], tok);
          __syncwarp();
          tmem_store1(o_at + i, tmem_load1(o_at + i) + extra);
          tmem_stored();
        }
#pragma unroll 1
      for (int i = 0; i < mine; i += 4) {
        float o[4];
        __syncwarp();
        tmem_load4(o_at + i, o);
        const float4 f = *reinterpret_cast<const float4 *>(out_fac + i);
        const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(out_at + i);
        const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(out_at + i + 2);
        const float y[4] = {f.x != 0.0f ? o[0] * f.x : 0.0f, f.y != 0.0f ? o[1] * f.y : 0.0f,
                            f.z != 0.0f ? o[2] * f.z : 0.0f, f.w != 0.0f ? o[3] * f.w : 0.0f};
        const unsigned long long at[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool here = at[k] != 0 && tok < kv.D;
          if (whole)
            store_global16(here, at[k] + 2 * tok, pack_bf16x2(y[k], 0.0f));
          else
            store_global32(here, at[k] + 4 * tok, y[k]);
        }
      }
      // the request's first segment sets the status, the join adds what others find
      if (leader && group == 0 && w.h == 0 && w.rt == 0 && t0 == 0) p.row_status[w.b] = bad;
      if (leader) sm.done[group] = index + 1;
      if (!(ok = meet_all())) break;
    }
  }

  // q . k of one row and one drafted token, from global memory, term by term.
  static __device__ __noinline__ float plain_dot(const AttendParams &p, int b, int h, int row, int node) {
    const int D = p.cache.D, n = row / p.G, hq = h * p.G + row - n * p.G;
    float s = 0.0f;
#pragma unroll 1
    for (int e = 0; e < D; ++e)
      s += load_elem(p.q, SPECDEC_BF16, ((long long)b * p.N + n) * p.q_stride + (long long)hq * D + e) *
           load_elem(p.k_new, SPECDEC_BF16,
                     ((long long)b * p.N + node) * p.k_stride + (long long)h * D + e);
    return s;
  }

  // The sum of what is not finite among the v that a row sees in tiles [t0, t1), at
  // element d: drafted tokens', and cached ones' at the window's edge.  A score of
  // -infinity, which takes a k that is not finite, leaves its token out.
  static __device__ __noinline__ float stray(const AttendParams &p, int box, int b, int h, int t0, int t1,
                                      int row, int pos, int d) {
    const specdec_kv_cache &kv = p.cache;
    const Request r = request_of(p, b, box);
    float sum = 0.0f;
    const int j0 = t0 * kTok, j1 = min(t1, r.drafted) * kTok;
    int a = row / p.G;
#pragma unroll 1
    for (int step = 0; a >= 0 && (p.window == 0 || step < p.window); ++step) {
      if (a >= j0 && a < j1) {
        const float y = load_elem(p.v_new, SPECDEC_BF16,
                                  ((long long)b * p.N + a) * p.v_stride + (long long)h * kv.D + d);
        if (!finite(y) && !(p.softcap == 0.0f && plain_dot(p, b, h, row, a) * p.scale == -INFINITY)) sum += y;
      }
      int up = a - 1;
      if (p.parent && a > 0) {
        up = p.parent[(long long)b * p.N + a];
        if (up >= a) up = -1;
      }
      a = up;
    }
#pragma unroll 1
    for (int t = max(t0, r.drafted); t < t1 && partly_hidden(p, r, t); ++t)
#pragma unroll 1
      for (int i = 0; i < kTok; ++i) {
        const int at = r.from + (t - r.drafted) * kTok + i;
        if (at >= r.len || pos - at >= p.window) continue;
        const int id = kv.block_table[(long long)b * kv.max_blocks + at / kv.block];
        if (id < 0 || id >= kv.n_blocks) continue;
        const uint8_t code = reinterpret_cast<const uint8_t *>(
            kv.v)[(((long long)id * kv.Hkv + h) * kv.block + at % kv.block) * kv.D + d];
        if ((code & 0x7Fu) == 0x7Fu) sum = __int_as_float(0x7fc00000);
      }
    return sum;
  }

  // After a wait ran out: the segments that were not finished get no result, and the
  // note says which requests that leaves without one.
  __device__ __noinline__ static void give_up_results(const AttendParams &p, int box,
                                                      const Plan &plan, int finished, int columns) {
    const specdec_kv_cache &kv = p.cache;
    const bool first = threadIdx.x == 32 * C::kFirst;
    Note *note = notes_of(p.part, RN, kv.D) + blockIdx.x;
    Walk walk(p, box, plan);
    Segment w;
#pragma unroll 1
    for (int index = 0; walk.next(p, box, w); ++index) {
      if (index < finished) continue;
      if (first) {
        if (note->lost < 0) note->lost = w.b;
        note->lost_to = w.b;
        if (w.h == 0 && w.rt == 0 && w.t0 == 0) p.row_status[w.b] = SPECDEC_ROW_INTERNAL;
      }
      float *part = p.part + (size_t)(2 * blockIdx.x + (w.t0 == 0)) * partial_floats(RN, kv.D);
#pragma unroll 1
      for (int col = threadIdx.x - 32 * C::kFirst; col < columns; col += C::kThreads - 32 * C::kFirst) {
        const int row = w.rt * RN + col, n = row / p.G;
        if (row >= p.N * p.G) continue;
        const long long at = ((long long)w.b * p.N + n) * p.Hq + w.h * p.G + row - n * p.G;
        if (w.whole) {
#pragma unroll 1
          for (int d = 0; d < kv.D; ++d) reinterpret_cast<unsigned short *>(p.out)[at * kv.D + d] = 0;
          if (p.lse) p.lse[at] = -INFINITY;
        } else {
          part[(size_t)col * (kv.D + 2)] = -INFINITY;
          part[(size_t)col * (kv.D + 2) + 1] = -(float)SPECDEC_ROW_INTERNAL;
        }
      }
    }
  }
};

template <int RN, bool kPlain>
__global__ void __launch_bounds__(Cfg<RN>::kThreads, Cfg<RN>::kCtas)
    attend_tile_kernel(const __grid_constant__ AttendParams p,
                       const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map, int box) {
  extern __shared__ __align__(1024) uint8_t raw[];
  using S = Smem<RN>;
  using C = Cfg<RN>;
  // an offset, not a rounded pointer: the compiler has to know that it is shared memory
  S &sm = *reinterpret_cast<S *>(raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid < 8) {
    sm.bad[tid] = sm.dirty[tid] = 0;
    mbar_init(&sm.seg_full[tid], 1);
    mbar_init(&sm.box_full[tid], 4);
    if (tid < C::kK) {
      mbar_init(&sm.k_full[tid], 1);
      mbar_init(&sm.k_empty[tid], 1);
    }
    if (tid < C::kV) {
      mbar_init(&sm.v_full[tid], 1);
      mbar_init(&sm.v_empty[tid], C::kWorkers);
    }
    if (tid < 2) {
      mbar_init(&sm.s_full[tid], 1);
      mbar_init(&sm.s_empty[tid], 4 * C::kGroups);
    }
    if (tid < C::kBuf) {
      mbar_init(&sm.p_full[tid], 4 * C::kGroups);
      mbar_init(&sm.vh_full[tid], C::kWorkers);
      mbar_init(&sm.pv_done[tid], 1);
    }
    if (tid < C::kGroups) {
      mbar_init(&sm.group[tid], 4);
      mbar_init(&sm.again[tid], 4);
      sm.moves[tid] = 0;
      sm.done[tid] = 0;
    }
    if (tid == 0) {
      mbar_init(&sm.q_full, C::kWorkers);
      mbar_init(&sm.q_empty, 1);
      mbar_init(&sm.both, 4 * C::kGroups);
      mbar_init(&sm.fin, 1);
      sm.give_up = 0;
    }
    fence_mbar_init();
    fence_async_smem();
  }
  if (tid < C::kCols) sm.ones[tid] = 1.0f;
  if (tid < 4 * C::kGroups) sm.vote[tid >> 2][tid & 3] = 0;
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&sm.tmem)),
                 "r"(C::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();
  fence_before();
  __syncthreads();
  fence_after();
  const Plan plan = make_plan(p, box, blockIdx.x, gridDim.x, sm.scan, &sm.plan);
  Tile<RN, kPlain> tile(p, sm, &k_map, &v_map, box);
  // warps 0-3: copies, products (two stay idle); 4-7: operands; the others: softmax
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kIssue));
    if (warp == 0)
      tile.copies(plan);
    else if (warp == 1)
      tile.products();
  } else if (warp < C::kFirst) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kWiden));
    tile.operands();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoft));
    tile.softmax();
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (sm.give_up) {
    if (warp == 0) tile.drain();
    if (warp >= C::kFirst) {
      int finished = sm.done[0];
      for (int i = 1; i < C::kGroups; ++i) finished = min(finished, sm.done[i]);
      tile.give_up_results(p, box, plan, finished, tile.columns);
    }
    __syncthreads();
  }
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sm.tmem),
                 "r"(C::kTmem));
}

// Joins the units that the cuts between CTAs divide.  Block (i, y): the unit that
// CTA i was in the middle of at its start, if it is the first that was; the y-th
// part of its rows.  Flags are added to the status that each request's first segment
// has set: those of the parts, and of what CTA i gave up, whatever head that was of.
constexpr int kJoinRows = 8;  // a warp each
__global__ void __launch_bounds__(32 * kJoinRows)
    attend_tile_join_kernel(const __grid_constant__ AttendParams p, int ctas, int RN) {
  pdl_wait();
  pdl_launch_dependents();
  const int i = blockIdx.x, D = p.cache.D, lane = threadIdx.x & 31;
  const int size = (int)partial_floats(RN, D);
  const Note *notes = notes_of(p.part, RN, D);
  const int mine = notes[i].first, unit = notes[i].unit, lost = notes[i].lost;
  if (lost >= 0 && blockIdx.y == 0)
    for (int b = lost + threadIdx.x; b <= notes[i].lost_to; b += blockDim.x)
      atomicOr(p.row_status + b, SPECDEC_ROW_INTERNAL);
  if (mine == 0) return;  // begins with a unit, or has no tile
  // the CTAs before: the one that began the unit is the last that has tiles
  int begun = -1;
#pragma unroll 1
  for (int at = i - 1; at >= 0 && begun < 0; at -= 32) {
    const unsigned full = __ballot_sync(kAll, at - lane >= 0 && notes[at - lane].tiles > 0);
    if (full) begun = at - (__ffs(full) - 1);
  }
  if (begun < 0 || notes[begun].open != mine) return;  // it was in the middle, too
  const int row = notes[i].rt * RN + blockIdx.y * kJoinRows + (threadIdx.x >> 5);
  const int r = row - notes[i].rt * RN;
  if (r >= RN || row >= p.N * p.G) return;
  // Parts: that one's second slot, then first slots until the unit's end.  32 at a
  // time, a lane each: its maximum, sum and flags; the factors that bring both and
  // the outputs under the largest maximum; then the outputs, four elements a lane.
  float all = -INFINITY, sum = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  int bad = 0, left = unit - mine;
  const float *const part = p.part + r * (D + 2);
#pragma unroll 1
  for (int at = i - 1; left > 0 && at < ctas; at += 32) {  // CTA at + lane; i - 1 stands for `begun`
    const int cta = at + lane;
    int head = 0, slot = 2 * cta;
    if (cta < i) {
      slot = 2 * begun + 1;
    } else if (cta < ctas && notes[cta].tiles > 0) {
      head = notes[cta].head;
    }
    int upto = head;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kAll, upto, d);
      if (lane >= d) upto += o;
    }
    const bool in = cta < i || (head > 0 && upto - head < left);
    float m = -INFINITY, l = 0.0f;
    if (in) {
      m = part[slot * size];
      l = part[slot * size + 1];
    }
    if (l < 0.0f) bad |= (int)-l;
    float most = m;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, d));
    most = fmaxf(all, most);
    // (square roots, as a factor may be out of range where what it scales is not)
    const float before = all > -INFINITY ? ex2_approx(0.5f * (all - most)) : 0.0f;
    const float f = m > -INFINITY ? ex2_approx(0.5f * (m - most)) : 0.0f;
    all = most;
    sum = sum * before * before + l * f * f;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = acc[k] * before * before;
    // (a part under a factor of 0 takes part all the same: its outputs may be NaN)
    const unsigned full = __ballot_sync(kAll, m > -INFINITY);
#pragma unroll 1
    for (int s = 0; full >> s; s += 4) {
      float2 x[4][2];
      float g[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int from = (s + u) & 31;
        g[u] = (full >> s >> u & 1) ? __shfl_sync(kAll, f * f, from) : 0.0f;
        const float *rec = part + __shfl_sync(kAll, slot, from) * size + 2 + 4 * lane;
        x[u][0] = x[u][1] = make_float2(0.0f, 0.0f);
        if ((full >> s >> u & 1) && 4 * lane < D) {
          x[u][0] = *reinterpret_cast<const float2 *>(rec);
          x[u][1] = *reinterpret_cast<const float2 *>(rec + 2);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        acc[0] += g[u] * x[u][0].x;
        acc[1] += g[u] * x[u][0].y;
        acc[2] += g[u] * x[u][1].x;
        acc[3] += g[u] * x[u][1].y;
      }
      if (s == 28) break;
    }
    left -= __shfl_sync(kAll, upto, 31);
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
  bad = __reduce_or_sync(kAll, bad);
  const bool empty = bad || all == -INFINITY;
  const float inv = empty ? 0.0f : __fdividef(kUnit, sum);
  const int n = row / p.G, h = notes[i].h, b = notes[i].b;
  const long long at = ((long long)b * p.N + n) * p.Hq + h * p.G + row - n * p.G;
  if (4 * lane < D) {
    unsigned short *out = reinterpret_cast<unsigned short *>(p.out) + at * D + 4 * lane;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      out[k] = (unsigned short)pack_bf16x2(empty ? 0.0f : acc[k] * inv, 0.0f);
  }
  if (p.lse && lane == 0) p.lse[at] = empty ? -INFINITY : (all + log2f(sum)) * 0.6931471805599453f;
  if (bad && lane == 0) atomicOr(p.row_status + b, bad);
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static std::atomic<EncodeFn> cached{nullptr};
  EncodeFn f = cached.load(std::memory_order_acquire);
  if (f) return f;
  void *sym = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &sym, 12000, cudaEnableDefault,
                                       &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<EncodeFn>(sym);
  cached.store(f, std::memory_order_release);
  return f;
}

// The pool as rows of D bytes (a token of a head each); boxes of `box` rows and
// 128 bytes, what lies past D read as zeros.
bool encode(CUtensorMap *map, void *codes, const specdec_kv_cache &kv, int box) {
  const EncodeFn f = encode_fn();
  if (!f) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)kv.D, (cuuint64_t)kv.n_blocks * kv.Hkv * kv.block};
  const cuuint64_t strides[1] = {(cuuint64_t)kv.D};
  const cuuint32_t size[2] = {(cuuint32_t)kRow, (cuuint32_t)box}, step[2] = {1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, strides, size, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int box_rows(int block) {  // the largest power of two that divides the block and half a tile
  int box = 16;
  while (box < kTok / 2 && block % (2 * box) == 0) box *= 2;
  return box;
}

int rows_of(int N, int G) {  // the classes of the kernel
  const int rows = N * G;
  return rows <= 32 ? 32 : rows <= 48 ? 48 : rows <= 64 ? 64 : 128;
}

template <int RN, bool kPlain>
cudaError_t launch_rn(AttendParams p, cudaStream_t stream) {
  static DeviceOnce once;
  const int smem = (int)sizeof(Smem<RN>) + 1024;
  static_assert(offsetof(Smem<RN>, rf) % 16 == 0 && offsetof(Smem<RN>, nm) % 16 == 0 &&
                    offsetof(Smem<RN>, ones) % 16 == 0 && offsetof(Smem<RN>, fac) % 16 == 0 &&
                    offsetof(Smem<RN>, q) % 1024 == 0,
                "read in 16-byte vectors, and by swizzled copies and products");
  static_assert((sizeof(Smem<RN>) + 2048) * Cfg<RN>::kCtas <= 233472, "shared memory of an SM");
  cudaError_t err = smem_opt_in_once(once, attend_tile_kernel<RN, kPlain>, smem);
  if (err != cudaSuccess) return err;
  CUtensorMap k_map, v_map;
  const int box = box_rows(p.cache.block);
  if (!encode(&k_map, p.cache.k, p.cache, box) || !encode(&v_map, p.cache.v, p.cache, box))
    return cudaErrorInvalidValue;
  p.row_tiles = (p.N * p.G + RN - 1) / RN;
  const int sms = device_sm_count();
  const int ctas = (sms < kMaxSms ? sms : kMaxSms) * Cfg<RN>::kCtas;
  err = launch_pdl(attend_tile_kernel<RN, kPlain>, dim3((unsigned)ctas), dim3(Cfg<RN>::kThreads),
                   (size_t)smem, stream, p, k_map, v_map, box);
  if (err != cudaSuccess) return err;
  const int rows = p.N * p.G < RN ? p.N * p.G : RN;
  return launch_pdl(attend_tile_join_kernel,
                    dim3((unsigned)ctas, (unsigned)((rows + kJoinRows - 1) / kJoinRows)),
                    dim3(32 * kJoinRows), 0, stream, p, ctas, RN);
}

}  // namespace

size_t attend_tile_workspace_bytes(int N, int G, int D) {
  const int RN = rows_of(N, G);
  return 4 * kMaxSms * partial_floats(RN, D) * sizeof(float) + 2 * kMaxSms * sizeof(Note);
}

bool attend_tile_applies(const AttendParams &p) {
  const specdec_kv_cache &kv = p.cache;
  const long long units = (long long)kv.Hkv * ((p.N * p.G + 127) / 128 + 1);
  return p.dtype == SPECDEC_BF16 && kv.D <= kRow &&
         (long long)kv.n_blocks * kv.Hkv * kv.block < (1ll << 31) - kTok &&
         ((long long)kv.max_blocks * kv.block / kTok + p.N + kExtra) * units < (1ll << 31);
}

cudaError_t launch_attend_tile(const AttendParams &p, cudaStream_t stream) {
  const bool plain = p.softcap == 0.0f && !p.slopes;
  const int rows = rows_of(p.N, p.G);
  if (rows == 32)
    return plain ? launch_rn<32, true>(p, stream) : launch_rn<32, false>(p, stream);
  if (rows == 48)
    return plain ? launch_rn<48, true>(p, stream) : launch_rn<48, false>(p, stream);
  if (rows == 64)
    return plain ? launch_rn<64, true>(p, stream) : launch_rn<64, false>(p, stream);
  return plain ? launch_rn<128, true>(p, stream) : launch_rn<128, false>(p, stream);
}

}  // namespace specdec
