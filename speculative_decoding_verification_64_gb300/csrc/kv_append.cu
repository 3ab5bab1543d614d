// Append of accepted tokens to the 8-bit paged cache (specdec_kv_append).
//
// For each block of tokens and head that gets tokens, with x the new values:
//     s = max(2^ceil(log2(max |x| / 448)), 2^-100, s_old if tokens stand before),
//     code = e4m3(x / s), and old codes c -> e4m3(c s_old / s) where s grew.
// A power of two as the scale makes x / s exact, so a code is one rounding of
// its value, and a grown scale only rounds off bits below the new smallest
// step; e4m3's own exponent covers the factor of two that a finer scale would
// give.
//
// One task is one block of tokens, of one head, of k or of v; a thread takes 16
// elements at a time and holds its first ones in registers between the maximum
// and the codes (only what is beyond them is read again, from L1 or L2).  A verify
// step's few tokens are a warp's work, a prompt's blocks a CTA's.
//
// Measured: 8 prompts of 8191 tokens, 8 heads of 128, 111 us, 3.6 TB/s, against
// 139 us with every value read twice; what is left is each CTA's chain of length,
// table and values, eighteen rounds of CTAs.  256 requests of up to 9
// tokens 12.3 us, the same chain once, in cold caches.
#include "attention_common.cuh"

namespace specdec {
namespace {

// The smallest power of two s >= 2^-100 with a <= 448 s (a finite, >= 0), from
// a's exponent field: 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_for(float a) {
  if (!(a > 448.0f * 0x1p-100f)) return 0x1p-100f;
  const uint32_t u = __float_as_uint(a);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// 16 consecutive elements, as they stand in memory and as float32 values.
template <int DT>
struct Raw {
  uint4 w[DT == SPECDEC_F32 ? 4 : 2];
};

template <int DT, bool kVec>
__device__ __forceinline__ Raw<DT> load16(const char *in) {
  constexpr int kWords = sizeof(Raw<DT>) / 16;
  Raw<DT> r;
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    if constexpr (kVec) {
      r.w[i] = __ldg(reinterpret_cast<const uint4 *>(in) + i);
    } else {
      uint32_t a[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (DT == SPECDEC_F32) {
          a[k] = __ldg(reinterpret_cast<const uint32_t *>(in) + 4 * i + k);
        } else {
          const unsigned short *h = reinterpret_cast<const unsigned short *>(in) + 8 * i + 2 * k;
          a[k] = __ldg(h) | (uint32_t)__ldg(h + 1) << 16;
        }
      }
      r.w[i] = make_uint4(a[0], a[1], a[2], a[3]);
    }
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void values16(const Raw<DT> &r, float *x) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(r) / 16; ++i) {
    const uint32_t a[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (DT == SPECDEC_F32) {
        x[4 * i + k] = __uint_as_float(a[k]);
      } else {
        x[8 * i + 2 * k] = bf16_lo(a[k]);
        x[8 * i + 2 * k + 1] = bf16_hi(a[k]);
      }
    }
  }
}

// The largest finite size of 16 elements and `top`.
template <int DT>
__device__ __forceinline__ float top16(const Raw<DT> &r, float top) {
  float x[16];
  values16<DT>(r, x);
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float a = fabsf(x[k]);
    if (a < INFINITY) top = fmaxf(top, a);
  }
  return top;
}

// kT threads work on one task: 32 (a warp) or the whole CTA.
template <int kT>
__device__ __forceinline__ void task_sync() {
  if (kT == 32)
    __syncwarp();
  else
    __syncthreads();
}

template <int kT>
__device__ __forceinline__ bool task_any(bool x) {
  if (kT == 32) return __any_sync(0xffffffffu, x);
  return __syncthreads_or(x) != 0;
}

// Six CTAs an SM for bfloat16 prompts: 111 us for the prompts above, with the 62
// registers that the compiler would take 123, with eight CTAs 119.
template <int DT, bool kVec, int kT>
__global__ void __launch_bounds__(256, kT == 256 && DT != SPECDEC_F32 ? 6 : 3) kv_append_kernel(const AppendParams p) {
  __shared__ float red[8];
  pdl_wait();
  pdl_launch_dependents();
  constexpr int es = DT == SPECDEC_F32 ? 4 : 2;
  constexpr int kHeld = DT == SPECDEC_F32 ? 2 : kT == 32 ? 4 : 2;  // a thread's first values
  const specdec_kv_cache &c = p.cache;
  const int t = kT == 32 ? threadIdx.x & 31 : threadIdx.x;
  // task = ((b * blocks + m) * 2 + side) * Hkv + h
  uint32_t task = blockIdx.x;
  if (kT == 32) {
    task = task * 8 + (threadIdx.x >> 5);
    if (task >= (uint32_t)p.B * p.blocks * 2 * c.Hkv) return;
  }
  const int h = (int)(task % (uint32_t)c.Hkv);
  task /= (uint32_t)c.Hkv;
  const int side = (int)(task & 1);
  task >>= 1;
  const int m = (int)(task % (uint32_t)p.blocks);
  const long long b = task / (uint32_t)p.blocks;

  const int len = c.length[b];
  const long long count = (long long)(p.count ? p.count[b] : p.N) + p.extra;
  const long long most = (long long)c.max_blocks * c.block;
  int status = 0;
  if (len < 0 || len > most || count < 0 || count > (p.path ? min(p.path_len, p.N) : p.N) ||
      len + count > most)
    status = SPECDEC_ROW_BAD_CACHE;
  const int first = status ? 0 : len / c.block;

  // this task's tokens: slots [off, off + take) of the block, tokens j0 ...
  const long long start = (long long)(first + m) * c.block;
  const int off = m == 0 ? len - first * c.block : 0;
  const long long j0 = start + off - len;
  const int take = status ? 0 : (int)max(min((long long)(c.block - off), count - j0), 0ll);
  const char *src = reinterpret_cast<const char *>(side ? p.v : p.k) + (long long)h * c.D * es;
  const long long stride = (side ? p.v_stride : p.k_stride) * es;
  const uint32_t per = c.D / 16, vecs = take * per;
  auto load = [&](uint32_t i) {
    const uint32_t j = i / per, e = (i - j * per) * 16;
    int n = (int)j0 + (int)j;
    if (p.path) n = min(max(p.path[b * p.path_len + n], 0), p.N - 1);  // (checked below)
    return load16<DT, kVec>(src + (b * p.N + n) * stride + (int)e * es);
  };
  // the first values are under way while the blocks and the path are checked
  Raw<DT> held[kHeld];
#pragma unroll
  for (int q = 0; q < kHeld; ++q)
    if (t + q * kT < vecs) held[q] = load(t + q * kT);

  if (!status && count > 0) {
    // every task of a request checks all that the request touches, so that a
    // request is appended whole or not at all
    const int last = (int)((len + count - 1) / c.block);
    bool bad_id = false, bad_node = false;
    for (int i = first + t; i <= last; i += kT) {
      const int id = c.block_table[b * c.max_blocks + i];
      bad_id |= id < 0 || id >= c.n_blocks;
    }
    if (p.path)
      for (int i = t; i < count; i += kT) {
        const int n = p.path[b * p.path_len + i];
        bad_node |= n < 0 || n >= p.N;
      }
    if (task_any<kT>(bad_id)) status = SPECDEC_ROW_BAD_CACHE;
    if (task_any<kT>(bad_node)) status |= SPECDEC_ROW_BAD_TREE;
  }
  if (m == 0 && side == 0 && h == 0 && t == 0) {
    p.new_length[b] = len + (status ? 0 : (int)count);
    p.row_status[b] = status;
  }
  if (status || count == 0) return;

  if (take <= 0) return;
  const int id = c.block_table[b * c.max_blocks + first + m];
  const long long cell = (long long)id * c.Hkv + h;
  uint8_t *codes = reinterpret_cast<uint8_t *>(side ? c.v : c.k) + cell * c.block * c.D;
  float *scale = (side ? c.v_scale : c.k_scale) + cell;

  float top = 0.0f;
#pragma unroll
  for (int q = 0; q < kHeld; ++q)
    if (t + q * kT < vecs) top = top16<DT>(held[q], top);
#pragma unroll 1
  for (uint32_t i = t + kHeld * kT; i < vecs; i += kT) top = top16<DT>(load(i), top);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (kT > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) top = fmaxf(top, red[w]);
  }
  float s = scale_for(top);
  if (off > 0) {
    const float was = *scale;
    task_sync<kT>();  // read by all before one of them writes it
    if (was >= s) {
      s = was;
    } else {
      // the tokens that stand before: 16 codes a thread, each thread its own
      const float ratio = __fdiv_rn(was, s);
      for (uint32_t i = t; i < off * per; i += kT) {
        uint4 w = reinterpret_cast<uint4 *>(codes)[i];
        uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t lo = e4m3x2_to_half2(a[k] & 0xFFFFu), hi = e4m3x2_to_half2(a[k] >> 16);
          a[k] = pack_e4m3x2(half_bits_to_float(lo & 0xFFFFu) * ratio,
                             half_bits_to_float(lo >> 16) * ratio) |
                 pack_e4m3x2(half_bits_to_float(hi & 0xFFFFu) * ratio,
                             half_bits_to_float(hi >> 16) * ratio)
                     << 16;
        }
        reinterpret_cast<uint4 *>(codes)[i] = make_uint4(a[0], a[1], a[2], a[3]);
      }
    }
  }
  if (t == 0) *scale = s;
  // x / s is exact for a power of two; an old scale of another kind needs the division
  const bool pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0;
  const float inv = pow2 ? __fdiv_rn(1.0f, s) : 0.0f;
  auto put = [&](uint32_t i, const Raw<DT> &r) {  // (token, element) of the block: slot off + i / per
    float x[16];
    values16<DT>(r, x);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float y = pow2 ? x[k] * inv : __fdiv_rn(x[k], s);
      x[k] = finite(x[k]) ? y : __int_as_float(0x7fc00000);
    }
    uint32_t a[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      a[k] = pack_e4m3x2(x[4 * k], x[4 * k + 1]) | pack_e4m3x2(x[4 * k + 2], x[4 * k + 3]) << 16;
    reinterpret_cast<uint4 *>(codes)[off * per + i] = make_uint4(a[0], a[1], a[2], a[3]);
  };
#pragma unroll
  for (int q = 0; q < kHeld; ++q)
    if (t + q * kT < vecs) put(t + q * kT, held[q]);
#pragma unroll 1
  for (uint32_t i = t + kHeld * kT; i < vecs; i += kT) put(i, load(i));
}

template <int DT, bool kVec>
cudaError_t launch_vec(const AppendParams &p, cudaStream_t stream) {
  const long long tasks = (long long)p.B * p.blocks * 2 * p.cache.Hkv;
  if (p.N <= 64)
    return launch_pdl(kv_append_kernel<DT, kVec, 32>, dim3((unsigned)((tasks + 7) / 8)), dim3(256),
                      0, stream, p);
  return launch_pdl(kv_append_kernel<DT, kVec, 256>, dim3((unsigned)tasks), dim3(256), 0, stream,
                    p);
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream) {
  const int es = p.dtype == SPECDEC_F32 ? 4 : 2;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v) |
                       (uintptr_t)(p.k_stride * es) | (uintptr_t)(p.v_stride * es);
  const bool vec = (at & 15) == 0;  // heads start on multiples of 16 elements
  if (p.dtype == SPECDEC_F32)
    return vec ? launch_vec<SPECDEC_F32, true>(p, stream)
               : launch_vec<SPECDEC_F32, false>(p, stream);
  return vec ? launch_vec<SPECDEC_BF16, true>(p, stream)
             : launch_vec<SPECDEC_BF16, false>(p, stream);
}

}  // namespace specdec
