// Rotary positions of q and k (specdec_rope): pair i of a head at position p
// turns by a = 2 pi p f_i,
//     y1 = m (x1 cos a - x2 sin a),   y2 = m (x2 cos a + x1 sin a),
// the gradient by -a.  f_i comes in units of 2^-64 turns, so p f_i mod 2^64 is
// an integer product that drops the whole turns without rounding; its top 32
// bits, as a signed fraction of a half turn, go through sincospi.  A float32
// angle would be off by up to 4e-3 at position 100000 already.
//
// One CTA per token: its first rot/2 threads make the token's sines and cosines
// once, and all heads of q and k then read them from shared memory.  Bound by
// HBM: every element is read and written once, in 16-byte vectors where
// pointers, strides and the split of the head allow, else element by element.
//
// Measured (32 + 8 heads of 128): 8 x 8191 tokens, the gradient, 218 us, 6.1 TB/s;
// 32 trees of 64 nodes, half of the head, 16.5 us, 2.5 TB/s, a chain of the depth
// walk, the sines and one pass over the heads; one request of 5 nodes 4.8 us.
#include "attention_common.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 256;

template <int DT>
__device__ __forceinline__ float load_one(const void *p, long long i) {
  return load_elem(p, DT, i);
}

template <int DT>
__device__ __forceinline__ void store_one(void *p, long long i, float x) {
  if (DT == SPECDEC_F32)
    reinterpret_cast<float *>(p)[i] = x;
  else
    reinterpret_cast<unsigned short *>(p)[i] = (unsigned short)pack_bf16x2(x, 0.0f);
}

// A 16-byte vector as float32 values and back.
template <int DT>
__device__ __forceinline__ void unpack(const uint4 &w, float *x) {
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

template <int DT>
__device__ __forceinline__ uint4 pack(const float *x) {
  if (DT == SPECDEC_F32)
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ void turn(float &a, float &b, float2 cs) {
  const float u = a * cs.x - b * cs.y;
  b = b * cs.x + a * cs.y;
  a = u;
}

template <int DT, bool kVec, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  __shared__ float2 cs[SPECDEC_MAX_HEAD_DIM / 2];
  pdl_wait();
  pdl_launch_dependents();
  const long long token = blockIdx.x;
  const int half = p.rot / 2;
  if (threadIdx.x < half) {
    int pos;
    if (p.positions) {
      pos = p.positions[token];
    } else {
      const long long b = token / p.N;
      const int n = (int)(token - b * p.N);
      int depth = n;
      if (p.parent) {
        const int32_t *parent = p.parent + b * p.N;
        depth = 0;
        for (int a = n; a > 0; ++depth) {  // the index falls with every step
          const int up = parent[a];
          if (up < 0 || up >= a) break;
          a = up;
        }
      }
      pos = (p.base ? p.base[b] : 0) + depth;
    }
    const unsigned long long phase =
        (unsigned long long)(long long)pos * p.freq[threadIdx.x];
    float s, c;
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
    if (p.backward) s = -s;
    cs[threadIdx.x] = make_float2(c * p.magnitude, s * p.magnitude);
  }
  __syncthreads();

  constexpr int kE = kVec ? (DT == SPECDEC_F32 ? 4 : 8) : 1;  // elements an access
  constexpr int es = DT == SPECDEC_F32 ? 4 : 2;
  const int heads = p.Hq + p.Hk;
  // items of one head: its pairs (vectors of pairs), then what is copied
  const int turned = (kInterleaved && kVec) ? p.rot / kE : half / kE;
  const int per = turned + (p.D - p.rot) / kE;
  for (int i = threadIdx.x; i < heads * per; i += kThreads) {
    const int head = i / per, j = i - head * per;
    const bool is_q = head < p.Hq;
    const int h = is_q ? head : head - p.Hq;
    const char *in = reinterpret_cast<const char *>(is_q ? p.q : p.k) +
                     (token * (is_q ? p.q_stride : p.k_stride) + (long long)h * p.D) * es;
    char *out = reinterpret_cast<char *>(is_q ? p.q_out : p.k_out) +
                (token * (is_q ? p.Hq : p.Hk) + h) * (long long)p.D * es;
    if (j >= turned) {  // not rotated
      const int e = p.rot + (j - turned) * kE;
      if (kVec)
        *reinterpret_cast<uint4 *>(out + e * es) = *reinterpret_cast<const uint4 *>(in + e * es);
      else
        store_one<DT>(out, e, load_one<DT>(in, e));
    } else if (!kVec) {
      const int e1 = kInterleaved ? 2 * j : j, e2 = kInterleaved ? 2 * j + 1 : j + half;
      float a = load_one<DT>(in, e1), b = load_one<DT>(in, e2);
      turn(a, b, cs[j]);
      store_one<DT>(out, e1, a);
      store_one<DT>(out, e2, b);
    } else if (kInterleaved) {
      float x[kE];
      unpack<DT>(*reinterpret_cast<const uint4 *>(in + j * 16), x);
#pragma unroll
      for (int k = 0; k < kE; k += 2) turn(x[k], x[k + 1], cs[j * (kE / 2) + k / 2]);
      *reinterpret_cast<uint4 *>(out + j * 16) = pack<DT>(x);
    } else {
      float x[kE], y[kE];
      unpack<DT>(*reinterpret_cast<const uint4 *>(in + j * 16), x);
      unpack<DT>(*reinterpret_cast<const uint4 *>(in + half * es + j * 16), y);
#pragma unroll
      for (int k = 0; k < kE; ++k) turn(x[k], y[k], cs[j * kE + k]);
      *reinterpret_cast<uint4 *>(out + j * 16) = pack<DT>(x);
      *reinterpret_cast<uint4 *>(out + half * es + j * 16) = pack<DT>(y);
    }
  }
}

template <int DT>
cudaError_t launch_dt(const RopeParams &p, bool vec, cudaStream_t stream) {
  const dim3 grid((unsigned)((long long)p.B * p.N)), block(kThreads);
  if (vec)
    return p.interleaved ? launch_pdl(rope_kernel<DT, true, true>, grid, block, 0, stream, p)
                         : launch_pdl(rope_kernel<DT, true, false>, grid, block, 0, stream, p);
  return p.interleaved ? launch_pdl(rope_kernel<DT, false, true>, grid, block, 0, stream, p)
                       : launch_pdl(rope_kernel<DT, false, false>, grid, block, 0, stream, p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, cudaStream_t stream) {
  // 16-byte vectors need every row, and the two halves of its rotated part, on
  // 16-byte boundaries.
  const int es = p.dtype == SPECDEC_F32 ? 4 : 2;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) |
                       reinterpret_cast<uintptr_t>(p.q_out) | reinterpret_cast<uintptr_t>(p.k_out) |
                       (uintptr_t)(p.q_stride * es) | (uintptr_t)(p.k_stride * es) |
                       (uintptr_t)(p.D * es) |
                       (uintptr_t)((p.interleaved ? p.rot : p.rot / 2) * es);
  const bool vec = (at & 15) == 0;
  return p.dtype == SPECDEC_F32 ? launch_dt<SPECDEC_F32>(p, vec, stream)
                                : launch_dt<SPECDEC_BF16>(p, vec, stream);
}

}  // namespace specdec
