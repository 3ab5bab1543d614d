// Parameter blocks and device helpers of the attention side of the step:
// rotary positions (rope.cu), the append to the 8-bit cache (kv_append.cu) and
// the attention of drafted tokens over it (attend.cu, attend_tile.cu).
#pragma once

#include "common.cuh"

namespace specdec {

struct RopeParams {
  const void *q, *k;
  void *q_out, *k_out;
  long long q_stride, k_stride;
  const uint64_t *freq;
  const int32_t *positions, *base, *parent;
  int B, N, Hq, Hk, D, rot, dtype;
  bool interleaved, backward;
  float magnitude;
};

struct AppendParams {
  const void *k, *v;
  long long k_stride, v_stride;
  const int32_t *count, *path;
  int extra, path_len;
  specdec_kv_cache cache;
  int B, N, dtype;
  int blocks;  // most blocks that one request's tokens can touch
  int32_t *new_length, *row_status;
};

struct AttendParams {
  const void *q, *k_new, *v_new;
  long long q_stride, k_stride, v_stride;
  const int32_t *parent, *n_nodes;
  specdec_kv_cache cache;
  int B, N, Hq, G, dtype;
  float scale, softcap;
  const float *slopes;
  int window;
  void *out;
  float *lse;
  int32_t *row_status;
  float *part;  // split partials in the workspace
  int splits, row_tiles;
  bool clustered;   // the splits are one cluster
  int block_shift;  // log2(cache.block), or -1
};

cudaError_t launch_rope(const RopeParams &p, cudaStream_t stream);
cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream);
cudaError_t launch_attend(AttendParams p, cudaStream_t stream);
// attend_tile.cu: the tensor-core kernel, for the calls that it takes
bool attend_tile_applies(const AttendParams &p);
size_t attend_tile_workspace_bytes(int N, int G, int D);
cudaError_t launch_attend_tile(const AttendParams &p, cudaStream_t stream);
size_t attend_workspace_bytes(long long B, int N, int Hq, int Hkv, int D, int dtype);

#ifdef __CUDACC__

// two e4m3 codes (the low 16 bits of `two`) as two fp16 values: exact
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
      : "=r"(r)
      : "r"(two));
  return r;
}

__device__ __forceinline__ float half_bits_to_float(uint32_t h) {
  float r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.f32.f16 %0, t;\n\t}" : "=f"(r) : "r"(h));
  return r;
}

// (lo, hi) rounded to fp16 and packed, lo in the low half
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// (lo, hi) rounded to e4m3 and packed into 16 bits, lo in the low byte;
// beyond 448 the largest code, NaN to the NaN code
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// tanh(u) / u by its Taylor series, 1 + kTanh1 u^2 + ... + kTanh4 u^8, for sizes of u
// below kTanhNear: the terms alternate and fall, so the error is below the next one,
// 1382 / 155925 u^10 < 2^-26.  As a factor of the score it keeps the score's own bits
// under a cap of any size, where cap (1 - 2 / (1 + e^2u)) is off by 2^-22 of the cap.
constexpr float kTanhNear = 0.25f;
constexpr double kTanh1 = -1.0 / 3, kTanh2 = 2.0 / 15, kTanh3 = -17.0 / 315, kTanh4 = 62.0 / 2835;

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

#endif

}  // namespace specdec
