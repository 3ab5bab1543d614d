// C ABI of the attention side of the step: argument checks and launches of
// specdec_rope, specdec_kv_append and specdec_attend (include/specdec.h).
// Like the verify calls these are asynchronous, allocate nothing and check
// their arguments before any device work.
#include <climits>
#include <cmath>

#include "attention_common.cuh"

using namespace specdec;

namespace {

int cuda_status(cudaError_t e) { return e == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA; }

int elem_bytes(int dtype) { return dtype == SPECDEC_F32 ? 4 : 2; }

bool misaligned(const void *ptr, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(ptr) & (to - 1)) != 0;
}

int token_status(int dtype, int B, int N) {
  if ((dtype != SPECDEC_F32 && dtype != SPECDEC_BF16) || B < 0 || N < 0)
    return SPECDEC_ERR_INVALID_ARG;
  return (long long)B * N > INT_MAX ? SPECDEC_ERR_UNSUPPORTED : SPECDEC_OK;
}

int cache_status(const specdec_kv_cache *c) {
  if (!c) return SPECDEC_ERR_INVALID_ARG;
  if (c->n_blocks < 1 || c->max_blocks < 1 || c->block < 16 || c->block % 16 || c->Hkv < 1 ||
      c->D < 16 || c->D % 16)
    return SPECDEC_ERR_INVALID_ARG;
  if (c->block > SPECDEC_MAX_KV_BLOCK || c->D > SPECDEC_MAX_HEAD_DIM ||
      c->Hkv > SPECDEC_MAX_HEADS || (long long)c->max_blocks * c->block > INT_MAX / 2)
    return SPECDEC_ERR_UNSUPPORTED;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->block_table || !c->length)
    return SPECDEC_ERR_INVALID_ARG;
  if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->k_scale, 4) ||
      misaligned(c->v_scale, 4) || misaligned(c->block_table, 4) || misaligned(c->length, 4))
    return SPECDEC_ERR_INVALID_ARG;
  return SPECDEC_OK;
}

// Whether [a, a + an) and [b, b + bn) share a byte.
bool overlap(const void *a, size_t an, const void *b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

// An output over its input: allowed only element by element (same start, contiguous).
bool bad_overlap(const void *in, long long stride, const void *out, long long tokens, int H, int D,
                 int es) {
  const size_t row = (size_t)H * D * es;
  if (row == 0 || tokens == 0) return false;
  if (in == out) return stride != (long long)H * D;
  return overlap(in, (size_t)(tokens - 1) * stride * es + row, out, (size_t)tokens * row);
}

}  // namespace

extern "C" {

int specdec_rope(const void *q, const void *k, int dtype, long long q_stride, long long k_stride,
                 const uint64_t *freq, const int32_t *positions, const int32_t *base,
                 const int32_t *parent, int B, int N, int Hq, int Hk, int D, int rot,
                 unsigned flags, float magnitude, void *q_out, void *k_out, void *stream) {
  const int st = token_status(dtype, B, N);
  if (st != SPECDEC_OK) return st;
  if (Hq < 1 || Hk < 0 || D < 1 || rot < 2 || rot % 2 || rot > D ||
      (flags & ~(SPECDEC_ROPE_INTERLEAVED | SPECDEC_ROPE_BACKWARD)))
    return SPECDEC_ERR_INVALID_ARG;
  if (D > SPECDEC_MAX_HEAD_DIM || Hq > SPECDEC_MAX_HEADS || Hk > SPECDEC_MAX_HEADS)
    return SPECDEC_ERR_UNSUPPORTED;
  if (q_stride < (long long)Hq * D || (Hk && k_stride < (long long)Hk * D) ||
      (positions && (base || parent)))
    return SPECDEC_ERR_INVALID_ARG;
  if (B == 0 || N == 0) return SPECDEC_OK;
  if (!q || !freq || !q_out || (Hk > 0) != (k != nullptr) || (Hk > 0) != (k_out != nullptr))
    return SPECDEC_ERR_INVALID_ARG;
  const int es = elem_bytes(dtype);
  if (misaligned(q, es) || misaligned(k, es) || misaligned(q_out, es) || misaligned(k_out, es) ||
      misaligned(freq, 8) || misaligned(positions, 4) || misaligned(base, 4) ||
      misaligned(parent, 4))
    return SPECDEC_ERR_INVALID_ARG;
  const long long tokens = (long long)B * N;
  if (bad_overlap(q, q_stride, q_out, tokens, Hq, D, es) ||
      bad_overlap(k, k_stride, k_out, tokens, Hk, D, es) ||
      (Hk && (overlap(q, (size_t)((tokens - 1) * q_stride + Hq * D) * es, k_out,
                      (size_t)tokens * Hk * D * es) ||
              overlap(k, (size_t)((tokens - 1) * k_stride + Hk * D) * es, q_out,
                      (size_t)tokens * Hq * D * es) ||
              overlap(q_out, (size_t)tokens * Hq * D * es, k_out, (size_t)tokens * Hk * D * es))))
    return SPECDEC_ERR_INVALID_ARG;
  RopeParams p;
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_stride = q_stride;
  p.k_stride = Hk ? k_stride : 0;
  p.freq = freq;
  p.positions = positions;
  p.base = base;
  p.parent = parent;
  p.B = B;
  p.N = N;
  p.Hq = Hq;
  p.Hk = Hk;
  p.D = D;
  p.rot = rot;
  p.dtype = dtype;
  p.interleaved = (flags & SPECDEC_ROPE_INTERLEAVED) != 0;
  p.backward = (flags & SPECDEC_ROPE_BACKWARD) != 0;
  p.magnitude = magnitude;
  return cuda_status(launch_rope(p, static_cast<cudaStream_t>(stream)));
}

int specdec_kv_append(const void *k, const void *v, int dtype, long long k_stride,
                      long long v_stride, const int32_t *count, int extra, const int32_t *path,
                      int path_len, const specdec_kv_cache *cache, int B, int N,
                      int32_t *new_length, int32_t *row_status, void *stream) {
  int st = token_status(dtype, B, N);
  if (st != SPECDEC_OK) return st;
  if (B == 0) return SPECDEC_OK;
  st = cache_status(cache);
  if (st != SPECDEC_OK) return st;
  const long long row = (long long)cache->Hkv * cache->D;
  if (k_stride < row || v_stride < row || (path && path_len < 1)) return SPECDEC_ERR_INVALID_ARG;
  if (!new_length || !row_status || new_length == cache->length || (N > 0 && (!k || !v)))
    return SPECDEC_ERR_INVALID_ARG;
  const int es = elem_bytes(dtype);
  if (misaligned(k, es) || misaligned(v, es) || misaligned(count, 4) || misaligned(path, 4) ||
      misaligned(new_length, 4) || misaligned(row_status, 4))
    return SPECDEC_ERR_INVALID_ARG;
  AppendParams p;
  p.k = k;
  p.v = v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.count = count;
  p.path = path;
  p.extra = extra;
  p.path_len = path_len;
  p.cache = *cache;
  p.B = B;
  p.N = N;
  p.dtype = dtype;
  const int most = path && path_len < N ? path_len : N;
  p.blocks = most > 0 ? (int)((cache->block - 1LL + most + cache->block - 1) / cache->block) : 1;
  p.new_length = new_length;
  p.row_status = row_status;
  if ((long long)B * p.blocks * 2 * cache->Hkv > INT_MAX) return SPECDEC_ERR_UNSUPPORTED;
  return cuda_status(launch_kv_append(p, static_cast<cudaStream_t>(stream)));
}

static int attend_size_status(int B, int N, int Hq, int Hkv, int D, int dtype) {
  const int st = token_status(dtype, B, N);
  if (st != SPECDEC_OK) return st;
  if (Hq < 1 || Hkv < 1 || Hq % Hkv || D < 16 || D % 16) return SPECDEC_ERR_INVALID_ARG;
  if (N > SPECDEC_MAX_TREE_NODES || Hq > SPECDEC_MAX_HEADS || D > SPECDEC_MAX_HEAD_DIM ||
      (long long)B * N * Hq > INT_MAX / 4 || (long long)B * Hkv > INT_MAX / 1024)
    return SPECDEC_ERR_UNSUPPORTED;
  return SPECDEC_OK;
}

size_t specdec_attend_workspace_size(int B, int N, int Hq, int Hkv, int D, int dtype) {
  if (attend_size_status(B, N, Hq, Hkv, D, dtype) != SPECDEC_OK || B == 0 || N == 0) return 0;
  return attend_workspace_bytes(B, N, Hq, Hkv, D, dtype);
}

int specdec_attend(const void *q, const void *k_new, const void *v_new, int dtype,
                   long long q_stride, long long k_stride, long long v_stride,
                   const int32_t *parent, const int32_t *n_nodes, const specdec_kv_cache *cache,
                   int B, int N, int Hq, float scale, float softcap, const float *slopes,
                   int window, void *out, float *lse, int32_t *row_status, void *workspace,
                   size_t workspace_bytes, void *stream) {
  int st = token_status(dtype, B, N);
  if (st != SPECDEC_OK) return st;
  if (!std::isfinite(scale) || !(softcap >= 0.0f) || !std::isfinite(softcap) || window < 0)
    return SPECDEC_ERR_INVALID_ARG;
  if (B == 0 || N == 0) return SPECDEC_OK;
  st = cache_status(cache);
  if (st != SPECDEC_OK) return st;
  st = attend_size_status(B, N, Hq, cache->Hkv, cache->D, dtype);
  if (st != SPECDEC_OK) return st;
  const long long row = (long long)cache->Hkv * cache->D;
  if (q_stride < (long long)Hq * cache->D || k_stride < row || v_stride < row)
    return SPECDEC_ERR_INVALID_ARG;
  if (!q || !k_new || !v_new || !out || !row_status) return SPECDEC_ERR_INVALID_ARG;
  const int es = elem_bytes(dtype);
  if (misaligned(q, es) || misaligned(k_new, es) || misaligned(v_new, es) || misaligned(out, es) ||
      misaligned(parent, 4) || misaligned(n_nodes, 4) || misaligned(slopes, 4) ||
      misaligned(lse, 4) || misaligned(row_status, 4))
    return SPECDEC_ERR_INVALID_ARG;
  const size_t need = attend_workspace_bytes(B, N, Hq, cache->Hkv, cache->D, dtype);
  if (need > 0 && (!workspace || workspace_bytes < need || misaligned(workspace, 16)))
    return SPECDEC_ERR_WORKSPACE;
  AttendParams p = {};
  p.q = q;
  p.k_new = k_new;
  p.v_new = v_new;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.parent = parent;
  p.n_nodes = n_nodes;
  p.cache = *cache;
  p.B = B;
  p.N = N;
  p.Hq = Hq;
  p.G = Hq / cache->Hkv;
  p.dtype = dtype;
  p.scale = scale;
  p.softcap = softcap;
  p.slopes = slopes;
  p.window = window;
  p.out = out;
  p.lse = lse;
  p.row_status = row_status;
  p.part = reinterpret_cast<float *>(workspace);
  return cuda_status(launch_attend(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
