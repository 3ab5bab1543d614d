// C ABI of the draft side of the step: argument checks and launches of specdec_sample,
// specdec_top_logits and specdec_distill (include/specdec.h).  Like the verify calls these
// are asynchronous, allocate nothing and check their arguments before any device work.
#include <climits>
#include <cmath>
#include <initializer_list>

#include "draft_common.cuh"

using namespace specdec;

namespace {

int cuda_status(cudaError_t e) { return e == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA; }

int elem_bytes(int dtype) { return dtype == SPECDEC_F32 ? 4 : 2; }

bool misaligned(const void *ptr, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(ptr) & (to - 1)) != 0;
}

bool words_misaligned(std::initializer_list<const void *> words) {
  for (const void *w : words)
    if (misaligned(w, 4)) return true;
  return false;
}

int rows_status(int dtype, int B, int R, int V, int most) {
  if ((dtype != SPECDEC_F32 && dtype != SPECDEC_BF16) || B < 0 || R < 1 || V < 1)
    return SPECDEC_ERR_INVALID_ARG;
  if (V > most || (long long)B * R > INT_MAX / kMaxCluster) return SPECDEC_ERR_UNSUPPORTED;
  return SPECDEC_OK;
}

bool temperature_bad(float T) { return !(T >= 0x1p-20f && T <= 0x1p20f); }

// More bytes than any address space has, and few enough for the kernels' offsets of 64 bits.
constexpr __int128 kMostBytes = (__int128)1 << 56;

// Strides under which the rows of V elements share none: rows of a request together, or
// the requests' rows of one number together.  A single row's or request's stride is not used.
bool strides_bad(int B, int R, int V, RowsAt at, int es) {
  const __int128 request = B > 1 ? at.request : 0, row = R > 1 ? at.row : 0;
  if (request < 0 || row < 0) return true;
  const __int128 requests = (B > 1 ? B - 1 : 0) * request, rows = (R - 1) * row;
  if ((requests + rows + V) * es > kMostBytes) return true;
  const bool by_request = (R == 1 || row >= V) && (B <= 1 || request >= rows + V);
  const bool by_row = (B <= 1 || request >= V) && (R == 1 || row >= requests + V);
  return !by_request && !by_row;
}

size_t extent(int B, int R, int V, RowsAt at, int es) {
  return (size_t)((B - 1) * at.request + (R - 1) * at.row + V) * es;
}

// Rows written over rows that are read: element by element, or apart.
bool bad_overlap(const void *in, const void *out, int B, int R, int V, int es, RowsAt i, RowsAt o) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(in), y = reinterpret_cast<uintptr_t>(out);
  if (x == y) return (B > 1 && i.request != o.request) || (R > 1 && i.row != o.row);
  return x < y + extent(B, R, V, o, es) && y < x + extent(B, R, V, i, es);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

size_t top_part_bytes(long long rows, int V, int dtype) {
  return align256((size_t)rows * stages_per_row(V, elem_bytes(dtype)) * sizeof(float2));
}

// Checks of both distillation calls, and their common parameters.
int distill_params(DistillParams &p, const void *logits, int dtype, RowsAt at, const int32_t *ids,
                   const float *teacher, const float *lse, const float *weight, float temperature,
                   int B, int R, int V, int K, void *grad, RowsAt grad_at) {
  const int st = rows_status(dtype, B, R, V, SPECDEC_MAX_DRAFT_V);
  if (st != SPECDEC_OK) return st;
  if (K < 1 || temperature_bad(temperature) || strides_bad(B, R, V, at, elem_bytes(dtype)) ||
      (grad && strides_bad(B, R, V, grad_at, elem_bytes(dtype))))
    return SPECDEC_ERR_INVALID_ARG;
  if (K > SPECDEC_MAX_TOPK) return SPECDEC_ERR_UNSUPPORTED;
  if (B == 0) return SPECDEC_OK;
  if (!logits || !ids || !teacher) return SPECDEC_ERR_INVALID_ARG;
  const int es = elem_bytes(dtype);
  if (misaligned(logits, es) || misaligned(grad, es) || words_misaligned({ids, teacher, lse, weight}))
    return SPECDEC_ERR_INVALID_ARG;
  if (grad && bad_overlap(logits, grad, B, R, V, es, at, grad_at)) return SPECDEC_ERR_INVALID_ARG;
  p.x = logits;
  p.x_at = at;
  p.ids = ids;
  p.teacher = teacher;
  p.lse = lse;
  p.weight = weight;
  p.temperature = temperature;
  p.inv_t = (float)(1.0 / (double)temperature);
  p.inv_t_low = (float)(1.0 / (double)temperature - (double)p.inv_t);
  p.dtype = dtype;
  p.B = B;
  p.R = R;
  p.V = V;
  p.K = K;
  p.grad = grad;
  p.grad_at = grad_at;
  return SPECDEC_OK;
}

}  // namespace

extern "C" {

int specdec_sample(const void *logits, int dtype, long long request_stride, long long row_stride,
                   const float *temperature, const int32_t *top_k, const float *top_p,
                   const float *min_p, const float *uniforms, int B, int R, int V, int S,
                   unsigned flags, int32_t *tokens, void *rows, long long rows_request_stride,
                   long long rows_row_stride, int32_t *kept, int32_t *row_status, void *stream) {
  const int st = rows_status(dtype, B, R, V, SPECDEC_MAX_DRAFT_V);
  if (st != SPECDEC_OK) return st;
  SampleParams p = {};
  p.x_at = {request_stride, row_stride};
  p.rows_at = {rows_request_stride, rows_row_stride};
  if (S < 0 || (flags & ~SPECDEC_SAMPLE_LOGITS) || strides_bad(B, R, V, p.x_at, elem_bytes(dtype)) ||
      (rows && strides_bad(B, R, V, p.rows_at, elem_bytes(dtype))))
    return SPECDEC_ERR_INVALID_ARG;
  if (S > SPECDEC_MAX_DRAWS) return SPECDEC_ERR_UNSUPPORTED;
  if (B == 0) return SPECDEC_OK;
  if (!logits || !temperature || !kept || !row_status || (S > 0 && (!uniforms || !tokens)))
    return SPECDEC_ERR_INVALID_ARG;
  const int es = elem_bytes(dtype);
  if (misaligned(logits, es) || misaligned(rows, es) ||
      words_misaligned({temperature, top_k, top_p, min_p, uniforms, tokens, kept, row_status}))
    return SPECDEC_ERR_INVALID_ARG;
  if (rows && bad_overlap(logits, rows, B, R, V, es, p.x_at, p.rows_at)) return SPECDEC_ERR_INVALID_ARG;
  p.x = logits;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.uniforms = uniforms;
  p.dtype = dtype;
  p.B = B;
  p.R = R;
  p.V = V;
  p.S = S;
  p.tokens = tokens;
  p.rows = rows;
  p.logits = (flags & SPECDEC_SAMPLE_LOGITS) != 0;
  p.kept = kept;
  p.row_status = row_status;
  return cuda_status(launch_sample(p, static_cast<cudaStream_t>(stream)));
}

size_t specdec_top_logits_workspace_size(int B, int R, int V, int dtype) {
  if (rows_status(dtype, B, R, V, SPECDEC_MAX_V) != SPECDEC_OK || B == 0) return 0;
  const long long rows = (long long)B * R;
  return top_part_bytes(rows, V, dtype) +
         align256((size_t)rows * stages_per_row(V, elem_bytes(dtype)) * kTopGroups *
                    sizeof(float));
}

int specdec_top_logits(const void *logits, int dtype, long long request_stride,
                       long long row_stride, float temperature, int B, int R, int V, int K,
                       float *values, int32_t *ids, float *lse, int32_t *row_status,
                       void *workspace, size_t workspace_bytes, void *stream) {
  const int st = rows_status(dtype, B, R, V, SPECDEC_MAX_V);
  if (st != SPECDEC_OK) return st;
  TopParams p = {};
  p.x_at = {request_stride, row_stride};
  if (K < 1 || K > V || temperature_bad(temperature) ||
      strides_bad(B, R, V, p.x_at, elem_bytes(dtype)))
    return SPECDEC_ERR_INVALID_ARG;
  if (K > SPECDEC_MAX_TOPK) return SPECDEC_ERR_UNSUPPORTED;
  if (B == 0) return SPECDEC_OK;
  if (!logits || !values || !ids || !lse || !row_status) return SPECDEC_ERR_INVALID_ARG;
  if (misaligned(logits, elem_bytes(dtype)) || words_misaligned({values, ids, lse, row_status}))
    return SPECDEC_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < specdec_top_logits_workspace_size(B, R, V, dtype) ||
      misaligned(workspace, 16))
    return SPECDEC_ERR_WORKSPACE;
  p.x = logits;
  p.temperature = temperature;
  p.inv_t = (float)(1.0 / (double)temperature);
  p.inv_t_low = (float)(1.0 / (double)temperature - (double)p.inv_t);
  p.dtype = dtype;
  p.B = B;
  p.R = R;
  p.V = V;
  p.K = K;
  p.spr = stages_per_row(V, elem_bytes(dtype));
  p.part = reinterpret_cast<float2 *>(workspace);
  p.group = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(workspace) +
                                      top_part_bytes((long long)B * R, V, dtype));
  p.values = values;
  p.ids = ids;
  p.lse = lse;
  p.row_status = row_status;
  return cuda_status(launch_top_logits(p, static_cast<cudaStream_t>(stream)));
}

int specdec_distill(const void *logits, int dtype, long long request_stride, long long row_stride,
                    const int32_t *ids, const float *teacher, const float *teacher_lse,
                    const float *weight, float temperature, int B, int R, int V, int K,
                    float *loss, void *grad, long long grad_request_stride,
                    long long grad_row_stride, int32_t *row_status, void *stream) {
  DistillParams p = {};
  const int st = distill_params(p, logits, dtype, {request_stride, row_stride}, ids, teacher,
                                teacher_lse, weight, temperature, B, R, V, K, grad,
                                {grad_request_stride, grad_row_stride});
  if (st != SPECDEC_OK || B == 0) return st;
  if (!loss || !row_status || words_misaligned({loss, row_status})) return SPECDEC_ERR_INVALID_ARG;
  p.loss = loss;
  p.row_status = row_status;
  return cuda_status(launch_distill(p, static_cast<cudaStream_t>(stream)));
}

int specdec_distill_backward(const void *logits, int dtype, long long request_stride,
                             long long row_stride, const int32_t *ids, const float *teacher,
                             const float *teacher_lse, const float *weight, const float *dloss,
                             float temperature, int B, int R, int V, int K, void *grad,
                             long long grad_request_stride, long long grad_row_stride,
                             void *stream) {
  DistillParams p = {};
  const int st = distill_params(p, logits, dtype, {request_stride, row_stride}, ids, teacher,
                                teacher_lse, weight, temperature, B, R, V, K, grad,
                                {grad_request_stride, grad_row_stride});
  if (st != SPECDEC_OK || B == 0) return st;
  // (over the logits, a second look would read the gradient)
  if (!grad || grad == logits || !dloss || misaligned(dloss, 4)) return SPECDEC_ERR_INVALID_ARG;
  p.dloss = dloss;
  return cuda_status(launch_distill(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
