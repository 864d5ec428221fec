// C ABI of the operators around the projections (layer norm, 8-bit linear, rotary positions):
// argument checks and launches. Declared and documented in include/svdq.h.
#include <math.h>
#include <string.h>

#include "block.h"

using namespace svdq;

namespace {

constexpr int kMaxRows = 1 << 30;
constexpr int kMaxNormColumns = 16384;
constexpr int kMaxHeads = 65536;
constexpr int kMaxI8Columns = 131072;  // 127 * 127 * K < 2^31

size_t elem_bytes(int dtype) {
  switch (dtype) {
    case SVDQ_BF16:
    case SVDQ_F16: return 2;
    case SVDQ_F32:
    case SVDQ_I32: return 4;
    case SVDQ_I64: return 8;
  }
  return 0;
}

bool is_float(int dtype) { return dtype == SVDQ_BF16 || dtype == SVDQ_F16 || dtype == SVDQ_F32; }

bool aligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

svdq_status done(cudaError_t e) { return e == cudaSuccess ? SVDQ_OK : SVDQ_ERR_CUDA; }

// The arguments that every layer norm call has; fills the shared fields of a.
svdq_status norm_args(const void *X, size_t x_stride, int dtype, int M, int K, const svdq_norm_affine *af, float eps,
                      NormLaunch *a) {
  memset(a, 0, sizeof(*a));
  if (!is_float(dtype) || M < 0 || M > kMaxRows || K < 1 || K > kMaxNormColumns || x_stride < static_cast<size_t>(K))
    return SVDQ_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !isfinite(eps)) return SVDQ_ERR_INVALID_ARG;
  if (!X && M > 0) return SVDQ_ERR_INVALID_ARG;
  a->X = X;
  a->x_stride = x_stride;
  a->dtype = dtype;
  a->M = M;
  a->K = K;
  a->eps = eps;
  a->param_dtype = SVDQ_F32;
  a->groups = 1;
  a->rows_per_group = M > 0 ? M : 1;
  if (af) {
    const size_t k = static_cast<size_t>(K);
    if (!is_float(af->dtype) || af->groups < 1 || af->rows_per_group < 1 ||
        static_cast<int64_t>(af->groups) * af->rows_per_group < M)
      return SVDQ_ERR_INVALID_ARG;
    if ((af->weight && af->groups > 1 && af->weight_stride < k) || (af->bias && af->groups > 1 && af->bias_stride < k))
      return SVDQ_ERR_INVALID_ARG;
    a->weight = af->weight;
    a->bias = af->bias;
    a->weight_stride = af->weight_stride;
    a->bias_stride = af->bias_stride;
    a->param_dtype = af->dtype;
    a->groups = af->groups;
    a->rows_per_group = af->rows_per_group < a->rows_per_group ? af->rows_per_group : a->rows_per_group;  // the same groups
    a->weight_offset = af->weight_offset;
    if (!aligned(af->weight, elem_bytes(af->dtype)) || !aligned(af->bias, elem_bytes(af->dtype)))
      return SVDQ_ERR_MISALIGNED;
  }
  return aligned(X, elem_bytes(dtype)) ? SVDQ_OK : SVDQ_ERR_MISALIGNED;
}

svdq_status check_axes(const svdq_positions *pos, int M, const svdq_rope_axes *ax, RopeLaunch *a) {
  memset(static_cast<void *>(a), 0, sizeof(*a));
  if (!pos || !ax || M < 0 || M > kMaxRows || ax->n_axes < 1 || ax->n_axes > 4) return SVDQ_ERR_INVALID_ARG;
  int P = 0;
  for (int i = 0; i < ax->n_axes; ++i) {
    if (ax->pairs[i] < 1 || ax->pairs[i] > 256) return SVDQ_ERR_INVALID_ARG;
    P += ax->pairs[i];
  }
  if (P > 256 || !(ax->theta > 0.0f) || !isfinite(ax->theta)) return SVDQ_ERR_INVALID_ARG;
  if ((ax->shared_ladder | 1) != 1 || (ax->halves | 1) != 1) return SVDQ_ERR_INVALID_ARG;
  if (pos->dtype != SVDQ_I32 && pos->dtype != SVDQ_I64 && pos->dtype != SVDQ_F32) return SVDQ_ERR_INVALID_ARG;
  if (!pos->data && M > 0) return SVDQ_ERR_INVALID_ARG;
  a->pos = *pos;
  a->axes = *ax;
  a->log2_theta = log2(static_cast<double>(ax->theta));
  a->n_pairs = P;
  a->M = M;
  return aligned(pos->data, elem_bytes(pos->dtype)) ? SVDQ_OK : SVDQ_ERR_MISALIGNED;
}

svdq_status check_gemm(const int8_t *xq, const float *x_scale, int M, const int8_t *wq, const float *w_scale,
                       const float *bias, int N, int K, const void *Y, int y_dtype, const void *workspace,
                       size_t workspace_bytes) {
  if (!is_float(y_dtype) || M < 0 || M > kMaxRows || N < 16 || N % 16 || K < 16 || K % 16 || K > kMaxI8Columns)
    return SVDQ_ERR_INVALID_ARG;
  if (!wq || !w_scale || (M > 0 && (!xq || !x_scale || !Y))) return SVDQ_ERR_INVALID_ARG;
  const size_t need = svdq_i8_workspace_bytes(M, N, K);
  if (need > 0 && (!workspace || workspace_bytes < need)) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(xq) || !aligned16(wq) || !aligned16(Y) || !aligned16(workspace) || !aligned(x_scale, 4) ||
      !aligned(w_scale, 4) || !aligned(bias, 4))
    return SVDQ_ERR_MISALIGNED;
  return SVDQ_OK;
}

svdq_status check_quantize(const void *X, size_t x_stride, int dtype, int M, int K, const float *col_scale,
                           const int8_t *xq, const float *x_scale) {
  if (!is_float(dtype) || M < 0 || M > kMaxRows || K < 16 || K % 16 || K > kMaxI8Columns || x_stride < static_cast<size_t>(K))
    return SVDQ_ERR_INVALID_ARG;
  if (M > 0 && (!X || !xq || !x_scale)) return SVDQ_ERR_INVALID_ARG;
  if (!aligned(X, elem_bytes(dtype)) || !aligned(col_scale, 4) || !aligned16(xq) || !aligned(x_scale, 4))
    return SVDQ_ERR_MISALIGNED;
  return SVDQ_OK;
}

svdq_status check_heads(const svdq_heads *in, const svdq_heads *out, int M, int head_dim, size_t e) {
  if (!in || !out || in->heads < 1 || in->heads > kMaxHeads || out->heads != in->heads) return SVDQ_ERR_INVALID_ARG;
  for (const svdq_heads *h : {in, out}) {
    if (!h->data && M > 0) return SVDQ_ERR_INVALID_ARG;
    if (!aligned(h->data, e)) return SVDQ_ERR_MISALIGNED;
  }
  // an output's heads must not overlap, in either order of tokens and heads (an input's may: shared heads)
  const size_t d = static_cast<size_t>(head_dim), t = out->token_stride, h = out->head_stride;
  const size_t tokens = M > 0 ? static_cast<size_t>(M) : 1, heads = static_cast<size_t>(out->heads);
  const bool heads_inside = (heads == 1 || h >= d) && (tokens == 1 || t >= (heads - 1) * h + d);
  const bool tokens_inside = (tokens == 1 || t >= d) && (heads == 1 || h >= (tokens - 1) * t + d);
  if (!heads_inside && !tokens_inside) return SVDQ_ERR_INVALID_ARG;
  return SVDQ_OK;
}

}  // namespace

extern "C" {

svdq_status svdq_layer_norm(const void *X, size_t x_stride, int dtype, int M, int K, const svdq_norm_affine *affine,
                            float eps, void *Y, size_t y_stride, float *mean, float *rstd, void *stream) {
  NormLaunch a;
  svdq_status st = norm_args(X, x_stride, dtype, M, K, affine, eps, &a);
  if (st != SVDQ_OK) return st;
  if ((!Y && M > 0) || y_stride < static_cast<size_t>(K)) return SVDQ_ERR_INVALID_ARG;
  if (!aligned(Y, elem_bytes(dtype)) || !aligned(mean, 4) || !aligned(rstd, 4)) return SVDQ_ERR_MISALIGNED;
  DeviceState *d = nullptr;
  if ((st = device_check(&d)) != SVDQ_OK) return st;
  if (M == 0) return SVDQ_OK;
  a.Y = Y;
  a.y_stride = y_stride;
  a.mean = mean;
  a.rstd = rstd;
  a.num_sms = d->num_sms;
  a.stream = static_cast<cudaStream_t>(stream);
  return done(launch_layer_norm(a));
}

size_t svdq_layer_norm_workspace_bytes(int M, int K, int groups, int rows_per_group) {
  if (M < 1 || M > kMaxRows || K < 1 || K > kMaxNormColumns || groups < 1 || rows_per_group < 1) return 0;
  return layer_norm_partial_bytes(M, K, rows_per_group < M ? rows_per_group : M);
}

svdq_status svdq_layer_norm_backward(const void *dY, size_t dy_stride, const void *X, size_t x_stride, int dtype, int M,
                                     int K, const svdq_norm_affine *affine, const float *mean, const float *rstd,
                                     void *dX, size_t dx_stride, float *dweight, float *dbias, void *workspace,
                                     size_t workspace_bytes, void *stream) {
  NormLaunch a;
  svdq_status st = norm_args(X, x_stride, dtype, M, K, affine, 0.0f, &a);
  if (st != SVDQ_OK) return st;
  const size_t k = static_cast<size_t>(K);
  if (M > 0 && (!dY || !mean || !rstd)) return SVDQ_ERR_INVALID_ARG;
  if (dy_stride < k || (dX && dx_stride < k)) return SVDQ_ERR_INVALID_ARG;
  const size_t need = svdq_layer_norm_workspace_bytes(M, K, a.groups, a.rows_per_group);
  if ((dweight || dbias) && need > 0 && (!workspace || workspace_bytes < need)) return SVDQ_ERR_INVALID_ARG;
  if (!aligned(dY, elem_bytes(dtype)) || !aligned(dX, elem_bytes(dtype)) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(dweight, 4) || !aligned(dbias, 4) || !aligned16(workspace))
    return SVDQ_ERR_MISALIGNED;
  DeviceState *d = nullptr;
  if ((st = device_check(&d)) != SVDQ_OK) return st;
  a.stream = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    const size_t bytes = static_cast<size_t>(a.groups) * k * sizeof(float);
    for (float *p : {dweight, dbias})
      if (p && (st = done(reported(cudaMemsetAsync(p, 0, bytes, a.stream)))) != SVDQ_OK) return st;
    return SVDQ_OK;
  }
  if (!dX && !dweight && !dbias) return SVDQ_OK;
  a.dY = dY;
  a.dy_stride = dy_stride;
  a.mean = const_cast<float *>(mean);
  a.rstd = const_cast<float *>(rstd);
  a.dX = dX;
  a.dx_stride = dx_stride;
  a.dweight = dweight;
  a.dbias = dbias;
  a.partial = static_cast<float *>(workspace);
  a.num_sms = d->num_sms;
  return done(launch_layer_norm_backward(a));
}

svdq_status svdq_i8_quantize_rows(const void *X, size_t x_stride, int dtype, int M, int K, const float *col_scale,
                                  int8_t *xq, float *x_scale, void *stream) {
  svdq_status st = check_quantize(X, x_stride, dtype, M, K, col_scale, xq, x_scale);
  if (st != SVDQ_OK) return st;
  DeviceState *d = nullptr;
  if ((st = device_check(&d)) != SVDQ_OK || M == 0) return st;
  const QuantRowsLaunch a{X, x_stride, dtype, M, K, col_scale, xq, x_scale, d->num_sms, static_cast<cudaStream_t>(stream)};
  return done(launch_i8_quantize_rows(a));
}

svdq_status svdq_i8_layer_norm_quantize(const void *X, size_t x_stride, int dtype, int M, int K,
                                        const svdq_norm_affine *affine, float eps, int8_t *xq, float *x_scale,
                                        void *stream) {
  NormLaunch a;
  svdq_status st = norm_args(X, x_stride, dtype, M, K, affine, eps, &a);
  if (st != SVDQ_OK) return st;
  if (K % 16 || (M > 0 && (!xq || !x_scale))) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(xq) || !aligned(x_scale, 4)) return SVDQ_ERR_MISALIGNED;
  DeviceState *d = nullptr;
  if ((st = device_check(&d)) != SVDQ_OK || M == 0) return st;
  a.xq = xq;
  a.x_scale = x_scale;
  a.num_sms = d->num_sms;
  a.stream = static_cast<cudaStream_t>(stream);
  return done(launch_layer_norm_quantize(a));
}

size_t svdq_i8_workspace_bytes(int M, int N, int K) {
  if (M < 1 || N < 16 || N % 16 || K < 16 || K % 16 || K > kMaxI8Columns) return 0;
  return i8_gemm_workspace_bytes(M, N, K);
}

svdq_status svdq_i8_gemm(const int8_t *xq, const float *x_scale, int M, const int8_t *wq, const float *w_scale,
                         const float *bias, int N, int K, void *Y, int y_dtype, void *workspace, size_t workspace_bytes,
                         void *stream) {
  svdq_status st = check_gemm(xq, x_scale, M, wq, w_scale, bias, N, K, Y, y_dtype, workspace, workspace_bytes);
  if (st != SVDQ_OK) return st;
  DeviceState *d = nullptr;
  if ((st = device_check(&d)) != SVDQ_OK || M == 0) return st;
  const I8GemmLaunch a{xq, wq, x_scale, w_scale, bias, M, N, K, Y, y_dtype, workspace, d,
                       static_cast<cudaStream_t>(stream)};
  return done(launch_i8_gemm(a));
}

svdq_status svdq_i8_linear_forward(const void *X, size_t x_stride, int dtype, int M, const float *col_scale,
                                   const int8_t *wq, const float *w_scale, const float *bias, int N, int K, int8_t *xq,
                                   float *x_scale, void *Y, void *workspace, size_t workspace_bytes, void *stream) {
  svdq_status st = check_gemm(xq, x_scale, M, wq, w_scale, bias, N, K, Y, dtype, workspace, workspace_bytes);
  if (st != SVDQ_OK) return st;
  if (M > 0 && i8_few_fits(M, N, K)) {
    // few tokens and short rows: quantized where they are multiplied, in one launch
    if ((st = check_quantize(X, x_stride, dtype, M, K, col_scale, xq, x_scale)) != SVDQ_OK) return st;
    DeviceState *d = nullptr;
    if ((st = device_check(&d)) != SVDQ_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const QuantRowsLaunch q{X, x_stride, dtype, M, K, col_scale, xq, x_scale, d->num_sms, s};
    const I8GemmLaunch g{xq, wq, x_scale, w_scale, bias, M, N, K, Y, dtype, workspace, d, s};
    if (i8_few_quantizes(q)) return done(launch_i8_few_quantized(q, g));
  }
  st = svdq_i8_quantize_rows(X, x_stride, dtype, M, K, col_scale, xq, x_scale, stream);
  if (st != SVDQ_OK) return st;
  return svdq_i8_gemm(xq, x_scale, M, wq, w_scale, bias, N, K, Y, dtype, workspace, workspace_bytes, stream);
}

svdq_status svdq_rope_axes_table(const svdq_positions *pos, int M, const svdq_rope_axes *axes, float *table,
                                 void *stream) {
  RopeLaunch a;
  svdq_status st = check_axes(pos, M, axes, &a);
  if (st != SVDQ_OK) return st;
  if (!table && M > 0) return SVDQ_ERR_INVALID_ARG;
  if (!aligned(table, 8)) return SVDQ_ERR_MISALIGNED;
  DeviceState *d = nullptr;
  if ((st = device_check(&d)) != SVDQ_OK || M == 0) return st;
  a.table = table;
  a.num_sms = d->num_sms;
  a.stream = static_cast<cudaStream_t>(stream);
  return done(launch_rope_table(a));
}

svdq_status svdq_rope_axes_apply(const svdq_heads *q, const svdq_heads *q_out, const svdq_heads *k,
                                 const svdq_heads *k_out, int dtype, int M, int head_dim, const svdq_positions *pos,
                                 const svdq_rope_axes *axes, int inverse, void *stream) {
  RopeLaunch a;
  svdq_status st = check_axes(pos, M, axes, &a);
  if (st != SVDQ_OK) return st;
  if (!is_float(dtype) || head_dim < 2 || head_dim % 2 || head_dim > 512 || 2 * a.n_pairs > head_dim ||
      (inverse | 1) != 1)
    return SVDQ_ERR_INVALID_ARG;
  if ((st = check_heads(q, q_out, M, head_dim, elem_bytes(dtype))) != SVDQ_OK) return st;
  if (!k != !k_out) return SVDQ_ERR_INVALID_ARG;
  if (k && (st = check_heads(k, k_out, M, head_dim, elem_bytes(dtype))) != SVDQ_OK) return st;
  DeviceState *d = nullptr;
  if ((st = device_check(&d)) != SVDQ_OK || M == 0) return st;
  a.in[0] = *q;
  a.out[0] = *q_out;
  if (k) {
    a.in[1] = *k;
    a.out[1] = *k_out;
  }
  a.dtype = dtype;
  a.head_dim = head_dim;
  a.inverse = inverse != 0;
  a.num_sms = d->num_sms;
  a.stream = static_cast<cudaStream_t>(stream);
  return done(launch_rope_apply(a));
}

}  // extern "C"
