// Layer norm with a weight and a bias for each group of rows, its int8 output form and its gradient.
#include "block.h"
#include "i8_quant.cuh"
#include "types.cuh"

namespace svdq {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += part[w];
  return s;
}

__device__ __forceinline__ float param(const void *p, int dtype, size_t i) {
  if (dtype == SVDQ_F32) return static_cast<const float *>(p)[i];
  if (dtype == SVDQ_F16) return to_f32(static_cast<const __half *>(p)[i]);
  return to_f32(static_cast<const __nv_bfloat16 *>(p)[i]);
}

struct RowStats {
  float mean, rstd;
};

template <typename T>
__device__ RowStats row_stats(const T *x, int K, float eps) {
  float s = 0.0f;
  for (int k = threadIdx.x; k < K; k += kThreads) s += to_f32(x[k]);
  const float mean = block_sum(s) / K;
  float q = 0.0f;
  for (int k = threadIdx.x; k < K; k += kThreads) {
    const float d = to_f32(x[k]) - mean;
    q = fmaf(d, d, q);
  }
  return {mean, 1.0f / sqrtf(block_sum(q) / K + eps)};
}

__device__ __forceinline__ float affine(const NormLaunch &a, size_t g, int k, float xhat) {
  const float w = a.weight ? a.weight_offset + param(a.weight, a.param_dtype, g * a.weight_stride + k) : 1.0f;
  const float b = a.bias ? param(a.bias, a.param_dtype, g * a.bias_stride + k) : 0.0f;
  return fmaf(xhat, w, b);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_layer_norm(NormLaunch a) {
  const size_t m = blockIdx.x, g = m / a.rows_per_group;
  const T *x = static_cast<const T *>(a.X) + m * a.x_stride;
  const RowStats s = row_stats(x, a.K, a.eps);
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[m] = s.mean;
    if (a.rstd) a.rstd[m] = s.rstd;
  }
  T *y = static_cast<T *>(a.Y) + m * a.y_stride;
  for (int k = threadIdx.x; k < a.K; k += kThreads)
    y[k] = from_f32<T>(affine(a, g, k, (to_f32(x[k]) - s.mean) * s.rstd));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_layer_norm_quantize(NormLaunch a) {
  const size_t m = blockIdx.x, g = m / a.rows_per_group;
  const T *x = static_cast<const T *>(a.X) + m * a.x_stride;
  const RowStats s = row_stats(x, a.K, a.eps);
  uint32_t top = 0;
  for (int k = threadIdx.x; k < a.K; k += kThreads)
    top = max(top, abs_bits(affine(a, g, k, (to_f32(x[k]) - s.mean) * s.rstd)));
  const RowScale r = row_scale(block_max<kThreads>(top));
  if (threadIdx.x == 0) a.x_scale[m] = r.scale;
  int8_t *q = a.xq + m * a.K;
  for (int k = threadIdx.x; k < a.K; k += kThreads)
    q[k] = i8_code(affine(a, g, k, (to_f32(x[k]) - s.mean) * s.rstd), r);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_layer_norm_dx(NormLaunch a) {
  const size_t m = blockIdx.x, g = m / a.rows_per_group;
  const T *x = static_cast<const T *>(a.X) + m * a.x_stride;
  const T *dy = static_cast<const T *>(a.dY) + m * a.dy_stride;
  T *dx = static_cast<T *>(a.dX) + m * a.dx_stride;
  const float mean = a.mean[m], rstd = a.rstd[m];
  auto gy = [&](int k) {
    const float w = a.weight ? a.weight_offset + param(a.weight, a.param_dtype, g * a.weight_stride + k) : 1.0f;
    return to_f32(dy[k]) * w;
  };
  float s0 = 0.0f, s1 = 0.0f;
  for (int k = threadIdx.x; k < a.K; k += kThreads) {
    const float v = gy(k);
    s0 += v;
    s1 = fmaf(v, (to_f32(x[k]) - mean) * rstd, s1);
  }
  const float m0 = block_sum(s0) / a.K, m1 = block_sum(s1) / a.K;
  for (int k = threadIdx.x; k < a.K; k += kThreads)
    dx[k] = from_f32<T>(rstd * (gy(k) - m0 - (to_f32(x[k]) - mean) * rstd * m1));
}

// One thread per column and group.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_layer_norm_dparam(NormLaunch a) {
  const int k = blockIdx.x * kThreads + threadIdx.x;
  if (k >= a.K) return;
  const size_t g = blockIdx.y;
  const size_t m0 = g * a.rows_per_group, m1 = min(static_cast<size_t>(a.M), m0 + a.rows_per_group);
  float w = 0.0f, b = 0.0f;
  for (size_t m = m0; m < m1; ++m) {
    const float dy = to_f32(static_cast<const T *>(a.dY)[m * a.dy_stride + k]);
    const float x = to_f32(static_cast<const T *>(a.X)[m * a.x_stride + k]);
    w = fmaf(dy, (x - a.mean[m]) * a.rstd[m], w);
    b += dy;
  }
  if (a.dweight) a.dweight[g * a.K + k] = w;
  if (a.dbias) a.dbias[g * a.K + k] = b;
}

template <typename T>
cudaError_t backward_t(const NormLaunch &a) {
  // the sums first: dX may overwrite dY or X
  if (a.dweight || a.dbias)
    k_layer_norm_dparam<T><<<dim3((a.K + kThreads - 1) / kThreads, a.groups), kThreads, 0, a.stream>>>(a);
  if (a.dX && a.M > 0) k_layer_norm_dx<T><<<a.M, kThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_layer_norm(const NormLaunch &a) {
  if (a.dtype == SVDQ_F32) k_layer_norm<float><<<a.M, kThreads, 0, a.stream>>>(a);
  else if (a.dtype == SVDQ_F16) k_layer_norm<__half><<<a.M, kThreads, 0, a.stream>>>(a);
  else k_layer_norm<__nv_bfloat16><<<a.M, kThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_layer_norm_quantize(const NormLaunch &a) {
  if (a.dtype == SVDQ_F32) k_layer_norm_quantize<float><<<a.M, kThreads, 0, a.stream>>>(a);
  else if (a.dtype == SVDQ_F16) k_layer_norm_quantize<__half><<<a.M, kThreads, 0, a.stream>>>(a);
  else k_layer_norm_quantize<__nv_bfloat16><<<a.M, kThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

size_t layer_norm_partial_bytes(int, int, int, int) { return 0; }

cudaError_t launch_layer_norm_backward(const NormLaunch &a) {
  if (a.dtype == SVDQ_F32) return backward_t<float>(a);
  if (a.dtype == SVDQ_F16) return backward_t<__half>(a);
  return backward_t<__nv_bfloat16>(a);
}

}  // namespace svdq
