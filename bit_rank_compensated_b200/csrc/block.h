// Launch interfaces of the operators around the projections (layer norm, 8-bit linear, rotary
// positions) between their C ABI (api_block.cu) and their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "host.h"
#include "svdq.h"

namespace svdq {

// Pieces of `each` that make up n >= 1 (n + each may pass 31 bits).
constexpr int pieces(int n, int each) { return (n - 1) / each + 1; }

// Rows of X and the weight and bias their layer norm takes.
struct NormLaunch {
  const void *X;
  size_t x_stride;
  int dtype, M, K;
  const void *weight, *bias;  // or null
  size_t weight_stride, bias_stride;
  int param_dtype, groups, rows_per_group;
  float weight_offset, eps;
  // forward
  void *Y;
  size_t y_stride;
  float *mean, *rstd;  // out (forward, may be null) or in (backward)
  // int8 rows instead of Y
  int8_t *xq;
  float *x_scale;
  // backward
  const void *dY;
  size_t dy_stride;
  void *dX;
  size_t dx_stride;
  float *dweight, *dbias;
  float *partial;  // workspace
  int num_sms;
  cudaStream_t stream;
};
cudaError_t launch_layer_norm(const NormLaunch &a);
cudaError_t launch_layer_norm_quantize(const NormLaunch &a);
cudaError_t launch_layer_norm_backward(const NormLaunch &a);
size_t layer_norm_partial_bytes(int M, int K, int rows_per_group);

// int8 rows of X (or of X * col_scale).
struct QuantRowsLaunch {
  const void *X;
  size_t x_stride;
  int dtype, M, K;
  const float *col_scale;
  int8_t *xq;
  float *x_scale;
  int num_sms;
  cudaStream_t stream;
};
cudaError_t launch_i8_quantize_rows(const QuantRowsLaunch &a);

// Y = (xq wq^T) x_scale w_scale + bias.
struct I8GemmLaunch {
  const int8_t *xq, *wq;
  const float *x_scale, *w_scale, *bias;
  int M, N, K;
  void *Y;
  int y_dtype;
  void *workspace;
  const DeviceState *dev;
  cudaStream_t stream;
};
cudaError_t launch_i8_gemm(const I8GemmLaunch &a);
// The same of up to eight tokens, from int8 rows or floating ones: whether they are few, and whether their rows are
// quantized where they are multiplied.
bool i8_few_fits(int M, int N, int K);
bool i8_few_quantizes(const QuantRowsLaunch &q);
cudaError_t launch_i8_few(const I8GemmLaunch &a);
cudaError_t launch_i8_few_quantized(const QuantRowsLaunch &q, const I8GemmLaunch &a);
size_t i8_gemm_workspace_bytes(int M, int N, int K);

// Rotary positions: table, or the heads' rotation.
struct RopeLaunch {
  svdq_positions pos;
  svdq_rope_axes axes;
  double log2_theta;
  int n_pairs;
  int M;
  float *table;
  svdq_heads in[2], out[2];  // Q and K (heads 0: none)
  int dtype, head_dim;
  bool inverse;
  int num_sms;
  cudaStream_t stream;
};
cudaError_t launch_rope_table(const RopeLaunch &a);
cudaError_t launch_rope_apply(const RopeLaunch &a);

// A call's error, on its way to the caller. The runtime keeps a failed call's error for whoever asks for the last one
// next, which would be another call, whose own launch succeeded.
inline cudaError_t reported(cudaError_t e) {
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

// Lets a kernel have up to MOST bytes of dynamic shared memory on the current device: the most that any launch
// of it takes, never one call's. The attribute belongs to the process, and what a thread sets replaces what another
// one did, so that a smaller call would take from a larger one; with one value setting it again is harmless.
// It costs the host some 3 us, so a thread remembers what it has set (a slot per kernel and device, lost to another
// one at worst).
template <int MOST, typename... Args>
cudaError_t allow_smem(void (*kern)(Args...)) {
  if constexpr (MOST <= 40 * 1024) return cudaSuccess;  // within the default, static arrays included
  struct Granted {
    const void *kern;
    int device;
  };
  static thread_local Granted slots[64];
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return reported(e);
  const void *key = reinterpret_cast<const void *>(kern);
  Granted &s = slots[(reinterpret_cast<uintptr_t>(key) / 64 + static_cast<uintptr_t>(device) * 17) % 64];
  if (s.kern == key && s.device == device) return cudaSuccess;
  e = cudaFuncSetAttribute(key, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST);
  if (e == cudaSuccess) s = {key, device};
  return reported(e);
}

// Launches a kernel, after the stream's previous one has ended or (DEPENDENT, below) before.
template <bool DEPENDENT, typename... Args>
cudaError_t launch_kernel(void (*kern)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                          std::type_identity_t<Args>... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = DEPENDENT ? 1 : 0;
  return reported(cudaLaunchKernelEx(&cfg, kern, args...));
}
template <typename... Args>
cudaError_t launch(void (*kern)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t st, std::type_identity_t<Args>... args) {
  return launch_kernel<false>(kern, grid, threads, smem, st, args...);
}
// Of a kernel that waits (grid_dep_wait) before it touches global memory, so that its start may overlap the end of
// the stream's previous kernel.
template <typename... Args>
cudaError_t launch_dependent(void (*kern)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                             std::type_identity_t<Args>... args) {
  return launch_kernel<true>(kern, grid, threads, smem, st, args...);
}

}  // namespace svdq
