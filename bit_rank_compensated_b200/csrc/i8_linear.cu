// 8-bit linear: int8 rows with one scale each, and their product.
#include "block.h"
#include "i8_quant.cuh"
#include "types.cuh"

namespace svdq {
namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads) k_quantize_rows(QuantRowsLaunch a) {
  const size_t m = blockIdx.x;
  const T *x = static_cast<const T *>(a.X) + m * a.x_stride;
  auto value = [&](int k) { return a.col_scale ? __fmul_rn(to_f32(x[k]), a.col_scale[k]) : to_f32(x[k]); };
  uint32_t top = 0;
  for (int k = threadIdx.x; k < a.K; k += kThreads) top = max(top, abs_bits(value(k)));
  const RowScale r = row_scale(block_max<kThreads>(top));
  if (threadIdx.x == 0) a.x_scale[m] = r.scale;
  for (int k = threadIdx.x; k < a.K; k += kThreads) a.xq[m * a.K + k] = i8_code(value(k), r);
}

// Y[m, n] from the integer sum: scaled in fp32, rounded once.
__device__ __forceinline__ float scaled(int acc, float xs, float ws, float b) {
  return fmaf(__fmul_rn(static_cast<float>(acc), xs), ws, b);
}

// 64 x 64 tile, 16 bytes of K at a time, 4 x 4 sums per thread.
template <typename T>
__global__ void __launch_bounds__(256) k_gemm(I8GemmLaunch a) {
  __shared__ int xs[64][5], ws[64][5];
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int r = threadIdx.x >> 2, c = threadIdx.x & 3;
  int acc[4][4] = {};
  for (int k = 0; k < a.K; k += 16) {
    const int m = m0 + r, n = n0 + r;
    xs[r][c] = m < a.M ? reinterpret_cast<const int *>(a.xq + static_cast<size_t>(m) * a.K + k)[c] : 0;
    ws[r][c] = n < a.N ? reinterpret_cast<const int *>(a.wq + static_cast<size_t>(n) * a.K + k)[c] : 0;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(xs[ty + 16 * i][e], ws[tx + 16 * j][e], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < a.M && n < a.N)
        static_cast<T *>(a.Y)[static_cast<size_t>(m) * a.N + n] =
            from_f32<T>(scaled(acc[i][j], a.x_scale[m], a.w_scale[n], a.bias ? a.bias[n] : 0.0f));
    }
}

}  // namespace

cudaError_t launch_i8_quantize_rows(const QuantRowsLaunch &a) {
  if (a.dtype == SVDQ_F32) k_quantize_rows<float><<<a.M, kThreads, 0, a.stream>>>(a);
  else if (a.dtype == SVDQ_F16) k_quantize_rows<__half><<<a.M, kThreads, 0, a.stream>>>(a);
  else k_quantize_rows<__nv_bfloat16><<<a.M, kThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

size_t i8_gemm_workspace_bytes(int, int, int) { return 0; }

cudaError_t launch_i8_gemm(const I8GemmLaunch &a) {
  const dim3 grid((a.N + 63) / 64, (a.M + 63) / 64);
  if (a.y_dtype == SVDQ_F32) k_gemm<float><<<grid, 256, 0, a.stream>>>(a);
  else if (a.y_dtype == SVDQ_F16) k_gemm<__half><<<grid, 256, 0, a.stream>>>(a);
  else k_gemm<__nv_bfloat16><<<grid, 256, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace svdq
