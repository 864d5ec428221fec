// Int8 rows with one scale each, of X or of X under a smoothing of its columns.
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

}  // namespace

cudaError_t launch_i8_quantize_rows(const QuantRowsLaunch &a) {
  if (a.dtype == SVDQ_F32) k_quantize_rows<float><<<a.M, kThreads, 0, a.stream>>>(a);
  else if (a.dtype == SVDQ_F16) k_quantize_rows<__half><<<a.M, kThreads, 0, a.stream>>>(a);
  else k_quantize_rows<__nv_bfloat16><<<a.M, kThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace svdq
