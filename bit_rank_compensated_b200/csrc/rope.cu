// Rotary positions with several axes: the (cos, sin) table and the rotation of Q and K heads.
#include "block.h"
#include "types.cuh"

namespace svdq {
namespace {

constexpr double kTwoPi = 6.283185307179586476925;

// (cos, sin) of pair p of token m. The angle is formed and brought into [-pi, pi] in fp64: a far
// position times a frequency has no fraction left in fp32.
__device__ __forceinline__ float2 turn(const svdq_positions &pos, const svdq_rope_axes &ax, int P, size_t m, int p) {
  int axis = 0, i = p;
  while (i >= ax.pairs[axis]) i -= ax.pairs[axis++];
  const double power = ax.shared_ladder ? static_cast<double>(p) / P : static_cast<double>(i) / ax.pairs[axis];
  const size_t at = m * pos.token_stride + axis * pos.axis_stride;
  const double v = pos.dtype == SVDQ_I64   ? static_cast<double>(static_cast<const int64_t *>(pos.data)[at])
                   : pos.dtype == SVDQ_I32 ? static_cast<double>(static_cast<const int32_t *>(pos.data)[at])
                                           : static_cast<double>(static_cast<const float *>(pos.data)[at]);
  const double angle = v * exp2(-power * log2(static_cast<double>(ax.theta)));
  const float r = static_cast<float>(fma(-kTwoPi, rint(angle * (1.0 / kTwoPi)), angle));
  float2 cs;
  sincosf(r, &cs.y, &cs.x);
  return cs;
}

__global__ void __launch_bounds__(256) k_rope_table(RopeLaunch a) {
  const size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<size_t>(a.M) * a.n_pairs) return;
  reinterpret_cast<float2 *>(a.table)[i] = turn(a.pos, a.axes, a.n_pairs, i / a.n_pairs, static_cast<int>(i % a.n_pairs));
}

// One block per token, one thread per pair of a head or pair of columns behind the rotated ones.
template <typename T>
__global__ void __launch_bounds__(256) k_rope_apply(RopeLaunch a) {
  __shared__ float2 cs[256];
  const size_t m = blockIdx.x;
  const int P = a.n_pairs;
  if (static_cast<int>(threadIdx.x) < P) {
    cs[threadIdx.x] = turn(a.pos, a.axes, P, m, threadIdx.x);
    if (a.inverse) cs[threadIdx.x].y = -cs[threadIdx.x].y;
  }
  __syncthreads();
  const int half = a.head_dim / 2;
#pragma unroll
  for (int t = 0; t < 2; ++t)
    for (int i = threadIdx.x; i < a.in[t].heads * half; i += 256) {
      const int h = i / half, p = i % half;
      const T *in = static_cast<const T *>(a.in[t].data) + m * a.in[t].token_stride + h * a.in[t].head_stride;
      T *out = static_cast<T *>(a.out[t].data) + m * a.out[t].token_stride + h * a.out[t].head_stride;
      const int c0 = p < P && a.axes.halves ? p : 2 * p;
      const int c1 = p < P && a.axes.halves ? p + P : 2 * p + 1;
      if (p < P) {
        const float u0 = to_f32(in[c0]), u1 = to_f32(in[c1]);
        out[c0] = from_f32<T>(fmaf(u0, cs[p].x, -__fmul_rn(u1, cs[p].y)));
        out[c1] = from_f32<T>(fmaf(u1, cs[p].x, __fmul_rn(u0, cs[p].y)));
      } else {
        out[c0] = in[c0];
        out[c1] = in[c1];
      }
    }
}

}  // namespace

cudaError_t launch_rope_table(const RopeLaunch &a) {
  const size_t n = static_cast<size_t>(a.M) * a.n_pairs;
  k_rope_table<<<static_cast<unsigned>((n + 255) / 256), 256, 0, a.stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_rope_apply(const RopeLaunch &a) {
  if (a.dtype == SVDQ_F32) k_rope_apply<float><<<a.M, 256, 0, a.stream>>>(a);
  else if (a.dtype == SVDQ_F16) k_rope_apply<__half><<<a.M, 256, 0, a.stream>>>(a);
  else k_rope_apply<__nv_bfloat16><<<a.M, 256, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace svdq
