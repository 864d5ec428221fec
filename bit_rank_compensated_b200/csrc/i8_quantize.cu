// Int8 rows with one scale each, of X or of X under a smoothing of its columns. Bound by memory: a row of
// up to 16384 values is read once into the registers of a block (row.cuh), which finds its maximum and
// writes its codes; a longer one is read a second time, from L2.
#include "block.h"
#include "common.cuh"
#include "row.cuh"

namespace svdq {
namespace {

// Rows in flight, and threads on an SM (registers for the row and its smoothing).
constexpr int kDepth = 2;
template <typename T, int TEAM, int VEC, int E, bool FULL>
using Ahead = RowsAhead<T, TEAM, VEC, E, FULL, kDepth>;
constexpr int kQuantThreads = 1024;

template <typename T, int TEAM, int E, int VEC, bool FULL>
__global__ void __launch_bounds__(TEAM, blocks_per_sm(TEAM, kQuantThreads)) k_quantize_rows(QuantRowsLaunch a, int rows_per_block) {
  __shared__ BlockMax<TEAM> top;
  top.clear();
  grid_dep_wait();
  grid_dep_launch();
  uint32_t turn = 0;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * rows_per_block;
  const int64_t m1 = m0 + rows_per_block < a.M ? m0 + rows_per_block : a.M;
  const T *x0 = static_cast<const T *>(a.X);
  extern __shared__ __align__(16) uint8_t ring[];
  Ahead<T, TEAM, VEC, E, FULL> ahead;
#pragma unroll
  for (int d = 0; d < kDepth; ++d) {
    ahead.start(ring, d, x0, a.x_stride, m0, m1, a.K);
    copies_commit();
  }
  f32x2 c[E / 2];
  if (a.col_scale) load_params<TEAM, VEC, E, FULL>(a.col_scale, SVDQ_F32, 0, a.K, 0.0f, c);
  auto write = [&]<bool SHORT>(int64_t m, const f32x2(&x)[E / 2], uint32_t most) {
    const RowScale r = row_scale<SHORT>(most);
    if (threadIdx.x == 0) a.x_scale[m] = scale_of(r);
    store_codes<TEAM, VEC, E, FULL, SHORT>(a.xq + static_cast<size_t>(m) * a.K, a.K, x, r);
  };
  int slot = 0;
  for (int64_t m = m0; m < m1; ++m) {
    f32x2 x[E / 2];
    copies_wait<kDepth - 1>();
    ahead.take(slot, a.K, x);
    if (a.col_scale) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) x[i] = mul2(x[i], c[i]);
    }
    const uint32_t most = top(thread_top(x), turn);
    ahead.refill(slot, x0, a.x_stride, m, m1, a.K);
    copies_commit();
    slot = slot + 1 == kDepth ? 0 : slot + 1;
    if (sizeof(T) == 2 && !a.col_scale) write.template operator()<true>(m, x, most);
    else write.template operator()<false>(m, x, most);
  }
}

// Rows of more than 16384 values, read twice (the second time from L2), value by value. Such rows are weights, once,
// or one long reduction: 1024 x 20000 of bf16 in 30 us (2.0 TB/s; 1024 x 16384 by the kernel above in 11, 4.4 TB/s),
// one row of 131072 in 30 us by its one block.
template <typename T>
__global__ void __launch_bounds__(1024) k_quantize_long_rows(QuantRowsLaunch a) {
  __shared__ BlockMax<1024> top;
  const size_t m = blockIdx.x;
  const T *x = static_cast<const T *>(a.X) + m * a.x_stride;
  auto value = [&](int k) { return a.col_scale ? __fmul_rn(to_f32(x[k]), a.col_scale[k]) : to_f32(x[k]); };
  uint32_t t = 0, turn = 0;
  for (int k = threadIdx.x; k < a.K; k += 1024) t = max(t, __float_as_uint(value(k)) & 0x7fffffffu);
  const RowScale r = row_scale<false>(top(t, turn));
  if (threadIdx.x == 0) a.x_scale[m] = scale_of(r);
  for (int k = threadIdx.x; k < a.K; k += 1024) a.xq[m * a.K + k] = static_cast<int8_t>(i8_code(value(k), r));
}

template <typename T>
cudaError_t quantize_t(const QuantRowsLaunch &a) {
  if (a.K > kMaxRow) {
    return launch(k_quantize_long_rows<T>, dim3(a.M), 1024, 0, a.stream, a);
  }
  const bool vec = a.K % kVec<T> == 0 && rows_aligned(a.X, a.M > 1 ? a.x_stride : 0, sizeof(T), 16) &&
                   rows_aligned(a.col_scale, 0, 4, 16);
  return for_row(a.K, [&]<int TEAM, int E>() {
    const int threads = vec ? row_threads(a.K, E) : TEAM;
    const int blocks = a.num_sms * blocks_per_sm(threads, kQuantThreads);
    const int rows = (a.M + blocks - 1) / blocks;
    const dim3 grid((a.M + rows - 1) / rows);
    auto kern = !vec                 ? k_quantize_rows<T, TEAM, E, 1, false>
                : row_full(a.K, E) ? k_quantize_rows<T, TEAM, E, kVec<T>, true>
                                   : k_quantize_rows<T, TEAM, E, kVec<T>, false>;
    using Ring = Ahead<T, TEAM, kVec<T>, E, true>;
    const int smem = vec ? Ring::bytes(threads) : 0;
    const cudaError_t e = vec ? allow_smem<Ring::bytes(TEAM)>(kern) : cudaSuccess;
    return e != cudaSuccess ? e : launch_dependent(kern, grid, threads, smem, a.stream, a, rows);
  });
}

}  // namespace

cudaError_t launch_i8_quantize_rows(const QuantRowsLaunch &a) {
  if (a.dtype == SVDQ_F32) return quantize_t<float>(a);
  if (a.dtype == SVDQ_F16) return quantize_t<__half>(a);
  return quantize_t<__nv_bfloat16>(a);
}

}  // namespace svdq
