// Layer norm with a weight and a bias for each group of rows, its int8 output form and its gradient.
//
//   xhat = (x - mean) rstd,  y = xhat (offset + w) + b;  dx = rstd (g - mean(g) - xhat mean(g xhat)),
//   g = dy (offset + w);  dw = sum over rows of dy xhat,  db = sum over rows of dy.
//
// All three are bound by memory: one read of each input row and one write of each output row. A row
// lives in the registers of one block (row.cuh), so x is read once although mean, variance (about the
// mean, not from squares), the maximum for int8 and the output each need it; a block walks consecutive
// rows with its columns' weights in registers and the next rows' loads in flight while it reduces the
// present one. Packed fp32 instructions (pair.cuh) keep the issue slots of a row below the time its
// bytes take.
//
// The gradient's column sums run in the same pass: a block adds its rows' dy xhat and dy into registers
// (each thread its own columns: no atomics, a fixed order) and writes one slice of partial sums; a
// second small kernel adds the slices of each group in order.
#include "block.h"
#include "common.cuh"
#include "row.cuh"

namespace svdq {
namespace {

// Rows in flight a block (two, three and four: 27.5, 28.4 and 28.6 us for 9216 x 4096 of bf16).
constexpr int kDepth = 2;
template <typename T, int TEAM, int VEC, int E, bool FULL>
using Ahead = RowsAhead<T, TEAM, VEC, E, FULL, kDepth>;

// Threads on an SM: registers for the row, its weight and bias; a row of 1024 threads has too few for
// that and reads its weights again for every row (from L1).
template <int TEAM>
constexpr int kForwardThreads = TEAM < 1024 ? 768 : 1024;
// So that they fit: by the block's own threads, which may be fewer than TEAM (2000 x 6144 of bf16, two blocks of 384:
// 9.7 us, 13.3 with 96 registers and one of them at a time; 1000 x 8192, one block of 512 in both: 8.6 and 8.4).
template <int TEAM>
constexpr int kForwardRegs = 65536 / kForwardThreads<TEAM> / 8 * 8;
template <int TEAM>
constexpr bool kKeepParams = TEAM < 1024;

// Standard deviations that a row's mean lies from zero before it is corrected. Below, its error of a few 2^-24 is
// as small as that of the other operations.
constexpr float kFarMean = 4.0f;

// Forward: rows [block's first, last) of X; QUANT writes int8 rows and their scales instead of Y.
template <typename T, int TEAM, int E, int VEC, bool FULL, bool QUANT>
__global__ void __launch_bounds__(TEAM) __maxnreg__(kForwardRegs<TEAM>) k_layer_norm(NormLaunch a, int rows_per_block) {
  __shared__ BlockSum<TEAM, 1> sum;
  __shared__ BlockMax<TEAM> top;
  sum.clear();
  if (QUANT) top.clear();
  grid_dep_wait();
  grid_dep_launch();
  uint32_t turn = 0, tmax = 0;
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
  f32x2 w[E / 2], b[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    w[i] = both(1.0f);
    b[i] = 0;
  }
  int64_t group_end = m0;  // first row of the next group
  const float inv_k = 1.0f / a.K;
  int slot = 0;
  for (int64_t m = m0; m < m1; ++m) {
    f32x2 x[E / 2];
    copies_wait<kDepth - 1>();
    ahead.take(slot, a.K, x);
    if (m >= group_end || !kKeepParams<TEAM>) {
      const size_t group = static_cast<uint32_t>(m) / static_cast<uint32_t>(a.rows_per_group);
      group_end = static_cast<int64_t>(group + 1) * a.rows_per_group;
      if (a.weight) load_params<TEAM, VEC, E, FULL>(a.weight, a.param_dtype, group * a.weight_stride, a.K, a.weight_offset, w);
      if (a.bias) load_params<TEAM, VEC, E, FULL>(a.bias, a.param_dtype, group * a.bias_stride, a.K, 0.0f, b);
    }
    float v[1] = {thread_sum(x)};
    sum(v, turn);
    ahead.refill(slot, x0, a.x_stride, m, m1, a.K);
    copies_commit();
    slot = slot + 1 == kDepth ? 0 : slot + 1;
    const float first = v[0] * inv_k;
    const f32x2 minus = both(-first);
    within_row<TEAM, VEC, E, FULL>(a.K, x, [&](f32x2 p, int) { return add2(p, minus); });
    v[0] = thread_dot(x, x);
    sum(v, turn);
    const float var = v[0] * inv_k;
    float mean = first, rstd = rsqrtf(var + a.eps);
    // The mean is a few steps of the values off, which counts where they lie close together far from zero (rstd
    // takes up to eps^-1/2 of it): there the mean of what is left is taken off too. For a row of one value that leaves
    // 0, whatever K: the differences are one small multiple of a step, their sum is exact, and one correction of
    // the quotient gives it back. (In every row, with a sum of two values: 30.0 us for 9216 x 4096 of bf16 against 27.7.
    // Squares compare without a root; where both are below fp32's range the row is corrected, but for the zeros that
    // a batch is padded with.)
    if (kFarMean * kFarMean * var <= first * first && first != 0.0f) [[unlikely]] {
      v[0] = thread_sum(x);
      sum(v, turn);
      const float guess = v[0] * inv_k, off = fmaf(fmaf(-guess, static_cast<float>(a.K), v[0]), inv_k, guess);
      const f32x2 rest = both(-off);
      within_row<TEAM, VEC, E, FULL>(a.K, x, [&](f32x2 p, int) { return add2(p, rest); });
      mean += off;
      rstd = rsqrtf(fmaxf(fmaf(-off, off, var), 0.0f) + a.eps);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[m] = mean;
      if (a.rstd) a.rstd[m] = rstd;
    }
    const f32x2 r2 = both(rstd);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[i] = fma2(mul2(x[i], r2), w[i], b[i]);
    if constexpr (!QUANT) {
      store_row<T, TEAM, VEC, E, FULL>(static_cast<T *>(a.Y) + m * a.y_stride, a.K, x);
    } else {
      // columns from K on are zeros still: their x and b are
      const RowScale r = row_scale<false>(top(thread_top(x), tmax));
      if (threadIdx.x == 0) a.x_scale[m] = scale_of(r);
      store_codes<TEAM, VEC, E, FULL, false>(a.xq + static_cast<size_t>(m) * a.K, a.K, x, r);
    }
  }
}

// Gradient: block (group g, slice s) takes rows [chunk s of the group]. Partial sums go to
// partial[block][2][K], or straight to dweight and dbias where a group has one slice.
// Threads on an SM: registers for x and g of a row, the weight and both sums of its columns (eight values a
// thread and twice the threads were slower: 67 us against 52 for 9216 x 4096).
constexpr int kBackwardThreads = 512;
// Rows of x and dy in flight (16384 fp32 values of each are 128 KiB).
template <typename T, int TEAM>
constexpr int kBackwardDepth = sizeof(T) == 2 ? 3 : (TEAM < 1024 ? 2 : 1);
template <typename T, int TEAM, int VEC, int E, bool FULL>
using BackwardAhead = RowsAhead<T, TEAM, VEC, E, FULL, kBackwardDepth<T, TEAM>>;

template <typename T, int TEAM, int E, int VEC, bool FULL>
__global__ void __launch_bounds__(TEAM, blocks_per_sm(TEAM, kBackwardThreads)) k_layer_norm_backward(NormLaunch a, int slices, int chunk) {
  __shared__ BlockSum<TEAM, 2> sum;
  grid_dep_launch();
  sum.clear();
  uint32_t turn = 0;
  const int group = blockIdx.x / slices, slice = blockIdx.x % slices;
  const int64_t g0 = static_cast<int64_t>(group) * a.rows_per_group;
  const int64_t g1 = g0 + a.rows_per_group < a.M ? g0 + a.rows_per_group : a.M;
  const int64_t m0 = g0 + static_cast<int64_t>(slice) * chunk;
  const int64_t m1 = m0 + chunk < g1 ? m0 + chunk : g1;
  if (m0 >= m1) return;
  const T *x0 = static_cast<const T *>(a.X), *dy0 = static_cast<const T *>(a.dY);
  extern __shared__ __align__(16) uint8_t ring[];
  BackwardAhead<T, TEAM, VEC, E, FULL> xs, ds;
#pragma unroll
  for (int d = 0; d < kBackwardDepth<T, TEAM>; ++d) {
    xs.start(ring, d, x0, a.x_stride, m0, m1, a.K);
    ds.start(ring + xs.bytes(blockDim.x), d, dy0, a.dy_stride, m0, m1, a.K);
    copies_commit();
  }
  float mean_n = a.mean[m0], rstd_n = a.rstd[m0];
  f32x2 w[E / 2], dw[E / 2], db[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    dw[i] = db[i] = 0;
    w[i] = both(1.0f);
  }
  if (a.weight) load_params<TEAM, VEC, E, FULL>(a.weight, a.param_dtype, group * a.weight_stride, a.K, a.weight_offset, w);
  const float inv_k = 1.0f / a.K;
  int slot = 0;
  for (int64_t m = m0; m < m1; ++m) {
    f32x2 x[E / 2], g[E / 2];
    copies_wait<kBackwardDepth<T, TEAM> - 1>();
    xs.take(slot, a.K, x);
    ds.take(slot, a.K, g);
    const f32x2 minus = both(-mean_n), r2 = both(rstd_n);
    const float rstd = rstd_n;
    if (m + 1 < m1) {
      mean_n = a.mean[m + 1];
      rstd_n = a.rstd[m + 1];
    }
    // (not beside the row, where -mean * rstd may overflow: 1537 x 1153 of fp32 in 11.4 us, 10.0 without the test of
    // every column that rows without vectors pay for it)
    within_row<TEAM, VEC, E, FULL>(a.K, x, [&](f32x2 p, int) { return mul2(add2(p, minus), r2); });
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      dw[i] = fma2(g[i], x[i], dw[i]);
      db[i] = add2(db[i], g[i]);
      g[i] = mul2(g[i], w[i]);
    }
    xs.refill(slot, x0, a.x_stride, m, m1, a.K);
    ds.refill(slot, dy0, a.dy_stride, m, m1, a.K);
    copies_commit();
    slot = slot + 1 == kBackwardDepth<T, TEAM> ? 0 : slot + 1;
    if (a.dX) {
      float v[2] = {thread_sum(g), thread_dot(g, x)};
      sum(v, turn);
      const f32x2 c0 = both(-v[0] * inv_k * rstd), c1 = both(-v[1] * inv_k * rstd);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) x[i] = fma2(g[i], r2, fma2(x[i], c1, c0));
      store_row<T, TEAM, VEC, E, FULL>(static_cast<T *>(a.dX) + m * a.dx_stride, a.K, x);
    }
  }
  if (!a.dweight && !a.dbias) return;
  float *pw = slices == 1 ? a.dweight : a.partial + static_cast<size_t>(blockIdx.x) * 2 * a.K;
  float *pb = slices == 1 ? a.dbias : pw + a.K;
  const size_t at = slices == 1 ? static_cast<size_t>(group) * a.K : 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int k = row_column<TEAM, VEC>(i);
    if (FULL || k < a.K) {
      if (pw) pw[at + k] = i % 2 ? hi(dw[i / 2]) : lo(dw[i / 2]);
      if (pb) pb[at + k] = i % 2 ? hi(db[i / 2]) : lo(db[i / 2]);
    }
  }
}

// dweight (blockIdx.z = 0) or dbias (1) of a group's 32 columns from the group's slices: 32 warps add every
// 32nd slice, then a warp adds their sums in order.
__global__ void __launch_bounds__(1024) k_layer_norm_slices(NormLaunch a, int slices, int chunk) {
  __shared__ float part[32][32];
  float *out = blockIdx.z == 0 ? a.dweight : a.dbias;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k = blockIdx.y * 32 + lane;
  const int group = blockIdx.x;  // (there may be more groups than a grid has rows)
  const int64_t left = a.M - static_cast<int64_t>(group) * a.rows_per_group;
  const int rows = left <= 0 ? 0 : static_cast<int>(left < a.rows_per_group ? left : a.rows_per_group);
  const int n = (rows + chunk - 1) / chunk;  // slices that have rows
  grid_dep_wait();
  if (!out) return;
  float v = 0.0f;
  if (k < a.K) {
    const float *p = a.partial + (static_cast<size_t>(group) * slices * 2 + blockIdx.z) * a.K + k;
#pragma unroll 16
    for (int s = warp; s < n; s += 32) v += __ldcg(p + static_cast<size_t>(s) * 2 * a.K);
  }
  part[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && k < a.K) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += part[i][lane];
    out[static_cast<size_t>(group) * a.K + k] = s;
  }
}

// Whether rows and parameters allow 16-byte vectors of T.
template <typename T>
bool vectors(const NormLaunch &a) {
  constexpr size_t e = sizeof(T);
  if (a.K % kVec<T>) return false;
  const size_t pe = a.param_dtype == SVDQ_F32 ? 4 : 2;
  const size_t pv = pe * kVec<T> < 16 ? pe * kVec<T> : 16;
  auto rows = [&](const void *p, size_t stride) { return !p || rows_aligned(p, a.M > 1 ? stride : 0, e, 16); };
  auto params = [&](const void *p, size_t stride) { return !p || rows_aligned(p, a.groups > 1 ? stride : 0, pe, pv); };
  return rows(a.X, a.x_stride) && rows(a.Y, a.y_stride) && rows(a.dY, a.dy_stride) && rows(a.dX, a.dx_stride) &&
         params(a.weight, a.weight_stride) && params(a.bias, a.bias_stride);
}

template <typename T, bool QUANT>
cudaError_t forward_t(const NormLaunch &a) {
  return for_row(a.K, [&]<int TEAM, int E>() {
    // a block's rows are consecutive: as many blocks as are resident at once
    const bool vec = vectors<T>(a);
    const int threads = vec ? row_threads(a.K, E) : TEAM;
    const int blocks = a.num_sms * blocks_per_sm(threads, kForwardThreads<TEAM>);
    const int rows = (a.M + blocks - 1) / blocks;
    const dim3 grid((a.M + rows - 1) / rows);
    using Ring = Ahead<T, TEAM, kVec<T>, E, true>;
    const int smem = vec ? Ring::bytes(threads) : 0;
    auto kern = !vec                 ? k_layer_norm<T, TEAM, E, 1, false, QUANT>
                : row_full(a.K, E) ? k_layer_norm<T, TEAM, E, kVec<T>, true, QUANT>
                                   : k_layer_norm<T, TEAM, E, kVec<T>, false, QUANT>;
    const cudaError_t e = vec ? allow_smem<Ring::bytes(TEAM)>(kern) : cudaSuccess;
    return e != cudaSuccess ? e : launch_dependent(kern, grid, threads, smem, a.stream, a, rows);
  });
}

template <bool QUANT>
cudaError_t forward(const NormLaunch &a) {
  if (a.dtype == SVDQ_F32) return forward_t<float, QUANT>(a);
  if (a.dtype == SVDQ_F16) return forward_t<__half, QUANT>(a);
  return forward_t<__nv_bfloat16, QUANT>(a);
}

// Slices of a group's rows in the backward pass and the rows of each: the blocks that the SMs hold at once,
// over all groups, but no slice of so few rows that its partial sums (8 bytes a column) would be more than
// about half of what they are the sums of (three times a row's bytes).
struct Slices {
  int used;  // groups that have rows
  int slices, chunk;
};
Slices slices_of(int M, int K, int rows_per_group, int least) {
  const int used = pieces(M, rows_per_group);
  const int rows = M < rows_per_group ? M : rows_per_group;
  const int threads = for_row(K, [K]<int TEAM, int E>() { return row_threads(K, E); });
  int s = 148 * blocks_per_sm(threads, kBackwardThreads) / used;
  if (s > (rows + least - 1) / least) s = (rows + least - 1) / least;
  if (s < 1) s = 1;
  const int chunk = (rows + s - 1) / s;
  return {used, (rows + chunk - 1) / chunk, chunk};
}
constexpr int least_rows(size_t elem_bytes) { return elem_bytes == 2 ? 3 : 2; }

template <typename T>
cudaError_t backward_t(const NormLaunch &a) {
  const Slices s = slices_of(a.M, a.K, a.rows_per_group, least_rows(sizeof(T)));
  const bool sums = a.dweight || a.dbias;
  if (sums && s.slices == 1 && s.used < a.groups) {
    // groups behind the last row (the second kernel zeroes them where there is one)
    const size_t at = static_cast<size_t>(s.used) * a.K, bytes = static_cast<size_t>(a.groups - s.used) * a.K * 4;
    for (float *p : {a.dweight, a.dbias}) {
      const cudaError_t e = p ? reported(cudaMemsetAsync(p + at, 0, bytes, a.stream)) : cudaSuccess;
      if (e != cudaSuccess) return e;
    }
  }
  const cudaError_t e = for_row(a.K, [&]<int TEAM, int E>() {
    const dim3 grid(static_cast<unsigned>(s.used) * s.slices);
    const bool vec = vectors<T>(a);
    const int threads = vec ? row_threads(a.K, E) : TEAM;
    using Ring = BackwardAhead<T, TEAM, kVec<T>, E, true>;
    const int smem = vec ? 2 * Ring::bytes(threads) : 0;
    auto kern = !vec                 ? k_layer_norm_backward<T, TEAM, E, 1, false>
                : row_full(a.K, E) ? k_layer_norm_backward<T, TEAM, E, kVec<T>, true>
                                   : k_layer_norm_backward<T, TEAM, E, kVec<T>, false>;
    const cudaError_t e = vec ? allow_smem<2 * Ring::bytes(TEAM)>(kern) : cudaSuccess;
    if (e != cudaSuccess) return e;
    return launch(kern, grid, threads, smem, a.stream, a, s.slices, s.chunk);
  });
  if (e != cudaSuccess || !sums || s.slices == 1) return e;
  return launch_dependent(k_layer_norm_slices, dim3(a.groups, (a.K + 31) / 32, 2), 1024, 0, a.stream, a, s.slices, s.chunk);
}

}  // namespace

cudaError_t launch_layer_norm(const NormLaunch &a) { return forward<false>(a); }

cudaError_t launch_layer_norm_quantize(const NormLaunch &a) { return forward<true>(a); }

size_t layer_norm_partial_bytes(int M, int K, int rows_per_group) {
  // enough for any type: fp32 rows make the shortest slices
  const Slices s = slices_of(M, K, rows_per_group, least_rows(4));
  if (s.slices == 1) return 0;
  return (static_cast<size_t>(s.used) * s.slices * 2 * K * sizeof(float) + 15) / 16 * 16;
}

cudaError_t launch_layer_norm_backward(const NormLaunch &a) {
  if (a.dtype == SVDQ_F32) return backward_t<float>(a);
  if (a.dtype == SVDQ_F16) return backward_t<__half>(a);
  return backward_t<__nv_bfloat16>(a);
}

}  // namespace svdq
