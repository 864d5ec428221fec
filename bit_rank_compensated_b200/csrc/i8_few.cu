// The 8-bit linear of up to eight tokens: bound by the weight's bytes, which are read once, and by latency.
//
// Y[m, n] = (sum_k xq[m, k] wq[n, k]) x_scale[m] w_scale[n] + bias[n], with exact 32-bit integer sums.
//
// A tensor-core tile would be nearly empty and its pipeline costs more than the product (19 us for 4096 x
// 4096 and one token), so the CUDA cores multiply: four int8 products an instruction (dp4a). The tokens'
// codes lie in shared memory; where the caller has floating rows and they are short, every block quantizes
// them itself (the row quantizer's own arithmetic: the same codes), which saves a launch.
//
// A block of eight warps takes CB channels for each WN-th of its warps and shares the K axis out among
// the WK = 8 / WN others: a lane multiplies 16 bytes of each channel's row with the same bytes of every
// token's, keeps CB x M sums, and fetches the next channels' weights meanwhile (8 or 16 KiB in flight
// a block). Integer sums need no order: lanes by redux, warps through shared memory.
#include "block.h"
#include "common.cuh"
#include "i8_quant.cuh"
#include "row.cuh"

namespace svdq {
namespace {

constexpr int kWarps = 8;
constexpr int CB = 4;        // channels of a warp
constexpr int CHUNK = 512;   // bytes of a row that a warp reads at once
constexpr int kMaxCodes = 96 * 1024;  // bytes of shared memory for the tokens' codes
constexpr int kMaxQuantized = 8192;   // codes that a block makes itself (i8_few_quantizes)
constexpr int kWideChannels = 37 * 256, kShortRow = 1536;  // i8_few_fits

struct FewArgs {
  // floating rows and their smoothing, or int8 rows and their scales
  const void *X;
  size_t x_stride;
  const float *col_scale;
  const int8_t *xq;
  const float *x_scale;
  const int8_t *wq;
  const float *w_scale, *bias;
  void *Y;
  int M, N, K;
  int chunks;  // of CHUNK columns
  int wk;      // warps that share the K axis: 1, 2, 4 or 8
  int tasks;   // of CB * (8 / wk) channels
};

__device__ __forceinline__ uint4 ldg_stream(const int8_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Codes and scales of the M rows into shared memory: 8 / MT warps a row, the row read twice (the second
// time from L1).
template <typename T, int MT>
__device__ __forceinline__ void quantize(const FewArgs &a, int8_t *codes, float *scale, uint32_t *top) {
  constexpr int WPR = kWarps / MT, V = kVec<T>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m = warp / WPR, part = warp % WPR;
  const T *x = static_cast<const T *>(a.X) + m * a.x_stride;
  auto vector = [&](int k, f32x2 (&v)[V / 2]) {
    const uint4 q = *reinterpret_cast<const uint4 *>(x + k);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      if constexpr (sizeof(T) == 2) v[i] = widen(w[i], T{});
      else v[i] = pair_bits(w[2 * i], w[2 * i + 1]);
    }
    if (a.col_scale) {
#pragma unroll
      for (int i = 0; i < V / 2; i += 2) {
        const float4 c = __ldg(reinterpret_cast<const float4 *>(a.col_scale + k + 2 * i));
        v[i] = mul2(v[i], pair(c.x, c.y));
        v[i + 1] = mul2(v[i + 1], pair(c.z, c.w));
      }
    }
  };
  uint32_t t = 0;
  if (m < a.M) {
#pragma unroll 4
    for (int k = (part * 32 + lane) * V; k < a.K; k += WPR * 32 * V) {
      f32x2 v[V / 2];
      vector(k, v);
      t = max(t, thread_top(v));
    }
  }
  t = __reduce_max_sync(0xffffffffu, t);
  if (lane == 0) top[warp] = t;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WPR; ++i) t = max(t, top[m * WPR + i]);
  const RowScale r = row_scale<false>(t);
  if (part == 0 && lane == 0) scale[m] = scale_of(r);
  int8_t *q = codes + static_cast<size_t>(m) * a.K;
#pragma unroll 2
  for (int k = (part * 32 + lane) * V; k < a.K; k += WPR * 32 * V) {
    uint32_t o[V / 4] = {};
    if (m < a.M) {
      f32x2 v[V / 2];
      vector(k, v);
      i8_pack<V / 2, false>(v, r, o);
    }
    if constexpr (V == 8) *reinterpret_cast<uint2 *>(q + k) = make_uint2(o[0], o[1]);
    else *reinterpret_cast<uint32_t *>(q + k) = o[0];
  }
}

// T: type of Y (and of X); MT: tokens the sums are kept for (rows from M on are zeros).
template <typename T, int MT, bool QUANT>
__global__ void __launch_bounds__(32 * kWarps, MT <= 2 ? 4 : (MT == 4 ? 3 : 2)) k_i8_few(FewArgs a) {
  extern __shared__ __align__(16) int8_t codes[];
  __shared__ int part[2][kWarps][CB * MT];
  __shared__ float scale[MT];
  __shared__ uint32_t top[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wn = warp / a.wk, wk = warp % a.wk;
  const int per_task = CB * (kWarps / a.wk);
  grid_dep_wait();
  grid_dep_launch();

  // the first channels' weights are on their way while the tokens are quantized
  int task = blockIdx.x, chunk = wk;
  uint4 w[CB];
  auto fetch = [&](int t, int c) {
    const bool there = t < a.tasks;  // (behind the last task the channel may pass 31 bits)
    const int n0 = there ? t * per_task + wn * CB : 0, k = c * CHUNK + lane * 16;
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      w[i] = make_uint4(0, 0, 0, 0);
      if (there && n0 + i < a.N && k < a.K) w[i] = ldg_stream(a.wq + static_cast<size_t>(n0 + i) * a.K + k);
    }
  };
  fetch(task, chunk);

  if constexpr (QUANT) {
    quantize<T, MT>(a, codes, scale, top);
  } else {
    for (int i = threadIdx.x; i < MT * a.K / 16; i += 32 * kWarps) {
      const bool there = i < a.M * a.K / 16;
      reinterpret_cast<uint4 *>(codes)[i] = there ? *reinterpret_cast<const uint4 *>(a.xq + 16 * static_cast<size_t>(i)) : make_uint4(0, 0, 0, 0);
    }
    if (threadIdx.x < MT) scale[threadIdx.x] = static_cast<int>(threadIdx.x) < a.M ? a.x_scale[threadIdx.x] : 0.0f;
  }
  __syncthreads();

  uint32_t buf = 0;
  for (; task < a.tasks; task += gridDim.x, buf ^= 1) {
    int acc[CB][MT] = {};
    for (chunk = wk; chunk < a.chunks; chunk += a.wk) {
      uint4 v[CB];
#pragma unroll
      for (int i = 0; i < CB; ++i) v[i] = w[i];
      const bool last = chunk + a.wk >= a.chunks;
      fetch(last ? task + static_cast<int>(gridDim.x) : task, last ? wk : chunk + a.wk);
      const int k = chunk * CHUNK + lane * 16;
      if (k < a.K) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint4 x = *reinterpret_cast<const uint4 *>(codes + static_cast<size_t>(m) * a.K + k);
#pragma unroll
          for (int i = 0; i < CB; ++i) {
            acc[i][m] = __dp4a(static_cast<int>(v[i].x), static_cast<int>(x.x), acc[i][m]);
            acc[i][m] = __dp4a(static_cast<int>(v[i].y), static_cast<int>(x.y), acc[i][m]);
            acc[i][m] = __dp4a(static_cast<int>(v[i].z), static_cast<int>(x.z), acc[i][m]);
            acc[i][m] = __dp4a(static_cast<int>(v[i].w), static_cast<int>(x.w), acc[i][m]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < CB; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int s = __reduce_add_sync(0xffffffffu, acc[i][m]);
        if (lane == 0) part[buf][warp][i * MT + m] = s;
      }
    __syncthreads();  // the other buffer is free again once every warp is here
    const int outputs = per_task * MT;
    if (static_cast<int>(threadIdx.x) < outputs) {
      // consecutive threads on consecutive channels
      const int m = threadIdx.x / per_task, c = threadIdx.x % per_task;
      const int n = task * per_task + c;
      if (m < a.M && n < a.N) {
        int s = 0;
        for (int i = 0; i < a.wk; ++i) s += part[buf][(c / CB) * a.wk + i][(c % CB) * MT + m];
        static_cast<T *>(a.Y)[static_cast<size_t>(m) * a.N + n] =
            from_f32<T>(fmaf(__fmul_rn(static_cast<float>(s), scale[m]), a.w_scale[n], a.bias ? a.bias[n] : 0.0f));
      }
    }
  }
}

template <typename T, int MT, bool QUANT>
cudaError_t launch_mt(FewArgs a, int num_sms, cudaStream_t st) {
  a.chunks = (a.K + CHUNK - 1) / CHUNK;
  a.wk = a.chunks >= 8 ? 8 : (a.chunks >= 4 ? 4 : (a.chunks >= 2 ? 2 : 1));
  const int per_task = CB * (kWarps / a.wk);
  a.tasks = pieces(a.N, per_task);
  const int smem = MT * a.K;
  // blocks that an SM holds at once, by registers and by the codes' share of its memory
  int resident = MT <= 2 ? 4 : (MT == 4 ? 3 : 2);
  while (resident > 1 && resident * (smem + 2048) > 220 * 1024) --resident;
  const int rounds = (a.tasks + resident * num_sms - 1) / (resident * num_sms);
  const dim3 grid((a.tasks + rounds - 1) / rounds);
  auto kern = k_i8_few<T, MT, QUANT>;
  const cudaError_t e = allow_smem<QUANT ? kMaxQuantized : kMaxCodes>(kern);
  return e != cudaSuccess ? e : launch_dependent(kern, grid, 32 * kWarps, smem, st, a);
}

template <typename T, bool QUANT>
cudaError_t launch_m(const FewArgs &a, int num_sms, cudaStream_t st) {
  if (a.M == 1) return launch_mt<T, 1, QUANT>(a, num_sms, st);
  if (a.M == 2) return launch_mt<T, 2, QUANT>(a, num_sms, st);
  if (a.M <= 4) return launch_mt<T, 4, QUANT>(a, num_sms, st);
  return launch_mt<T, 8, QUANT>(a, num_sms, st);
}

template <bool QUANT>
cudaError_t launch_type(const FewArgs &a, int dtype, int num_sms, cudaStream_t st) {
  if (dtype == SVDQ_F32) return launch_m<float, QUANT>(a, num_sms, st);
  if (dtype == SVDQ_F16) return launch_m<__half, QUANT>(a, num_sms, st);
  return launch_m<__nv_bfloat16, QUANT>(a, num_sms, st);
}

int padded_tokens(int M) { return M <= 2 ? M : (M <= 4 ? 4 : 8); }

}  // namespace

// Against the tensor cores, from int8 rows (us): 4096 x 4096 5.5 and 10.7 for one token, 7.5 and 10.7 for four, 9.7 and
// 10.7 for eight; 12288 x 4096 (N x K) 11.7 and 22.3, 14.7 and 19.3, 22.2 and 18.9. Five tokens and more multiply as
// eight and are bound by that: where the tensor cores' tiles are enough without a split of the K axis and it is not
// short (12288 x 1536: 9.9 and 9.5), they are left to them.
bool i8_few_fits(int M, int N, int K) {
  if (M > 8 || static_cast<int64_t>(padded_tokens(M)) * K > kMaxCodes) return false;
  return M <= 4 || N <= kWideChannels || K <= kShortRow;
}

// Each of several hundred blocks quantizes the rows for itself, which saves a launch (2 us of the host) but costs by
// what there is to quantize. In the block and by the row quantizer (us, bf16): one token, 4096 x 4096 7.4 and 6.6;
// two tokens 8.8 and 7.4; four, 4096 x 2048 7.8 and 6.4; eight, 4096 x 1024 6.3 and 5.2; and beyond, four tokens,
// 4096 x 4096 12.3 and 8.8; eight 17.9 and 11.0.
bool i8_few_quantizes(const QuantRowsLaunch &q) {
  if (padded_tokens(q.M) * q.K > kMaxQuantized) return false;
  const size_t e = q.dtype == SVDQ_F32 ? 4 : 2;
  return rows_aligned(q.X, q.M > 1 ? q.x_stride : 0, e, 16) && rows_aligned(q.col_scale, 0, 4, 16);
}

cudaError_t launch_i8_few(const I8GemmLaunch &g) {
  const FewArgs a{nullptr, 0, nullptr, g.xq, g.x_scale, g.wq, g.w_scale, g.bias, g.Y, g.M, g.N, g.K, 0, 0, 0};
  return launch_type<false>(a, g.y_dtype, g.dev->num_sms, g.stream);
}

cudaError_t launch_i8_few_quantized(const QuantRowsLaunch &q, const I8GemmLaunch &g) {
  const FewArgs a{q.X, q.x_stride, q.col_scale, nullptr, nullptr, g.wq, g.w_scale, g.bias, g.Y, g.M, g.N, g.K, 0, 0, 0};
  return launch_type<true>(a, g.y_dtype, g.dev->num_sms, g.stream);
}

}  // namespace svdq
