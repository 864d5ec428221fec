// Rotary positions with several axes: the (cos, sin) table and the rotation of Q and K heads.
//
// angle = pos[m][axis of p] theta^-(power of p); (u0, u1) -> (u0 cos - u1 sin, u1 cos + u0 sin).
//
// Both are bound by memory: the table by its writes, the rotation by one read and one write of the
// heads. Angles are formed in fp64 as fractions of a turn, since a far position times a frequency has
// no fraction left in fp32: pos * (frequency / 2 pi) less the nearest integer, rounded to fp32 only
// then. A frequency costs an fp64 exponential and belongs to a pair, an angle costs two fp64
// operations and belongs to a token and pair, and every head of a token uses the same ones: a block
// forms its frequencies once, the angles once for each tile of tokens, and turns all heads from them.
#include "block.h"
#include "common.cuh"
#include "row.cuh"

namespace svdq {
namespace {

constexpr int kMaxPairs = 256;
constexpr int kThreads = 256;

// Frequency (in turns per position) and axis of every pair.
struct Ladder {
  double turns[kMaxPairs];
  uint8_t axis[kMaxPairs];

  __device__ __forceinline__ void fill(const svdq_rope_axes &ax, int P, double log2_theta) {
    for (int p = threadIdx.x; p < P; p += blockDim.x) {
      int a = 0, i = p;
      while (i >= ax.pairs[a]) i -= ax.pairs[a++];
      const double power = ax.shared_ladder ? static_cast<double>(p) / P : static_cast<double>(i) / ax.pairs[a];
      turns[p] = exp2(-power * log2_theta) * 0.15915494309189533577;  // / 2 pi
      axis[p] = static_cast<uint8_t>(a);
    }
  }
  // (cos, sin) of pair p of token m.
  __device__ __forceinline__ float2 operator()(const svdq_positions &pos, size_t m, int p) const {
    const size_t at = m * pos.token_stride + axis[p] * pos.axis_stride;
    const double v = pos.dtype == SVDQ_I64   ? static_cast<double>(static_cast<const int64_t *>(pos.data)[at])
                     : pos.dtype == SVDQ_I32 ? static_cast<double>(static_cast<const int32_t *>(pos.data)[at])
                                             : static_cast<double>(static_cast<const float *>(pos.data)[at]);
    const double t = v * turns[p];
    float2 cs;
    sincospif(static_cast<float>(2.0 * (t - rint(t))), &cs.y, &cs.x);
    return cs;
  }
};

// A thread keeps its pair and takes every lanes-th token of the block's share.
__global__ void __launch_bounds__(kThreads) k_rope_table(RopeLaunch a, int tokens) {
  __shared__ Ladder ladder;
  ladder.fill(a.axes, a.n_pairs, a.log2_theta);
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  const int lanes = kThreads / a.n_pairs;
  const int p = threadIdx.x % a.n_pairs, lane = threadIdx.x / a.n_pairs;
  if (lane >= lanes) return;
  const size_t m0 = static_cast<size_t>(blockIdx.x) * tokens;
  const size_t m1 = m0 + tokens < static_cast<size_t>(a.M) ? m0 + tokens : a.M;
  // four tokens' positions in flight
#pragma unroll 4
  for (size_t m = m0 + lane; m < m1; m += lanes)
    __stcs(reinterpret_cast<float2 *>(a.table) + m * a.n_pairs + p, ladder(a.pos, m, p));
}

__device__ __forceinline__ void turn(float &u0, float &u1, float2 cs) {
  const float v0 = fmaf(u0, cs.x, -__fmul_rn(u1, cs.y));
  u1 = fmaf(u1, cs.x, __fmul_rn(u0, cs.y));
  u0 = v0;
}

// The vector of VEC values at p (16 bytes, or one value), and back; touched once, so marked as such (fp32
// heads that fit L2: 13.7 us against 15.1).
template <typename T, int VEC>
struct Vec {
  uint32_t w[VEC > 1 ? 4 : 1];

  __device__ __forceinline__ void load(const T *p) {
    if constexpr (VEC > 1) {
      const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(p));
      w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else {
      w[0] = __float_as_uint(to_f32(*p));
    }
  }
  __device__ __forceinline__ void store(T *p) const {
    if constexpr (VEC > 1) __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
    else *p = from_f32<T>(__uint_as_float(w[0]));
  }
  __device__ __forceinline__ void get(float (&x)[VEC]) const {
    if constexpr (VEC == 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2 p = widen(w[i], T{});
        x[2 * i] = lo(p);
        x[2 * i + 1] = hi(p);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[i] = __uint_as_float(w[i]);
    }
  }
  // value i, unless it is to stay as loaded
  __device__ __forceinline__ void set(const float (&x)[VEC]) {
    if constexpr (VEC == 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = narrow(pair(x[2 * i], x[2 * i + 1]), T{});
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) w[i] = __float_as_uint(x[i]);
    }
  }
};

// A head's columns are shared out in units, one to a thread: with HALVES the vector at column u VEC and
// its partner P columns on, else the vector at u VEC (VEC = 1: the pair 2u, 2u + 1); behind the rotated
// columns, the vectors (pairs) that are copied. Thread (head lane, unit) keeps its unit's (cos, sin) of a
// token for all heads that it turns, four of them in flight at a time.
template <typename T, int VEC, bool HALVES>
__global__ void __launch_bounds__(kThreads) k_rope_apply(RopeLaunch a, int units, int lanes, int tile, int tiles) {
  constexpr int TURN = VEC > 1 ? VEC / (HALVES ? 1 : 2) : 1;  // pairs of a unit
  constexpr int AHEAD = 4;
  __shared__ Ladder ladder;
  __shared__ float2 cs_s[2][kMaxPairs];
  const int P = a.n_pairs;
  ladder.fill(a.axes, P, a.log2_theta);
  grid_dep_wait();
  grid_dep_launch();
  const int u = threadIdx.x % units, lane = threadIdx.x / units;
  const int turned = HALVES ? P / TURN : (P + TURN - 1) / TURN;  // units that turn
  const bool turns = u < turned;
  // first column of the unit's vector, and of its partner
  const int c0 = VEC > 1 ? (HALVES && !turns ? 2 * P + (u - turned) * VEC : u * VEC) : (HALVES && turns ? u : 2 * u);
  const int c1 = HALVES && turns ? c0 + P : (VEC > 1 ? c0 : c0 + 1);
  const int heads = a.in[0].heads + a.in[1].heads;
  const int first = lane < lanes ? blockIdx.y * lanes + lane : heads;
  const int step = gridDim.y * lanes;
  uint32_t buf = 0;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x, buf ^= 1) {
    const size_t m0 = static_cast<size_t>(t) * tile;
    const int n = static_cast<int>(a.M - m0 < static_cast<size_t>(tile) ? a.M - m0 : tile);
    if (t == static_cast<int>(blockIdx.x)) __syncthreads();  // the ladder
    for (int i = threadIdx.x; i < n * P; i += blockDim.x) {
      float2 cs = ladder(a.pos, m0 + i / P, i % P);
      if (a.inverse) cs.y = -cs.y;
      cs_s[buf][i] = cs;
    }
    __syncthreads();  // this tile's angles; the next tile's go to the other buffer
    for (int j = 0; j < n; ++j) {
      float2 cs[TURN];
#pragma unroll
      for (int i = 0; i < TURN; ++i) cs[i] = turns && u * TURN + i < P ? cs_s[buf][j * P + u * TURN + i] : make_float2(1.0f, 0.0f);
      const size_t m = m0 + j;
      for (int h0 = first; h0 < heads; h0 += AHEAD * step) {
        Vec<T, VEC> v0[AHEAD], v1[AHEAD];
        T *out[AHEAD];
        bool copy[AHEAD];
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
          const int hh = h0 + e * step;
          copy[e] = hh < heads;
          if (!copy[e]) continue;
          const int k = hh >= a.in[0].heads;
          const int h = k ? hh - a.in[0].heads : hh;
          const T *in = static_cast<const T *>(a.in[k].data) + m * a.in[k].token_stride + h * a.in[k].head_stride;
          out[e] = static_cast<T *>(a.out[k].data) + m * a.out[k].token_stride + h * a.out[k].head_stride;
          v0[e].load(in + c0);
          if (HALVES || VEC == 1) v1[e].load(in + c1);
        }
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
          if (!copy[e]) continue;
          if (turns) {
            float x[VEC], y[VEC];
            v0[e].get(x);
            if constexpr (HALVES || VEC == 1) {
              v1[e].get(y);
#pragma unroll
              for (int i = 0; i < VEC; ++i) turn(x[i], y[i], cs[i]);
              v1[e].set(y);
            } else {
#pragma unroll
              for (int i = 0; i < TURN; ++i)
                if (u * TURN + i < P) turn(x[2 * i], x[2 * i + 1], cs[i]);  // a pair behind the rotated ones stays
            }
            v0[e].set(x);
          }
          v0[e].store(out[e] + c0);
          if ((HALVES && turns) || VEC == 1) v1[e].store(out[e] + c1);
        }
      }
    }
  }
}

template <typename T, int VEC, bool HALVES>
cudaError_t apply(const RopeLaunch &a) {
  const int P = a.n_pairs, D = a.head_dim;
  const int units = VEC == 1 ? D / 2 : (HALVES ? P / VEC + (D - 2 * P) / VEC : D / VEC);
  const int heads = a.in[0].heads + a.in[1].heads;
  int lanes = kThreads / units;
  if (lanes > heads) lanes = heads;
  const int threads = (units * lanes + 31) / 32 * 32;
  // tokens of a tile: as many as give every thread an angle to form, fewer where that leaves SMs idle
  int tile = kThreads / P;
  const int resident = 8 * a.num_sms;
  if (tile > (a.M + resident - 1) / resident) tile = (a.M + resident - 1) / resident;
  const int tiles = (a.M + tile - 1) / tile;
  const int gx = tiles < resident ? tiles : resident;
  // few tokens: their heads are shared out among blocks too
  const int rounds = (heads + lanes - 1) / lanes;
  int gy = 2 * a.num_sms / gx;
  gy = gy < 1 ? 1 : (gy > rounds ? rounds : gy);
  return launch_dependent(k_rope_apply<T, VEC, HALVES>, dim3(gx, gy), threads, 0, a.stream, a, units, lanes, tile, tiles);
}

template <typename T>
cudaError_t apply_t(const RopeLaunch &a) {
  constexpr int V = kVec<T>;
  bool vec = a.head_dim % V == 0 && (!a.axes.halves || a.n_pairs % V == 0);
  for (int t = 0; t < 2; ++t)
    for (const svdq_heads *h : {&a.in[t], &a.out[t]})
      if (a.in[t].heads)
        vec = vec && rows_aligned(h->data, a.M > 1 ? h->token_stride : 0, sizeof(T), 16) &&
              rows_aligned(h->data, h->heads > 1 ? h->head_stride : 0, sizeof(T), 16);
  if (a.axes.halves) return vec ? apply<T, V, true>(a) : apply<T, 1, true>(a);
  return vec ? apply<T, V, false>(a) : apply<T, 1, false>(a);
}

}  // namespace

cudaError_t launch_rope_table(const RopeLaunch &a) {
  const int lanes = kThreads / a.n_pairs;
  const int blocks = 4 * a.num_sms;
  int tokens = (a.M + blocks - 1) / blocks;
  tokens = (tokens + lanes - 1) / lanes * lanes;
  return launch_dependent(k_rope_table, dim3((a.M + tokens - 1) / tokens), kThreads, 0, a.stream, a, tokens);
}

cudaError_t launch_rope_apply(const RopeLaunch &a) {
  if (a.dtype == SVDQ_F32) return apply_t<float>(a);
  if (a.dtype == SVDQ_F16) return apply_t<__half>(a);
  return apply_t<__nv_bfloat16>(a);
}

}  // namespace svdq
