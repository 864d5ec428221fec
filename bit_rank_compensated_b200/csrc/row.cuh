// A row spread over the threads of a block, in registers: what the layer norm's kernels and the row
// quantizer share.
//
// Thread t of a block of T <= TEAM threads holds E values as E / 2 pairs: VEC consecutive ones at columns
// (v T + t) VEC, v = 0 .. E / VEC - 1, VEC values being 16 bytes (one load), or VEC = 1 where rows do not
// start on 16 bytes or do not end on a whole vector (consecutive threads on consecutive columns). With vectors T
// is the row's length over E, in whole warps; where that leaves nothing over (FULL), no column is checked.
// Else columns from K on hold zeros. Without them T = TEAM, so that every value's offset is a constant.
#pragma once

#include <stdint.h>

#include "i8_quant.cuh"
#include "pair.cuh"
#include "svdq.h"
#include "types.cuh"

namespace svdq {

template <typename T>
constexpr int kVec = 16 / sizeof(T);

template <int TEAM, int VEC>
__device__ __forceinline__ int row_column(int i) {
  const int t = TEAM == 32 || VEC == 1 ? TEAM : static_cast<int>(blockDim.x);
  return ((i / VEC) * t + static_cast<int>(threadIdx.x)) * VEC + i % VEC;
}

template <typename T, int TEAM, int VEC, int E, bool FULL>
__device__ __forceinline__ void store_row(T *p, int K, const f32x2 (&y)[E / 2]) {
  if constexpr (VEC == 1) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int k = row_column<TEAM, VEC>(i);
      if (FULL || k < K) p[k] = from_f32<T>(i % 2 ? hi(y[i / 2]) : lo(y[i / 2]));
    }
  } else {
#pragma unroll
    for (int v = 0; v < E / VEC; ++v) {
      const int k = row_column<TEAM, VEC>(v * VEC);
      if (!FULL && k >= K) continue;
      const f32x2 *s = y + v * VEC / 2;
      uint4 o;
      if constexpr (sizeof(T) == 4) o = make_uint4(lo_bits(s[0]), hi_bits(s[0]), lo_bits(s[1]), hi_bits(s[1]));
      else o = make_uint4(narrow(s[0], T{}), narrow(s[1], T{}), narrow(s[2], T{}), narrow(s[3], T{}));
      *reinterpret_cast<uint4 *>(p + k) = o;
    }
  }
}

// The int8 codes of a row, VEC bytes a store, each vector as soon as it is formed.
template <int TEAM, int VEC, int E, bool FULL, bool SHORT>
__device__ __forceinline__ void store_codes(int8_t *p, int K, const f32x2 (&x)[E / 2], const RowScale &r) {
#pragma unroll
  for (int v = 0; v < E / (VEC > 1 ? VEC : 2); ++v) {
    uint32_t o[VEC > 1 ? VEC / 4 : 1];
    if constexpr (VEC > 1) {
      const int k = row_column<TEAM, VEC>(v * VEC);
      if (!FULL && k >= K) continue;
      i8_pack<VEC / 2, SHORT>(x + v * VEC / 2, r, o);
      if constexpr (VEC == 8) *reinterpret_cast<uint2 *>(p + k) = make_uint2(o[0], o[1]);
      else *reinterpret_cast<uint32_t *>(p + k) = o[0];
    } else {
      i8_pack<1, SHORT>(x + v, r, o);
      const int k0 = row_column<TEAM, 1>(2 * v), k1 = row_column<TEAM, 1>(2 * v + 1);
      if (FULL || k0 < K) p[k0] = static_cast<int8_t>(o[0]);
      if (FULL || k1 < K) p[k1] = static_cast<int8_t>(o[0] >> 8);
    }
  }
}

// x[i] = f(x[i]) for the pairs within the row; columns from K on keep their zeros.
template <int TEAM, int VEC, int E, bool FULL, typename F>
__device__ __forceinline__ void within_row(int K, f32x2 (&x)[E / 2], F f) {
  if constexpr (VEC > 1) {
#pragma unroll
    for (int v = 0; v < E / VEC; ++v)
      if (FULL || row_column<TEAM, VEC>(v * VEC) < K)
#pragma unroll
        for (int i = v * VEC / 2; i < (v + 1) * VEC / 2; ++i) x[i] = f(x[i], i);
  } else {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const f32x2 y = f(x[i], i);
      x[i] = pair(FULL || row_column<TEAM, VEC>(2 * i) < K ? lo(y) : 0.0f, FULL || row_column<TEAM, VEC>(2 * i + 1) < K ? hi(y) : 0.0f);
    }
  }
}

// A row of parameters (of its own type, aligned to a vector's size where VEC > 1) in the same columns: kept
// in registers for all rows of a block.
template <int TEAM, int VEC, int E, bool FULL>
__device__ __forceinline__ void load_params(const void *base, int dtype, size_t at, int K, float add, f32x2 (&w)[E / 2]) {
  if constexpr (VEC == 1) {
    auto fill = [&](const auto *p) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const int k0 = row_column<TEAM, 1>(2 * i), k1 = row_column<TEAM, 1>(2 * i + 1);
        w[i] = pair(k0 < K ? add + to_f32(p[k0]) : 0.0f, k1 < K ? add + to_f32(p[k1]) : 0.0f);
      }
    };
    if (dtype == SVDQ_F32) fill(static_cast<const float *>(base) + at);
    else if (dtype == SVDQ_F16) fill(static_cast<const __half *>(base) + at);
    else fill(static_cast<const __nv_bfloat16 *>(base) + at);
  } else {
    const f32x2 add_both = both(add);
#pragma unroll
    for (int v = 0; v < E / VEC; ++v) {
      const int k = row_column<TEAM, VEC>(v * VEC);
      f32x2 *to = w + v * VEC / 2;
      if (!FULL && k >= K) {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) to[e] = 0;
      } else if (dtype == SVDQ_F32) {
        const float *p = static_cast<const float *>(base) + at + k;
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(p + e);
          to[e / 2] = add2(pair(f.x, f.y), add_both);
          to[e / 2 + 1] = add2(pair(f.z, f.w), add_both);
        }
      } else {
        const uint16_t *p = static_cast<const uint16_t *>(base) + at + k;
        uint32_t q[VEC / 2];
        if constexpr (VEC == 8) {
          const uint4 u = *reinterpret_cast<const uint4 *>(p);
          q[0] = u.x, q[1] = u.y, q[2] = u.z, q[3] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2 *>(p);
          q[0] = u.x, q[1] = u.y;
        }
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e)
          to[e] = add2(dtype == SVDQ_F16 ? widen(q[e], __half{}) : widen(q[e], __nv_bfloat16{}), add_both);
      }
    }
  }
}

// The copies of one row (of x, or of x and dy) make a group; groups complete in order.
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// The block's rows on their way: DEPTH of them in flight in a ring in shared memory, each thread's vectors
// in slots of its own (asynchronous copies: neither registers nor barriers). Rows without vectors (VEC = 1)
// are fetched one ahead, into registers.
template <typename T, int TEAM, int VEC, int E, bool FULL, int DEPTH>
struct RowsAhead {
  static constexpr int NV = E / VEC;
  uint32_t slot;  // shared address of this thread's first vector
  int threads;

  // Bytes of shared memory a block needs.
  static constexpr int bytes(int threads) { return threads * DEPTH * E * static_cast<int>(sizeof(T)); }

  __device__ __forceinline__ void fetch(int d, const T *p, int K, bool there) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int k = row_column<TEAM, VEC>(v * VEC);
      if (there && (FULL || k < K))
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + ((d * NV + v) * threads) * 16), "l"(p + k) : "memory");
    }
  }
  // Row m0 + d into slot d (the block's first rows).
  __device__ __forceinline__ void start(uint8_t *ring, int d, const T *x0, size_t stride, int64_t m0, int64_t m1, int K) {
    threads = TEAM == 32 ? 32 : blockDim.x;
    slot = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + threadIdx.x * 16;
    fetch(d, x0 + (m0 + d) * stride, K, m0 + d < m1);
  }
  // The values of the row in slot d.
  __device__ __forceinline__ void take(int d, int K, f32x2 (&x)[E / 2]) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      uint32_t w[4] = {0, 0, 0, 0};
      if (FULL || row_column<TEAM, VEC>(v * VEC) < K)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(slot + ((d * NV + v) * threads) * 16)
                     : "memory");
      f32x2 *to = x + v * VEC / 2;
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = widen(w[i], T{});
      } else {
        to[0] = pair_bits(w[0], w[1]);
        to[1] = pair_bits(w[2], w[3]);
      }
    }
  }
  // Row m + DEPTH into row m's slot d, once its values have been used.
  __device__ __forceinline__ void refill(int d, const T *x0, size_t stride, int64_t m, int64_t m1, int K) {
    fetch(d, x0 + (m + DEPTH) * stride, K, m + DEPTH < m1);
  }
};

template <typename T, int TEAM, int E, bool FULL, int DEPTH>
struct RowsAhead<T, TEAM, 1, E, FULL, DEPTH> {
  T next[E];  // as loaded: a conversion would wait for them

  static constexpr int bytes(int) { return 0; }
  __device__ __forceinline__ void fetch(const T *p, int K) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int k = row_column<TEAM, 1>(i);
      next[i] = FULL || k < K ? p[k] : from_f32<T>(0.0f);
    }
  }
  __device__ __forceinline__ void start(uint8_t *, int d, const T *x0, size_t stride, int64_t m0, int64_t m1, int K) {
    if (d == 0 && m0 < m1) fetch(x0 + m0 * stride, K);
  }
  __device__ __forceinline__ void take(int, int, f32x2 (&x)[E / 2]) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[i] = pair(to_f32(next[2 * i]), to_f32(next[2 * i + 1]));
  }
  __device__ __forceinline__ void refill(int, const T *x0, size_t stride, int64_t m, int64_t m1, int K) {
    if (m + 1 < m1) fetch(x0 + (m + 1) * stride, K);
  }
};

// A thread's sums, in four chains.
template <int N>
__device__ __forceinline__ float thread_sum(const f32x2 (&x)[N]) {
  f32x2 s = x[0], t = x[1];
#pragma unroll
  for (int i = 2; i < N; i += 2) {
    s = add2(s, x[i]);
    t = add2(t, x[i + 1]);
  }
  s = add2(s, t);
  return lo(s) + hi(s);
}
template <int N>
__device__ __forceinline__ float thread_dot(const f32x2 (&x)[N], const f32x2 (&y)[N]) {
  f32x2 s = mul2(x[0], y[0]), t = mul2(x[1], y[1]);
#pragma unroll
  for (int i = 2; i < N; i += 2) {
    s = fma2(x[i], y[i], s);
    t = fma2(x[i + 1], y[i + 1], t);
  }
  s = add2(s, t);
  return lo(s) + hi(s);
}
// Bits of the largest |x|, infinities and NaNs above all others.
template <int N>
__device__ __forceinline__ uint32_t thread_top(const f32x2 (&x)[N]) {
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) t = max_abs3(t, lo(x[i]), hi(x[i]));
  return __float_as_uint(t);
}

// Sums over the block, in every thread and in a fixed order: of one value, or of two, which the halves of
// a warp share out after their first exchange. Consecutive reductions use the two buffers in turn (turn
// is the caller's count), so one barrier each is enough. Warps that a block does not have count as zeros.
template <int TEAM, int N>
struct BlockSum {
  static constexpr int WARPS = TEAM / 32;
  static_assert(N == 1 || N == 2);
  alignas(16) float part[2][N][WARPS];

  __device__ __forceinline__ void clear() {
    if constexpr (WARPS > 1) {
      for (int i = threadIdx.x; i < 2 * N * WARPS; i += blockDim.x) part[0][0][i] = 0.0f;
      __syncthreads();
    }
  }
  __device__ __forceinline__ void operator()(float (&v)[N], uint32_t &turn) {
    const int lane = threadIdx.x & 31;
    if constexpr (WARPS == 1) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    } else {
      float s = v[0];
      if constexpr (N == 2) {
        const bool second = lane >= 16;
        s = (second ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, second ? v[0] : v[1], 16);
      } else {
        s += __shfl_xor_sync(0xffffffffu, s, 16);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      float(*p)[WARPS] = part[turn++ & 1];
      if (lane == 0) p[0][threadIdx.x >> 5] = s;
      if (N == 2 && lane == 16) p[N - 1][threadIdx.x >> 5] = s;
      __syncthreads();
#pragma unroll
      for (int n = 0; n < N; ++n) {
        v[n] = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; w += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(p[n] + w);
          v[n] += (f.x + f.y) + (f.z + f.w);
        }
      }
    }
  }
};

// Largest value over the block, in every thread; buffers as above.
template <int TEAM>
struct BlockMax {
  static constexpr int WARPS = TEAM / 32;
  alignas(16) uint32_t part[2][WARPS];

  __device__ __forceinline__ void clear() {
    if constexpr (WARPS > 1) {
      for (int i = threadIdx.x; i < 2 * WARPS; i += blockDim.x) part[0][i] = 0;
      __syncthreads();
    }
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t v, uint32_t &turn) {
    v = __reduce_max_sync(0xffffffffu, v);
    if constexpr (WARPS > 1) {
      uint32_t *p = part[turn++ & 1];
      if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = v;
      __syncthreads();
      v = 0;
#pragma unroll
      for (int w = 0; w < WARPS; w += 4) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p + w);
        v = max(max(v, max(q.x, q.y)), max(q.z, q.w));
      }
    }
    return v;
  }
};

// Calls f.operator()<TEAM, E>() with the kind of block that holds a row of K values: 8 a thread up to 256
// columns, else 16.
template <typename F>
auto for_row(int K, F f) {
  if (K <= 256) return f.template operator()<32, 8>();
  if (K <= 512) return f.template operator()<32, 16>();
  if (K <= 2048) return f.template operator()<128, 16>();
  if (K <= 4096) return f.template operator()<256, 16>();
  if (K <= 8192) return f.template operator()<512, 16>();
  return f.template operator()<1024, 16>();
}
// Threads of a row's block (with vectors), and whether they hold nothing but the row.
inline int row_threads(int K, int E) { return ((K + E - 1) / E + 31) / 32 * 32; }
inline bool row_full(int K, int E) { return K % (32 * E) == 0; }
constexpr int kMaxRow = 16384;

// Blocks of `team` threads that make about `threads` on an SM (at most 24 blocks).
constexpr int blocks_per_sm(int team, int threads) {
  const int b = threads / team;
  return b < 1 ? 1 : (b > 24 ? 24 : b);
}

inline bool rows_aligned(const void *p, size_t stride, size_t elem, size_t to) {
  return reinterpret_cast<uintptr_t>(p) % to == 0 && stride * elem % to == 0;
}

}  // namespace svdq
