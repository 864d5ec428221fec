// A row spread over the threads of a block, in registers: what the layer norm's kernels and the row
// quantizer share.
//
// Thread t of TEAM holds E values: VEC consecutive ones at columns (v TEAM + t) VEC, v = 0 ..
// E / VEC - 1, VEC values being 16 bytes (one load), or VEC = 1 where rows do not start on 16 bytes or
// do not end on a whole vector (consecutive threads on consecutive columns). Columns from K on are
// no one's: value(i) tells whether value i exists.
#pragma once

#include <stdint.h>

#include "i8_quant.cuh"
#include "svdq.h"
#include "types.cuh"

namespace svdq {

template <typename T>
constexpr int kVec = 16 / sizeof(T);

template <int TEAM, int VEC>
__device__ __forceinline__ int row_column(int i) {
  return ((i / VEC) * TEAM + static_cast<int>(threadIdx.x)) * VEC + i % VEC;
}

__device__ __forceinline__ void unpack2(uint32_t w, float &a, float &b, __nv_bfloat16) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack2(uint32_t w, float &a, float &b, __half) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
  a = f.x;
  b = f.y;
}
__device__ __forceinline__ uint32_t pack_pair(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_pair(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// A row's values as loaded (so that a row fetched ahead takes half the registers of its fp32 values).
template <typename T, int TEAM, int VEC, int E>
struct RawRow {
  static constexpr int WORDS = VEC > 1 ? E * static_cast<int>(sizeof(T)) / 4 : E;
  uint32_t w[WORDS];

  __device__ __forceinline__ void load(const T *p, int K) {
    if constexpr (VEC > 1) {
#pragma unroll
      for (int v = 0; v < E / VEC; ++v) {
        const int k = row_column<TEAM, VEC>(v * VEC);
        const uint4 q = k < K ? *reinterpret_cast<const uint4 *>(p + k) : make_uint4(0, 0, 0, 0);
        w[4 * v] = q.x;
        w[4 * v + 1] = q.y;
        w[4 * v + 2] = q.z;
        w[4 * v + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int k = row_column<TEAM, VEC>(i);
        w[i] = k < K ? __float_as_uint(to_f32(p[k])) : 0u;
      }
    }
  }
  __device__ __forceinline__ void values(float (&x)[E]) const {
    if constexpr (VEC > 1 && sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) unpack2(w[i], x[2 * i], x[2 * i + 1], T{});
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = __uint_as_float(w[i]);
    }
  }
};

template <typename T, int TEAM, int VEC, int E>
__device__ __forceinline__ void store_row(T *p, int K, const float (&y)[E]) {
#pragma unroll
  for (int v = 0; v < E / VEC; ++v) {
    const int k = row_column<TEAM, VEC>(v * VEC);
    if (k >= K) continue;
    if constexpr (VEC == 1) {
      p[k] = from_f32<T>(y[v]);
    } else if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4 *>(p + k) = make_float4(y[4 * v], y[4 * v + 1], y[4 * v + 2], y[4 * v + 3]);
    } else {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = pack_pair(y[8 * v + 2 * e], y[8 * v + 2 * e + 1], T{});
      *reinterpret_cast<uint4 *>(p + k) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// The int8 codes of a row, VEC bytes a store, each vector as soon as it is formed.
template <int TEAM, int VEC, int E>
__device__ __forceinline__ void store_codes(int8_t *p, int K, const float (&x)[E], const RowScale &r) {
#pragma unroll
  for (int v = 0; v < E / VEC; ++v) {
    const int k = row_column<TEAM, VEC>(v * VEC);
    if (k >= K) continue;
    uint32_t o[(VEC + 3) / 4];
    i8_pack<VEC>(x + v * VEC, r, o);
    if constexpr (VEC == 1) p[k] = static_cast<int8_t>(o[0]);
    else if constexpr (VEC == 8) *reinterpret_cast<uint2 *>(p + k) = make_uint2(o[0], o[1]);
    else *reinterpret_cast<uint32_t *>(p + k) = o[0];
  }
}

// VEC parameters (of their own type, aligned to the vector's size where VEC > 1) from element `at` on.
// They are read again for every row: the rows of a block, and of the SM's other blocks, find them in L1,
// and the registers stay with the rows in flight.
template <int VEC>
__device__ __forceinline__ void load_params(const void *base, int dtype, size_t at, float (&w)[VEC]) {
  if constexpr (VEC == 1) {
    w[0] = dtype == SVDQ_F32   ? __ldg(static_cast<const float *>(base) + at)
           : dtype == SVDQ_F16 ? to_f32(__ldg(static_cast<const __half *>(base) + at))
                               : to_f32(__ldg(static_cast<const __nv_bfloat16 *>(base) + at));
  } else if (dtype == SVDQ_F32) {
    const float *p = static_cast<const float *>(base) + at;
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      const float4 f = __ldg(reinterpret_cast<const float4 *>(p + e));
      w[e] = f.x, w[e + 1] = f.y, w[e + 2] = f.z, w[e + 3] = f.w;
    }
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(base) + at;
    uint32_t q[VEC / 2];
    if constexpr (VEC == 8) {
      const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
      q[0] = u.x, q[1] = u.y, q[2] = u.z, q[3] = u.w;
    } else {
      const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
      q[0] = u.x, q[1] = u.y;
    }
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      if (dtype == SVDQ_F16) unpack2(q[e], w[2 * e], w[2 * e + 1], __half{});
      else unpack2(q[e], w[2 * e], w[2 * e + 1], __nv_bfloat16{});
    }
  }
}

// f(i, parameter) for every value i of the thread that exists.
template <int TEAM, int VEC, int E, typename F>
__device__ __forceinline__ void with_params(const void *base, int dtype, size_t at, int K, F f) {
#pragma unroll
  for (int v = 0; v < E / VEC; ++v) {
    const int k = row_column<TEAM, VEC>(v * VEC);
    if (k >= K) continue;
    float w[VEC];
    load_params<VEC>(base, dtype, at + k, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) f(v * VEC + e, w[e]);
  }
}

// Rows fetched ahead of the present one: two of 16-bit types, one of fp32 (the same registers).
template <typename T, int TEAM, int VEC, int E>
struct RowsAhead {
  static constexpr int DEPTH = sizeof(T) == 2 && VEC > 1 ? 2 : 1;
  RawRow<T, TEAM, VEC, E> row[DEPTH];

  __device__ __forceinline__ void start(const T *x0, size_t stride, int64_t m0, int64_t m1, int K) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (m0 + d < m1) row[d].load(x0 + (m0 + d) * stride, K);
  }
  // row m's values; fetches row m + DEPTH
  __device__ __forceinline__ void take(const T *x0, size_t stride, int64_t m, int64_t m1, int K, float (&x)[E]) {
    row[0].values(x);
    if constexpr (DEPTH == 2) row[0] = row[1];
    if (m + DEPTH < m1) row[DEPTH - 1].load(x0 + (m + DEPTH) * stride, K);
  }
};

// Sums of N values over the block, in every thread and in a fixed order. Consecutive reductions use the
// two buffers in turn (turn is the caller's count), so one barrier each is enough.
template <int TEAM, int N>
struct BlockSum {
  static constexpr int WARPS = TEAM / 32;
  float part[2][WARPS][N];

  __device__ __forceinline__ void operator()(float (&v)[N], uint32_t &turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    if constexpr (WARPS > 1) {
      float(*p)[N] = part[turn++ & 1];
      if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int n = 0; n < N; ++n) p[threadIdx.x >> 5][n] = v[n];
      __syncthreads();
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += p[w][n];
    }
  }
};

// Largest value over the block, in every thread; buffers as above.
template <int TEAM>
struct BlockMax {
  static constexpr int WARPS = TEAM / 32;
  uint32_t part[2][WARPS];

  __device__ __forceinline__ uint32_t operator()(uint32_t v, uint32_t &turn) {
    v = __reduce_max_sync(0xffffffffu, v);
    if constexpr (WARPS > 1) {
      uint32_t *p = part[turn++ & 1];
      if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = v;
      __syncthreads();
      v = 0;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) v = max(v, p[w]);
    }
    return v;
  }
};

// Calls f.operator()<TEAM, E>() with the block that holds a row of K values: 8 a thread up to 256
// columns, else 16, so that every block of a row has 2 to 32 warps' loads in flight.
template <typename F>
auto for_row(int K, F f) {
  if (K <= 256) return f.template operator()<32, 8>();
  if (K <= 512) return f.template operator()<32, 16>();
  if (K <= 1024) return f.template operator()<64, 16>();
  if (K <= 2048) return f.template operator()<128, 16>();
  if (K <= 4096) return f.template operator()<256, 16>();
  if (K <= 8192) return f.template operator()<512, 16>();
  return f.template operator()<1024, 16>();
}
constexpr int kMaxRow = 16384;

// Blocks an SM holds at most: 1024 threads of 64 registers, at most 16 blocks.
template <int TEAM>
constexpr int kBlocksPerSm = TEAM >= 1024 ? 1 : (1024 / TEAM > 16 ? 16 : 1024 / TEAM);

inline bool rows_aligned(const void *p, size_t stride, size_t elem, size_t to) {
  return reinterpret_cast<uintptr_t>(p) % to == 0 && stride * elem % to == 0;
}

}  // namespace svdq
