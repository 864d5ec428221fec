// The int8 row quantizer's arithmetic, shared by the row quantizer and the layer norm's int8 form.
#pragma once

#include <stdint.h>

namespace svdq {

// |v| as an integer: ordered like |v| for finite values, infinities and NaNs above all of them.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

struct RowScale {
  float scale;  // max / 127; NaN for a row with an infinity or a NaN
  float top;    // max |v| of a finite row that is not all zeros, else 0
  float inv;    // about 127 / top
};

__device__ __forceinline__ RowScale row_scale(uint32_t top_bits) {
  if (top_bits >= 0x7f800000u) return {__uint_as_float(0x7fffffffu), 0.0f, 0.0f};
  const float top = __uint_as_float(top_bits);
  return {__fdiv_rn(top, 127.0f), top, top > 0.0f ? __fdiv_rn(127.0f, top) : 0.0f};
}

// rint(127 v / top), ties to even, as the exact quotient rounds. The fp32 product is within
// 127 * 2^-22 < 2^-14 of the quotient, so it decides unless it lies that near to a border; there
// the fp64 quotient does: 127 v is exact in it, and a quotient of 31 by 24 bits that is no tie is
// further than 2^-34 from one. top below 2^-120 (where 127 / top overflows) always takes that way.
__device__ __forceinline__ int8_t i8_code(float v, const RowScale &r) {
  if (r.top == 0.0f) return 0;
  const float t = v * r.inv;
  const float n = rintf(t);
  if (fabsf(t - n) < 0.4999f && r.inv < 0x1p120f) return static_cast<int8_t>(static_cast<int>(n));
  return static_cast<int8_t>(__double2int_rn(127.0 * static_cast<double>(v) / static_cast<double>(r.top)));
}

// Largest value over the block, in every thread.
template <int THREADS>
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
  __shared__ uint32_t part[THREADS / 32];
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t s = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) s = max(s, part[w]);
  return s;
}

}  // namespace svdq
