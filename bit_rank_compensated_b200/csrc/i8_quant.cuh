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

// rint(127 v / top), ties to even, as the exact quotient rounds: 127 v is exact in fp64, and a quotient
// of 31 by 24 bits that is no tie is further than 2^-34 from one.
__device__ __noinline__ inline int i8_code_exact(float v, float top) {
  return __double2int_rn(127.0 * static_cast<double>(v) / static_cast<double>(top));
}

// Whether the fp32 product t = v * (127 / top) decides the code: it is within 127 * 2^-22 < 2^-14 of the
// quotient, so it does unless it lies that near to a border. (A top below 2^-120, where 127 / top
// overflows, gives infinities and NaNs, which decide nothing.)
__device__ __forceinline__ bool i8_decided(float t, float n) { return fabsf(t - n) < 0.4999f; }

__device__ __forceinline__ int8_t i8_code(float v, const RowScale &r) {
  if (r.top == 0.0f) return 0;
  const float t = v * r.inv, n = rintf(t);
  return static_cast<int8_t>(i8_decided(t, n) ? static_cast<int>(n) : i8_code_exact(v, r.top));
}

// The codes of a thread's values. Hardly any lies near a border, so those that do are marked and taken
// from the exact quotient afterwards.
template <int E>
__device__ __forceinline__ void i8_codes(const float (&v)[E], const RowScale &r, int (&q)[E]) {
  uint32_t near = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float t = v[i] * r.inv, n = rintf(t);
    if (!i8_decided(t, n)) near |= 1u << i;
    q[i] = static_cast<int>(n);
  }
  if (near && r.top != 0.0f) {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (near >> i & 1) q[i] = i8_code_exact(v[i], r.top);
  }
}

}  // namespace svdq
