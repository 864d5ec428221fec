// The int8 row quantizer's arithmetic, shared by the row quantizer and the layer norm's int8 form.
#pragma once

#include <stdint.h>

namespace svdq {

// |v| as an integer: ordered like |v| for finite values, infinities and NaNs above all of them.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

struct RowScale {
  float scale;  // max / 127; NaN for a row with an infinity or a NaN
  float by;     // power of two that brings the row's values where the arithmetic below is exact
  float top;    // by * max |v| of a finite row, else 0
  float inv;    // about 127 / top; 0 for a row of zeros or of no finite maximum
};

__device__ __forceinline__ RowScale row_scale(uint32_t top_bits) {
  if (top_bits >= 0x7f800000u) return {__uint_as_float(0x7fffffffu), 0.0f, 0.0f, 0.0f};
  const float max = __uint_as_float(top_bits);
  const float by = max < 0x1p-60f ? 0x1p90f : (max > 0x1p100f ? 0x1p-30f : 1.0f);
  const float top = max * by;
  return {__fdiv_rn(max, 127.0f), by, top, top > 0.0f ? __fdiv_rn(127.0f, top) : 0.0f};
}

// Whether the fp32 product t = v * (127 / top) decides the code: it is within 127 * 2^-22 < 2^-14 of the
// quotient, so it does unless it lies that near to a border.
__device__ __forceinline__ bool i8_decided(float t, float n) { return fabsf(t - n) < 0.4999f; }

// The code of a value near a border k + 1/2, from the exact comparison of 127 |v| with (k + 1/2) top: the
// former is p + e (a product and its rounding error), and (k + 1/2) top - p, of 32 bits of which 12 at
// least cancel, is exact in one fma. A tie goes to the even code.
__device__ __forceinline__ int i8_code_exact(float v, float t, float top) {
  const float a = fabsf(v), k = floorf(fabsf(t));
  const float p = __fmul_rn(a, 127.0f), e = __fmaf_rn(a, 127.0f, -p);
  const float d = __fmaf_rn(k + 0.5f, top, -p);
  const int n = static_cast<int>(k);
  const int c = d > e ? n : (d < e ? n + 1 : n + (n & 1));
  return v < 0.0f ? -c : c;
}

// rint(127 v / max), ties to even, as the exact quotient rounds.
__device__ __forceinline__ int i8_code(float v, const RowScale &r) {
  if (r.inv == 0.0f) return 0;
  const float x = v * r.by, t = x * r.inv, n = rintf(t);
  return i8_decided(t, n) ? static_cast<int>(n) : i8_code_exact(x, t, r.top);
}

// Codes of VEC values, the first in the lowest byte of o[0]. Hardly any value lies near a border: one test
// for all of them.
template <int VEC>
__device__ __forceinline__ void i8_pack(const float *v, const RowScale &r, uint32_t (&o)[(VEC + 3) / 4]) {
  int q[VEC];
  bool decided = true;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const float t = v[i] * r.by * r.inv, n = rintf(t);
    decided = decided && i8_decided(t, n);
    q[i] = static_cast<int>(n);
  }
  if (!decided) {  // (NaNs of a row without a finite maximum too)
#pragma unroll
    for (int i = 0; i < VEC; ++i) q[i] = i8_code(v[i], r);
  }
  if constexpr (VEC == 1) {
    o[0] = static_cast<uint32_t>(q[0]);
  } else {
#pragma unroll
    for (int e = 0; e < VEC / 4; ++e)
      o[e] = __byte_perm(__byte_perm(q[4 * e], q[4 * e + 1], 0x0040), __byte_perm(q[4 * e + 2], q[4 * e + 3], 0x0040), 0x5410);
  }
}

}  // namespace svdq
