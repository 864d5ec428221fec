// The int8 row quantizer's arithmetic, shared by the row quantizer, the layer norm's int8 form and the
// 8-bit linear of few tokens.
#pragma once

#include <stdint.h>

#include "pair.cuh"

namespace svdq {

struct RowScale {
  float max;   // the row's largest |v|; NaN for a row with an infinity or a NaN
  float c;     // 127 / max, rounded up
  float by;    // power of two that brings the row's values where the exact way's arithmetic is exact
  float top;   // by * max
  float inv;   // about 127 / top; 0 for a row of zeros or of no finite maximum
  bool exact;  // every code of the row takes the exact way
};

// top_bits: the bits of the row's largest |v| (infinities and NaNs above all others). SHORT: the row's values
// have at most 11 significant bits (i8_pack).
template <bool SHORT>
__device__ __forceinline__ RowScale row_scale(uint32_t top_bits) {
  if (top_bits >= 0x7f800000u) return {__uint_as_float(0x7fffffffu), 0.0f, 0.0f, 0.0f, 0.0f, true};
  const float max = __uint_as_float(top_bits);
  const float by = max < 0x1p-60f ? 0x1p90f : (max > 0x1p100f ? 0x1p-30f : 1.0f);
  const float top = max * by;
  const float inv = top > 0.0f ? __fdiv_ru(127.0f, top) : 0.0f;
  bool exact = by != 1.0f;
  if (SHORT) {
    const uint32_t m = (top_bits >> 13 & 0x3ffu) | 0x400u;  // the 11 significant bits
    exact = exact || (m % 127u == 0 && m != 16 * 127);
  }
  return {max, inv, by, top, inv, exact};
}

// The scale of a row: correctly rounded, and so worth one thread's time only.
__device__ __forceinline__ float scale_of(const RowScale &r) { return __fdiv_rn(r.max, 127.0f); }

// rint(127 v / max), ties to even, as the exact quotient rounds: with k below the quotient, 127 |v| is
// compared with (k + 1/2) top. The former is p + e (a product and its rounding error); near the border
// (k + 1/2) top - p, of 32 bits of which 12 at least cancel, is exact in one fma.
__device__ __forceinline__ int i8_code(float v, const RowScale &r) {
  if (r.inv == 0.0f) return 0;
  const float x = v * r.by, t = x * r.inv, n = rintf(t);
  if (fabsf(t - n) < 0.4999f) return static_cast<int>(n);
  const float a = fabsf(x), k = floorf(fabsf(t));
  const float p = __fmul_rn(a, 127.0f), e = __fmaf_rn(a, 127.0f, -p);
  const float d = __fmaf_rn(k + 0.5f, r.top, -p);
  const int i = static_cast<int>(k);
  const int c = d > e ? i : (d < e ? i + 1 : i + (i & 1));  // a tie goes to the even code
  return x < 0.0f ? -c : c;
}

// Codes of 2 N values, the first in the lowest byte of o[0] (N = 1: both in o[0]). Adding 1.5 * 2^23 rounds
// v c to an integer whose last byte is the code.
//
// In general v c, at most 127 * 2^-23 = 1.5e-5 above the quotient, decides unless it lies that near to a
// border (0.49997 of a step from the integer): one value in 17000 does, and one test serves them all.
//
// Values of at most 11 bits need no test. With v = x 2^i and max = a 2^j, x and a integers below 2^11, a quotient
// t = 127 v / max that is no tie is further than t 2^-19 from one (254 x 2^i - (2 k + 1) a 2^j is a
// multiple of 2^i), and v c is within t 2^-23. A tie, 254 x 2^i = (2 k + 1) a 2^j, wants 127 to divide 2 k + 1
// or a. The former is half the maximum, 63.5, which often occurs: c above 127 / max sends it to 64, as the tie
// goes. The latter makes the row an exact one, unless a / 127 is a power of two: then c has no error and the
// addition rounds the tie itself. (Testing and taking the exact way for every vector with a half of the
// maximum in it took 16.4 us for 4608 x 4096 values of bf16; this takes 10.5.)
template <int N, bool SHORT>
__device__ __forceinline__ void i8_pack(const f32x2 *v, const RowScale &r, uint32_t (&o)[(N + 1) / 2]) {
  const f32x2 c = both(r.c), magic = both(12582912.0f);
  uint32_t q[2 * N];
  float far = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const f32x2 s = fma2(v[i], c, magic);
    q[2 * i] = lo_bits(s);
    q[2 * i + 1] = hi_bits(s);
    if constexpr (!SHORT) {
      const f32x2 d = fma2(v[i], c, sub2(magic, s));  // v c - n
      far = max_abs3(far, lo(d), hi(d));
    }
  }
  if (r.exact || !(far < 0.49997f)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      q[2 * i] = static_cast<uint32_t>(i8_code(lo(v[i]), r));
      q[2 * i + 1] = static_cast<uint32_t>(i8_code(hi(v[i]), r));
    }
  }
  if constexpr (N == 1) {
    o[0] = __byte_perm(q[0], q[1], 0x0040);
  } else {
#pragma unroll
    for (int e = 0; e < N / 2; ++e)
      o[e] = __byte_perm(__byte_perm(q[4 * e], q[4 * e + 1], 0x0040), __byte_perm(q[4 * e + 2], q[4 * e + 3], 0x0040), 0x5410);
  }
}

}  // namespace svdq
