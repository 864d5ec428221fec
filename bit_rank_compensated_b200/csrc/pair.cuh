// Two fp32 values in a register pair, for the packed fp32 instructions (each half rounds like its scalar
// counterpart, at half the instructions).
#pragma once

#include <stdint.h>

namespace svdq {

using f32x2 = uint64_t;

__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ f32x2 pair_bits(uint32_t a, uint32_t b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ f32x2 both(float a) { return pair(a, a); }
__device__ __forceinline__ uint32_t lo_bits(f32x2 v) { return static_cast<uint32_t>(v); }
__device__ __forceinline__ uint32_t hi_bits(f32x2 v) { return static_cast<uint32_t>(v >> 32); }
__device__ __forceinline__ float lo(f32x2 v) { return __uint_as_float(lo_bits(v)); }
__device__ __forceinline__ float hi(f32x2 v) { return __uint_as_float(hi_bits(v)); }
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 sub2(f32x2 a, f32x2 b) { return fma2(b, both(-1.0f), a); }

// max(|a|, |b|, |c|); a NaN if one of them is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

}  // namespace svdq
