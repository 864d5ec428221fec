// Activation types of the operators around the projections: conversions to and from fp32, of one value and of two.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "pair.cuh"

namespace svdq {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

// Round to nearest even; an fp16 overflow becomes an infinity, as in a plain cast.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

// Two 16-bit values of a word as fp32, and back.
__device__ __forceinline__ f32x2 widen(uint32_t w, __nv_bfloat16) { return pair_bits(w << 16, w & 0xffff0000u); }
__device__ __forceinline__ f32x2 widen(uint32_t w, __half) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
  return pair(f.x, f.y);
}
__device__ __forceinline__ uint32_t narrow(f32x2 v, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo(v), hi(v));
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t narrow(f32x2 v, __half) {
  const __half2 h = __floats2half2_rn(lo(v), hi(v));
  return *reinterpret_cast<const uint32_t *>(&h);
}

}  // namespace svdq
