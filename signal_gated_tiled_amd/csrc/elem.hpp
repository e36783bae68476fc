// Element conversions and wave reductions shared by the transformer-layer operators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sgt.h"

namespace sgt {

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// Round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint16_t f32_to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// Element i of a bf16 or fp32 array.
__device__ __forceinline__ float load_elem(const void* p, int dtype, int64_t i) {
  return dtype == SGT_BF16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void store_elem(void* p, int dtype, int64_t i, float v) {
  if (dtype == SGT_BF16)
    static_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
  else
    static_cast<float*>(p)[i] = v;
}

// e4m3 (OCP) of v, round to nearest even; |v| must not exceed 464 (the format ends at 448).
__device__ __forceinline__ uint8_t f32_to_e4m3(float v) {
  return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xFF);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Maximum of non-negative floats by their bits: a NaN is the largest of all, so it is not lost as fmaxf would lose it.
__device__ __forceinline__ float abs_max(float top, float v) {
  const uint32_t a = __float_as_uint(top), b = __float_as_uint(v) & 0x7FFFFFFFu;
  return __uint_as_float(a > b ? a : b);
}

constexpr float kF8Max = 448.f;             // largest e4m3 value
constexpr float kF8MinScale = 0x1p-126f;    // a row of zeros gets the smallest normal scale

// Scale of an 8-bit row or block whose largest magnitude is `top` (NaN stays NaN).
__device__ __forceinline__ float f8_scale(float top) {
  const float s = top / kF8Max;
  return s < kF8MinScale ? kF8MinScale : s;
}

}  // namespace sgt
