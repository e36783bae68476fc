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

// v of another lane of the row of 16 lanes.
template <int kCtrl> __device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, kCtrl, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), kCtrl, 0xF, 0xF, true);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <int kCtrl> __device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), kCtrl, 0xF, 0xF, true));
}

// f of the values 16 (or 32) lanes apart, in both: a swap of a value with itself leaves the even rows' (the lower half's)
// values in its first result everywhere and the others' in its second.
template <bool kHalves, class F> __device__ __forceinline__ float over_rows(float v, F f) {
  const uint32_t u = __float_as_uint(v);
  const auto r = kHalves ? __builtin_amdgcn_permlane32_swap(u, u, false, false) : __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
template <bool kHalves, class F> __device__ __forceinline__ double over_rows(double v, F f) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)u, hi = (uint32_t)(u >> 32);
  const auto l = kHalves ? __builtin_amdgcn_permlane32_swap(lo, lo, false, false) : __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
  const auto h = kHalves ? __builtin_amdgcn_permlane32_swap(hi, hi, false, false) : __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
  return f(__builtin_bit_cast(double, ((uint64_t)h[0] << 32) | l[0]), __builtin_bit_cast(double, ((uint64_t)h[1] << 32) | l[1]));
}

// Reduction over kL = 16 or 64 neighbouring lanes, the same in each: quad swaps, half-row and row mirrors, then the four rows.
template <int kL, class T, class F> __device__ __forceinline__ T over_lanes(T v, F f) {
  v = f(v, dpp<0xB1>(v));
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x141>(v));
  v = f(v, dpp<0x140>(v));
  if constexpr (kL == 64) {
    v = over_rows<false>(v, f);
    v = over_rows<true>(v, f);
  }
  return v;
}

__device__ __forceinline__ float wave_sum(float v) {
  return over_lanes<64>(v, [](float x, float y) { return x + y; });
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
