// Root-mean-square norm with the residual's addition, and an output in bf16,
// fp32 or 8 bits with scales.
//
// The bytes bound this: x and the residual are read once, the sum and the output
// written once.  A row stays in registers between the sum of its squares and its
// scaling: thread t of a row's `lanes` threads holds the vectors of 8 elements t,
// t + lanes, ... (kN of them), each read and written with one 16-byte access per
// 16 bytes.  Rows may start at any element: the accesses need no alignment, and
// the last H % 8 elements of a row are taken one by one by the thread whose
// vector they would begin.
//
// A row of up to 512 kN elements is one wave's (four rows per workgroup, no
// barrier); a longer one takes a workgroup, whose waves exchange their sums
// through LDS.
#include <hip/hip_runtime.h>

#include "elem.hpp"
#include "layer.hpp"

namespace sgt {

namespace {

constexpr int kVec = 8;

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

template <class T> __device__ __forceinline__ T load_any(const void* p) {
  T v;
  __builtin_memcpy(&v, p, sizeof v);   // any alignment
  return v;
}

template <class T> __device__ __forceinline__ void store_any(void* p, T v) { __builtin_memcpy(p, &v, sizeof v); }

// n (1 .. 8) elements from element `at` on; the missing ones are zero.
template <bool kF32>
__device__ __forceinline__ void read_vec(const void* p, int64_t at, int n, float (&v)[kVec]) {
  if (n == kVec) {
    if constexpr (kF32) {
      const u32x4_t a = load_any<u32x4_t>(static_cast<const float*>(p) + at), b = load_any<u32x4_t>(static_cast<const float*>(p) + at + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(a[i]);
        v[i + 4] = __uint_as_float(b[i]);
      }
    } else {
      const u32x4_t a = load_any<u32x4_t>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(a[i] << 16);
        v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    v[i] = 0.f;
    if (i < n) v[i] = kF32 ? static_cast<const float*>(p)[at + i] : bf16_to_f32(static_cast<const uint16_t*>(p)[at + i]);
  }
}

__device__ __forceinline__ void read_vec(const void* p, int dtype, int64_t at, int n, float (&v)[kVec]) {
  if (dtype == SGT_F32) read_vec<true>(p, at, n, v);
  else read_vec<false>(p, at, n, v);
}

__device__ __forceinline__ void write_vec(void* p, int dtype, int64_t at, int n, const float (&v)[kVec]) {
  if (n == kVec) {
    if (dtype == SGT_F32) {
      u32x4_t a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = __float_as_uint(v[i]);
        b[i] = __float_as_uint(v[i + 4]);
      }
      store_any(static_cast<float*>(p) + at, a);
      store_any(static_cast<float*>(p) + at + 4, b);
    } else if (dtype == SGT_BF16) {
      u32x4_t a;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{v[2 * i], v[2 * i + 1]}, bf16x2_t));
      store_any(static_cast<uint16_t*>(p) + at, a);
    } else {
      u32x2_t a;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        a[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(
            v[4 * i + 2], v[4 * i + 3], __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false), true);
      store_any(static_cast<uint8_t*>(p) + at, a);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i)
    if (i < n) {
      if (dtype == SGT_F8E4M3) static_cast<uint8_t*>(p)[at + i] = f32_to_e4m3(v[i]);
      else store_elem(p, dtype, at + i, v[i]);
    }
}

// Largest magnitude over 16 neighbouring lanes.
__device__ __forceinline__ float row16_abs_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = abs_max(v, __shfl_xor(v, o));
  return v;
}

// kWave: a row is one wave's; else the workgroup's.
template <bool kF32, int kN, bool kWave>
__global__ void __launch_bounds__(kWave ? 256 : 1024) rms_norm_kernel(NormArgs a) {
  __shared__ float red[2][16];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int lanes = kWave ? 64 : (int)blockDim.x, t = kWave ? lane : (int)threadIdx.x;
  const int64_t row = kWave ? (int64_t)blockIdx.x * 4 + wv : (int64_t)blockIdx.x;
  if (kWave && row >= a.T) return;
  const int64_t x0 = row * a.x_stride, r0 = row * a.H;
  float s[kN][kVec];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int at = (t + i * lanes) * kVec, n = min(a.H - at, kVec);
    if (n > 0) {
      read_vec<kF32>(a.x, x0 + at, n, s[i]);
      if (a.residual) {
        float r[kVec];
        read_vec(a.residual, a.r_dtype, r0 + at, n, r);
#pragma unroll
        for (int j = 0; j < kVec; ++j) s[i][j] += r[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) s[i][j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) ss += s[i][j] * s[i][j];
  }
  ss = wave_sum(ss);
  if constexpr (!kWave) {
    if (lane == 0) red[0][wv] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < lanes / 64; ++i) ss += red[0][i];
  }
  const float inv = rsqrtf(ss / (float)a.H + a.eps);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int at = (t + i * lanes) * kVec, n = min(a.H - at, kVec);
    if (n <= 0) continue;
    if (a.sum_out) write_vec(a.sum_out, a.r_dtype, r0 + at, n, s[i]);
    float w[kVec];
    read_vec(a.weight, a.w_dtype, at, n, w);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      s[i][j] = s[i][j] * inv * w[j];
      top = abs_max(top, j < n ? s[i][j] : 0.f);
    }
    if (a.out_dtype != SGT_F8E4M3) write_vec(a.out, a.out_dtype, r0 + at, n, s[i]);
  }
  if (a.out_dtype != SGT_F8E4M3) return;
  if (a.block == 0) {
    top = wave_abs_max(top);
    if constexpr (!kWave) {
      if (lane == 0) red[1][wv] = top;
      __syncthreads();
      for (int i = 0; i < lanes / 64; ++i) top = abs_max(top, red[1][i]);
    }
    if (t == 0) a.scales[row] = f8_scale(top);
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int at = (t + i * lanes) * kVec, n = min(a.H - at, kVec);
    if (a.block) {   // a block of 128 columns is 16 neighbouring lanes' vector i
      top = 0.f;
#pragma unroll
      for (int j = 0; j < kVec; ++j) top = abs_max(top, j < n ? s[i][j] : 0.f);
      top = row16_abs_max(top);
      if (n > 0 && (lane & 15) == 0) a.scales[row * ((a.H + 127) / 128) + at / 128] = f8_scale(top);
    }
    if (n <= 0) continue;
    const float scale = f8_scale(top);
#pragma unroll
    for (int j = 0; j < kVec; ++j) s[i][j] = s[i][j] / scale;
    write_vec(a.out, SGT_F8E4M3, r0 + at, n, s[i]);
  }
}

template <bool kF32, int kN>
hipError_t launch(const NormArgs& a, int vecs, hipStream_t stream) {
  if (vecs <= 64 * kN) {
    rms_norm_kernel<kF32, kN, true><<<dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, stream>>>(a);
  } else {
    const int lanes = ((vecs + kN - 1) / kN + 63) / 64 * 64;
    rms_norm_kernel<kF32, kN, false><<<dim3((unsigned)a.T), dim3((unsigned)lanes), 0, stream>>>(a);
  }
  return hipGetLastError();
}

template <bool kF32>
hipError_t launch_type(const NormArgs& a, hipStream_t stream) {
  const int vecs = (a.H + kVec - 1) / kVec;
  // Many rows fill the chip by themselves: four vectors in flight per thread.  Few rows: one each, so that the row's
  // loads are spread over as many waves as it has.  Rows past 8 x 1024 x 4 elements take eight.
  const int n = vecs > 4096 ? 8 : a.T >= 256 || vecs > 1024 ? (vecs > 128 ? 4 : 2) : 1;
  switch (n) {
    case 1: return launch<kF32, 1>(a, vecs, stream);
    case 2: return launch<kF32, 2>(a, vecs, stream);
    case 4: return launch<kF32, 4>(a, vecs, stream);
    default: return launch<kF32, 8>(a, vecs, stream);
  }
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream) {
  return a.x_dtype == SGT_F32 ? launch_type<true>(a, stream) : launch_type<false>(a, stream);
}

}  // namespace sgt
