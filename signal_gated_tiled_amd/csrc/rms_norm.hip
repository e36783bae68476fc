// Root-mean-square norm with the residual's addition, and an output in bf16,
// fp32 or 8 bits with scales.
#include <hip/hip_runtime.h>

#include "elem.hpp"
#include "layer.hpp"

namespace sgt {

namespace {

constexpr int kThreads = 256;

__device__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < kThreads / 64; ++i) t += red[i];
  __syncthreads();
  return t;
}

// One workgroup per row; the row is read once for the sum of squares and once
// more for each thing written.
__global__ void __launch_bounds__(kThreads) rms_norm_kernel(NormArgs a) {
  __shared__ float red[kThreads / 64];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t x0 = t * a.x_stride, r0 = t * a.H;
  auto value = [&](int i) {
    float v = load_elem(a.x, a.x_dtype, x0 + i);
    if (a.residual) v += load_elem(a.residual, a.r_dtype, r0 + i);
    return v;
  };
  float ss = 0.f;
  for (int i = tid; i < a.H; i += kThreads) {
    const float v = value(i);
    ss += v * v;
  }
  const float inv = rsqrtf(block_sum(ss, red) / (float)a.H + a.eps);
  if (a.out_dtype != SGT_F8E4M3) {
    for (int i = tid; i < a.H; i += kThreads) {
      const float v = value(i);
      if (a.sum_out) store_elem(a.sum_out, a.r_dtype, r0 + i, v);
      store_elem(a.out, a.out_dtype, r0 + i, v * inv * load_elem(a.weight, a.w_dtype, i));
    }
    return;
  }
  const int block = a.block > 0 ? a.block : a.H, nb = (a.H + block - 1) / block;
  for (int b = wv; b < nb; b += kThreads / 64) {
    const int end = min(a.H, (b + 1) * block);
    float top = 0.f;
    for (int i = b * block + lane; i < end; i += 64) {
      const float y = value(i) * inv * load_elem(a.weight, a.w_dtype, i);
      top = abs_max(top, y);
    }
    const float scale = f8_scale(wave_abs_max(top));
    for (int i = b * block + lane; i < end; i += 64) {
      const float v = value(i);
      const float y = v * inv * load_elem(a.weight, a.w_dtype, i);
      if (a.sum_out) store_elem(a.sum_out, a.r_dtype, r0 + i, v);
      static_cast<uint8_t*>(a.out)[r0 + i] = f32_to_e4m3(y / scale);
    }
    if (lane == 0) a.scales[t * nb + b] = scale;
  }
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream) {
  rms_norm_kernel<<<dim3((unsigned)a.T), dim3(kThreads), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace sgt
