// Attention of one new token per sequence over a paged key-value cache.
#include <hip/hip_runtime.h>

#include "elem.hpp"
#include "layer.hpp"

namespace sgt {

namespace {

constexpr int kWaves = 4;

// One wave per (sequence, query head), the head's dimensions over the lanes.
template <int kD>
__global__ void __launch_bounds__(64 * kWaves) attn_decode_kernel(DecodeArgs a) {
  constexpr int kPer = kD / 64;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int item = blockIdx.x * kWaves + wv;
  const int b = item / a.Hq, h = item % a.Hq;
  if (b >= a.B) return;
  const int hk = h / (a.Hq / a.Hkv);
  const int64_t room = (int64_t)a.max_pages * a.page_size;
  const int n = (int)min((int64_t)max(a.lens[b], 0), room);
  float q[kPer], acc[kPer] = {};
#pragma unroll
  for (int i = 0; i < kPer; ++i) q[i] = bf16_to_f32(a.q[b * a.q_stride + h * kD + lane + 64 * i]);
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < n; ++j) {
    const int64_t page = a.table[b * a.table_stride + j / a.page_size];
    if (page < 0 || page >= a.n_pages) continue;
    const int64_t at = page * a.page_stride + (j % a.page_size) * a.slot_stride + hk * a.head_stride + lane;
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) z += q[i] * bf16_to_f32(a.k[at + 64 * i]);
    z = wave_sum(z) * a.scale;
    const float mn = fmaxf(m, z);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float r = expf(m - base), p = expf(z - base);
    l = l * r + p;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = acc[i] * r + p * bf16_to_f32(a.v[at + 64 * i]);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int dt = a.out_f32 ? SGT_F32 : SGT_BF16;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    store_elem(a.out, dt, ((int64_t)b * a.Hq + h) * kD + lane + 64 * i, l == 0.f ? 0.f : acc[i] * inv);
  if (a.lse && lane == 0) a.lse[(int64_t)b * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

int64_t attn_decode_workspace(int, int, int, int) { return 16; }

hipError_t launch_attn_decode(const DecodeArgs& a, hipStream_t stream) {
  const unsigned grid = (unsigned)(((int64_t)a.B * a.Hq + kWaves - 1) / kWaves);
  if (a.D == 64)
    attn_decode_kernel<64><<<dim3(grid), dim3(64 * kWaves), 0, stream>>>(a);
  else
    attn_decode_kernel<128><<<dim3(grid), dim3(64 * kWaves), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace sgt
