// Attention over whole prompts: packed sequences, causal, grouped heads.
#include <hip/hip_runtime.h>

#include "elem.hpp"
#include "layer.hpp"

namespace sgt {

namespace {

constexpr int kWaves = 4;

// One wave per (token, query head), the head's dimensions over the lanes; one
// pass over the keys with a running maximum and sum.
template <int kD>
__global__ void __launch_bounds__(64 * kWaves) attn_prompt_kernel(PromptArgs a) {
  constexpr int kPer = kD / 64;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t item = (int64_t)blockIdx.x * kWaves + wv;
  const int64_t t = item / a.Hq;
  const int h = (int)(item % a.Hq);
  if (t >= a.total_q) return;
  int s = 0;
  while (s + 1 < a.n_seqs && (int64_t)a.cu_q[s + 1] <= t) ++s;
  const int64_t q0 = a.cu_q[s], q1 = a.cu_q[s + 1];
  if (t < q0 || t >= q1) return;
  const int64_t k0 = max((int64_t)a.cu_k[s], (int64_t)0), k1 = min((int64_t)a.cu_k[s + 1], a.total_k);
  const int64_t seen = a.causal ? min(k1, k0 + (t - q0) + (k1 - k0) - (q1 - q0) + 1) : k1;
  const int hk = h / (a.Hq / a.Hkv);
  float q[kPer], acc[kPer] = {};
#pragma unroll
  for (int i = 0; i < kPer; ++i) q[i] = bf16_to_f32(a.q[t * a.q_token + h * a.q_head + lane + 64 * i]);
  float m = -INFINITY, l = 0.f;
  for (int64_t j = k0; j < seen; ++j) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) z += q[i] * bf16_to_f32(a.k[j * a.k_token + hk * a.k_head + lane + 64 * i]);
    z = wave_sum(z) * a.scale;
    const float mn = fmaxf(m, z);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float r = expf(m - base), p = expf(z - base);
    l = l * r + p;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      acc[i] = acc[i] * r + p * bf16_to_f32(a.v[j * a.v_token + hk * a.v_head + lane + 64 * i]);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) a.out[(t * a.Hq + h) * kD + lane + 64 * i] = f32_to_bf16(l == 0.f ? 0.f : acc[i] * inv);
  if (a.lse && lane == 0) a.lse[t * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

hipError_t launch_attn_prompt(const PromptArgs& a, hipStream_t stream) {
  const unsigned grid = (unsigned)((a.total_q * a.Hq + kWaves - 1) / kWaves);
  if (a.D == 64)
    attn_prompt_kernel<64><<<dim3(grid), dim3(64 * kWaves), 0, stream>>>(a);
  else
    attn_prompt_kernel<128><<<dim3(grid), dim3(64 * kWaves), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace sgt
