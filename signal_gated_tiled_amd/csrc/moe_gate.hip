// Routing of tokens to experts: softmax or sigmoid scores, a bias that takes
// part in the choice only, groups of experts, top-k and renormalised weights.
#include <hip/hip_runtime.h>

#include "elem.hpp"
#include "layer.hpp"

namespace sgt {

namespace {

constexpr int kWaves = 4;
constexpr int kMaxSlots = 16;   // 1024 experts over 64 lanes

// (value, index) of the largest value over the wave, of equal ones the lowest index.
__device__ __forceinline__ void wave_best(float& v, int& i) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float ov = __shfl_xor(v, o);
    const int oi = __shfl_xor(i, o);
    if (ov > v || (ov == v && oi < i)) {
      v = ov;
      i = oi;
    }
  }
}

constexpr int kNone = 0x7FFFFFFF;

// One wave per token; lane l holds experts l, l + 64, ...
__global__ void __launch_bounds__(64 * kWaves) moe_gate_kernel(GateArgs a) {
  __shared__ float sc[kWaves][64 * kMaxSlots];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kWaves + wv;
  if (t >= a.T) return;
  float x[kMaxSlots], c[kMaxSlots], s[kMaxSlots];
  bool live[kMaxSlots];
  float top = -INFINITY;
#pragma unroll
  for (int q = 0; q < kMaxSlots; ++q) {
    const int e = lane + 64 * q;
    live[q] = e < a.E;
    x[q] = live[q] ? load_elem(a.logits, a.bf16 ? SGT_BF16 : SGT_F32, t * a.stride + e) : -INFINITY;
    if (x[q] != x[q]) x[q] = -INFINITY;
    top = fmaxf(top, x[q]);
  }
  top = wave_max(top);
  float total = 0.f;
#pragma unroll
  for (int q = 0; q < kMaxSlots; ++q) {
    if (a.sigmoid)
      s[q] = 1.f / (1.f + expf(-x[q]));
    else
      s[q] = x[q] == top ? (top == -INFINITY ? 0.f : 1.f) : expf(x[q] - top);
    if (!live[q]) s[q] = 0.f;
    total += s[q];
  }
  if (!a.sigmoid) {
    total = wave_sum(total);
    const float inv = total > 0.f ? 1.f / total : 0.f;
#pragma unroll
    for (int q = 0; q < kMaxSlots; ++q) s[q] *= inv;
  }
  const bool by_score = a.bias != nullptr || (a.n_group > 1 && a.group_top > 1);
#pragma unroll
  for (int q = 0; q < kMaxSlots; ++q) {
    const int e = lane + 64 * q;
    c[q] = live[q] && a.bias ? s[q] + a.bias[e] : x[q];
    if (c[q] != c[q]) c[q] = -INFINITY;
    if (a.n_group > 1 && live[q]) sc[wv][e] = by_score ? (a.bias ? c[q] : s[q]) : x[q];
  }
  if (a.n_group > 1) {
    const int per = a.E / a.n_group;
    float g = -INFINITY;
    if (lane < a.n_group) {
      float b1 = -INFINITY, b2 = -INFINITY;
      for (int j = 0; j < per; ++j) {
        const float v = sc[wv][lane * per + j];
        b2 = fmaxf(b2, fminf(b1, v));
        b1 = fmaxf(b1, v);
      }
      g = a.group_top > 1 ? b1 + b2 : b1;
    }
    bool left = lane < a.n_group;
    uint64_t kept = 0;
    for (int j = 0; j < a.topk_group; ++j) {
      float v = left ? g : -INFINITY;
      int i = left ? lane : kNone;
      wave_best(v, i);
      kept |= 1ull << i;
      if (lane == i) left = false;
    }
#pragma unroll
    for (int q = 0; q < kMaxSlots; ++q) {
      const int e = lane + 64 * q;
      if (live[q] && !((kept >> (e / per)) & 1)) live[q] = false;
    }
  }
  float sum = 0.f, mine = 0.f;
  for (int j = 0; j < a.k; ++j) {
    float v = -INFINITY;
    int i = kNone;
#pragma unroll
    for (int q = 0; q < kMaxSlots; ++q)
      if (live[q] && (i == kNone || c[q] > v)) {
        v = c[q];
        i = lane + 64 * q;
      }
    wave_best(v, i);
    float w = 0.f;
#pragma unroll
    for (int q = 0; q < kMaxSlots; ++q)
      if (lane + 64 * q == i) {
        w = s[q];
        live[q] = false;
      }
    w = __shfl(w, i & 63);
    sum += w;
    if (lane == j) {
      mine = w;
      a.ids[t * a.k + j] = i;
    }
  }
  if (lane < a.k) a.gate[t * a.k + lane] = (a.renormalize ? (sum > 0.f ? mine / sum : 0.f) : mine) * a.scale;
}

}  // namespace

hipError_t launch_moe_gate(const GateArgs& a, hipStream_t stream) {
  moe_gate_kernel<<<dim3((unsigned)((a.T + kWaves - 1) / kWaves)), dim3(64 * kWaves), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace sgt
