// Attention over whole prompts: packed sequences, causal, grouped heads.
//
// One pass over the keys with a running maximum m and sum l of each query row:
//   s = q k^T,  p = exp(scale (s - m)),  l += p,  O += p v,
// and out = O / l, lse = scale m + log l at the end.  m only moves when a
// row's maximum passes it by more than 2^8 in the weights (kSlack): the weights then
// stay below 2^8, which neither fp32 sums nor bf16 weights notice, and the
// accumulators are rarely rescaled.
//
// Rows.  The queries of a sequence that read one key head are one list of rows
// (token, query head), token-major, so grouped heads share every key tile; a
// workgroup takes 32 rows per wave and walks the keys in tiles of 64.
//
// Transposed products.  S^T = K Q^T leaves one query row per lane (and its
// other half-wave's lane): maximum and sum are in-lane, with one exchange
// between the halves.  Its registers are also the B operand of O^T += V^T P^T
// as they stand: the order of keys inside a product's 16 is free as long as
// both operands agree, and V^T is read out of the row-major V tile in that
// order by the transposing LDS read (four keys of one column per lane).
//
// LDS.  K and V tiles arrive by HBM-to-LDS DMA, two stages each; the loads of
// tile j + 1 are in flight while tile j is computed.  16-byte chunk c of row r is
// stored at chunk c ^ swizzle(r), so that the 16 lanes of a read touch all banks.
//
// Values of keys a row does not see get weight 0, which a NaN or infinity
// would survive.  Keys past a sequence's end read as zeros; a later key inside
// a tile cannot be told from a seen one by then, so a workgroup that ends with
// a non-finite accumulator runs again with the non-finite values of partly
// seen tiles zeroed, and recomputes by plain loops the rows that really see one.
#include <hip/hip_runtime.h>

#include "elem.hpp"
#include "layer.hpp"
#include "mfma_tile.hpp"

namespace sgt {

namespace {

constexpr int kKeys = 64;                    // keys per tile
constexpr float kSlack = 8.f;                // log2 of the largest weight before m moves
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4_t* lds_s16x4_ptr;

// Chunk swizzles of the K and V tiles (rows of kD * 2 bytes).
template <int kD> __device__ __forceinline__ int k_swz(int row) { return kD == 128 ? (row & 15) : ((row >> 1) & 7); }
template <int kD> __device__ __forceinline__ int v_swz(int row) {
  return kD == 128 ? (row & 3) << 2 : ((row >> 1) & 1) << 2;
}

// v of the lane 32 away.
__device__ __forceinline__ float other_half(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

struct Tile1 {
  int seq;        // sequence, or -1: no such tile
  int64_t q0, k0; // its first query and key
  int Lq, Lk;
  int tile;       // row tile inside the sequence
};

__device__ __forceinline__ int wave_sum_i(int v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Row tiles of sequence s (0 past the end).
__device__ __forceinline__ int seq_tiles(const PromptArgs& a, int s, int G, int rows) {
  if (s >= a.n_seqs) return 0;
  const int64_t b = min(max((int64_t)a.cu_q[s], (int64_t)0), a.total_q);
  const int64_t e = min(max((int64_t)a.cu_q[s + 1], b), a.total_q);
  return (int)(((e - b) * G + rows - 1) / rows);
}

// The w-th tile in the order: tiles far down their sequence first (with a
// causal mask they see the most keys), level by level, sequences in order
// inside a level.  Every wave of the workgroup computes it for itself, 64
// sequences at a time.
__device__ __forceinline__ Tile1 find_tile(const PromptArgs& a, int w, int G, int rows) {
  const int lane = threadIdx.x & 63;
  const bool one = a.n_seqs <= 64;
  const int mine = seq_tiles(a, lane, G, rows);
  int top = mine;
  for (int c = 64; c < a.n_seqs; c += 64) top = max(top, seq_tiles(a, c + lane, G, rows));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, __shfl_xor(top, o));
  auto above = [&](int level) {   // tiles at levels >= level
    int n = max(mine - level, 0);
    if (!one)
      for (int c = 64; c < a.n_seqs; c += 64) n += max(seq_tiles(a, c + lane, G, rows) - level, 0);
    return wave_sum_i(n);
  };
  Tile1 t{};
  t.seq = -1;
  if (above(0) <= w) return t;
  int lo = 0, hi = top;           // above(lo) > w, above(hi) = 0
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (above(mid) > w) lo = mid; else hi = mid;
  }
  int k = w - above(lo + 1);      // place inside level lo
  for (int c = 0; c < a.n_seqs; c += 64) {
    uint64_t has = __ballot((c == 0 ? mine : seq_tiles(a, c + lane, G, rows)) > lo);
    const int n = __popcll(has);
    if (k >= n) {
      k -= n;
      continue;
    }
    for (; k > 0; --k) has &= has - 1;
    const int s = c + __ffsll((unsigned long long)has) - 1;
    t.seq = s;
    t.tile = lo;
    t.q0 = min(max((int64_t)a.cu_q[s], (int64_t)0), a.total_q);
    t.Lq = (int)(min(max((int64_t)a.cu_q[s + 1], t.q0), a.total_q) - t.q0);
    t.k0 = min(max((int64_t)a.cu_k[s], (int64_t)0), a.total_k);
    t.Lk = (int)(min(max((int64_t)a.cu_k[s + 1], t.k0), a.total_k) - t.k0);
    break;
  }
  return t;
}

// DMA of one operand's tiles: kW waves fill kKeys rows of kD bf16.
template <int kD, int kW, bool kIsV>
struct TileDma {
  static constexpr int kLoads = kKeys * kD * 2 / 1024 / kW;   // 1 KiB loads per wave
  static constexpr int kRowChunks = kD / 8, kRowsPerLoad = 64 / kRowChunks;
  const uint16_t* base;   // key 0 of the sequence and head
  int64_t stride;         // bytes between keys
  int Lk;
  uint32_t off[kLoads];

  __device__ __forceinline__ void init(const uint16_t* p, int64_t token_stride, int keys) {
    const int lane = threadIdx.x & 63;
    base = p;
    stride = token_stride * 2;
    Lk = keys;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = (wave_id() * kLoads + i) * kRowsPerLoad + lane / kRowChunks;
      const int chunk = (lane % kRowChunks) ^ (kIsV ? v_swz<kD>(row) : k_swz<kD>(row));
      off[i] = (uint32_t)(row * stride + chunk * 16);
    }
  }
  // Rows past the sequence's end lie past the records and read as zero.
  __device__ __forceinline__ void issue(uint8_t* stage, int j0) const {
    const int rows = min(Lk - j0, kKeys);
    const char* p = reinterpret_cast<const char*>(base) + j0 * stride;
    const __amdgpu_buffer_rsrc_t rsrc = make_rsrc(p, rows > 0 ? (uint64_t)(rows - 1) * stride + kD * 2 : 0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr_t)(stage + (wave_id() * kLoads + i) * 1024), 16, off[i],
                                               0, 0, 0);
  }
};

template <int kD>
struct RowState {
  f32x16_t o[kD / 32];   // O^T: lane l holds row l % 32; o[b][r] is column 32 b + 8 (r / 4) + 4 (l / 32) + r % 4
  float m, l;            // reference maximum of the raw scores, sum of the weights (this lane's half of the keys)
  float limit;           // scores above it move m
  float mc;              // m in the weights' exponent, or 0 while m is -infinity
};

// One key tile: scores, weights, products.  `seen` is how many of the tile's
// keys this lane's row sees when kMask (from the first key on).
template <int kD>
__device__ __forceinline__ void tile_step(const uint8_t* sK, const uint8_t* sV, const bf16x8_t (&q)[kD / 16],
                                          RowState<kD>& st, const uint32_t (&ka)[kD / 16], const uint32_t (&va)[kD / 32],
                                          float c, bool mask, int seen) {
  const int half = (threadIdx.x >> 5) & 1;
  f32x16_t s[2];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) s[b][r] = 0.f;
#pragma unroll
  for (int t = 0; t < kD / 16; ++t)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const bf16x8_t k = *reinterpret_cast<const bf16x8_t*>(sK + ka[t] + b * 32 * kD * 2);
      s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q[t], s[b], 0, 0, 0);
    }
  if (mask) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int key = 32 * b + 8 * (r / 4) + 4 * half + r % 4;
        s[b][r] = key < seen ? s[b][r] : -INFINITY;
      }
  }
  float top = fmaxf(s[0][0], s[1][0]);
#pragma unroll
  for (int r = 1; r < 16; ++r) top = fmaxf(fmaxf(s[0][r], s[1][r]), top);
  top = fmaxf(top, other_half(top));
  if (__any(top > st.limit)) {
    const float m = fmaxf(st.m, top), mc = m == -INFINITY ? 0.f : m * c;
    const float f = st.m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(st.mc - mc);
    st.m = m;
    st.mc = mc;
    st.limit = m == -INFINITY ? -INFINITY : m + kSlack / c;
    st.l *= f;
#pragma unroll
    for (int b = 0; b < kD / 32; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) st.o[b][r] *= f;
  }
  bf16x8_t p[4];   // product step t covers keys 16 t .. 16 t + 15
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int r = 0; r < 16; r += 2) {
      const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][r], c, -st.mc));
      const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][r + 1], c, -st.mc));
      st.l += e0 + e1;
      const bf16x2_t two = __builtin_convertvector(f32x2_t{e0, e1}, bf16x2_t);
      p[2 * b + r / 8][r % 8] = two[0];
      p[2 * b + r / 8][r % 8 + 1] = two[1];
    }
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int b = 0; b < kD / 32; ++b) {
      const uint8_t* at = sV + va[b] + t * 16 * kD * 2;
      const s16x4_t v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(at));
      const s16x4_t v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(at + 8 * kD * 2));
      const auto v = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
      st.o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, v), p[t], st.o[b], 0, 0, 0);
    }
}

// Zero the non-finite values of a V tile in LDS.
template <int kD, int kW>
__device__ __forceinline__ void zero_nonfinite(uint8_t* sV) {
  uint32_t* w = reinterpret_cast<uint32_t*>(sV);
  for (int i = threadIdx.x; i < kKeys * kD / 2; i += 64 * kW) {
    uint32_t v = w[i];
    if ((v & 0x7F80u) == 0x7F80u) v &= 0xFFFF0000u;
    if ((v & 0x7F800000u) == 0x7F800000u) v &= 0xFFFFu;
    w[i] = v;
  }
}

// One row by plain loops, the dimensions over the lanes.  Returns whether it holds a value that is not finite, and
// if so stores it.
template <int kD>
__device__ __forceinline__ bool plain_row(const PromptArgs& a, int64_t t, int h, int hk, int64_t k0, int seen) {
  constexpr int kPer = kD / 64;
  const int lane = threadIdx.x & 63;
  float q[kPer], acc[kPer] = {};
#pragma unroll
  for (int i = 0; i < kPer; ++i) q[i] = bf16_to_f32(a.q[t * a.q_token + h * a.q_head + lane + 64 * i]);
  float m = -INFINITY, l = 0.f;
  for (int64_t j = k0; j < k0 + seen; ++j) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) z += q[i] * bf16_to_f32(a.k[j * a.k_token + hk * a.k_head + lane + 64 * i]);
    z = wave_sum(z) * a.scale;
    const float mn = fmaxf(m, z), base = mn == -INFINITY ? 0.f : mn;
    const float r = expf(m - base), p = expf(z - base);
    l = l * r + p;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      acc[i] = acc[i] * r + p * bf16_to_f32(a.v[j * a.v_token + hk * a.v_head + lane + 64 * i]);
    m = mn;
  }
  float out[kPer];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    out[i] = l == 0.f ? 0.f : acc[i] / l;
    bad |= !(fabsf(out[i]) < INFINITY);
  }
  if (!__any(bad)) return false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) a.out[(t * a.Hq + h) * kD + lane + 64 * i] = f32_to_bf16(out[i]);
  if (a.lse && lane == 0) a.lse[t * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
  return true;
}

template <int kD, int kW>
__global__ void __launch_bounds__(64 * kW, 2) attn_prompt_kernel(PromptArgs a) {
  constexpr int kTileBytes = kKeys * kD * 2, kRows = 32 * kW;
  __shared__ __attribute__((aligned(1024))) uint8_t sK0[kTileBytes], sK1[kTileBytes], sV0[kTileBytes], sV1[kTileBytes];
  const int lane = threadIdx.x & 63, half = lane >> 5, w = wave_id();
  const int G = a.Hq / a.Hkv, hk = blockIdx.x % a.Hkv;
  const Tile1 t = find_tile(a, blockIdx.x / a.Hkv, G, kRows);
  if (t.seq < 0) return;
  const int rows = t.Lq * G, r0 = t.tile * kRows;
  const int row = r0 + w * 32 + (lane & 31);
  const bool valid = row < rows;
  const int token = row / G, head = hk * G + row % G;
  auto limit_of = [&](int tok) { return a.causal ? min(max(t.Lk - t.Lq + tok + 1, 0), t.Lk) : t.Lk; };
  const int my_seen = valid ? limit_of(token) : 0;
  // keys the workgroup's last row, this wave's last row and its first row see
  const int wg_keys = limit_of((min(r0 + kRows, rows) - 1) / G);
  const int w_first = r0 + w * 32, w_last = min(w_first + 32, rows) - 1;
  const int w_keys = __builtin_amdgcn_readfirstlane(w_first < rows ? limit_of(w_last / G) : 0);
  const int w_all = __builtin_amdgcn_readfirstlane(w_first < rows ? limit_of(w_first / G) : 0);
  const int tiles = (wg_keys + kKeys - 1) / kKeys;

  // exponent of a weight per unit of score; a negative scale's sign goes to q, scale 0 to a factor that rounds away
  const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);
  bf16x8_t q[kD / 16];
  {
    const uint16_t* p = a.q + (t.q0 + token) * a.q_token + head * a.q_head + 8 * half;
    const u32x4_t flip = a.scale < 0.f ? u32x4_t{0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u} : u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kD / 16; ++i) {
      u32x4_t v = {0, 0, 0, 0};
      if (valid) v = *reinterpret_cast<const u32x4_t*>(p + 16 * i);
      q[i] = __builtin_bit_cast(bf16x8_t, v ^ flip);
    }
  }
  uint32_t ka[kD / 16], va[kD / 32];
#pragma unroll
  for (int i = 0; i < kD / 16; ++i)
    ka[i] = (uint32_t)((lane & 31) * kD * 2 + (((2 * i + half) ^ k_swz<kD>(lane & 31)) << 4));
#pragma unroll
  for (int b = 0; b < kD / 32; ++b) {
    const int key = 4 * half + ((lane & 15) >> 2), chunk = 4 * b + ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
    va[b] = (uint32_t)(key * kD * 2 + ((chunk ^ v_swz<kD>(key)) << 4) + (lane & 1) * 8);
  }
  TileDma<kD, kW, false> kd;
  TileDma<kD, kW, true> vd;
  kd.init(a.k + t.k0 * a.k_token + hk * a.k_head, a.k_token, t.Lk);
  vd.init(a.v + t.k0 * a.v_token + hk * a.v_head, a.v_token, t.Lk);

  RowState<kD> st;
  auto pass = [&](bool again) {
#pragma unroll
    for (int b = 0; b < kD / 32; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) st.o[b][r] = 0.f;
    st.m = -INFINITY;
    st.limit = -INFINITY;
    st.l = st.mc = 0.f;
    if (tiles == 0) return;
    kd.issue(sK0, 0);
    vd.issue(sV0, 0);
    auto step = [&](int j, const uint8_t* cK, uint8_t* cV, uint8_t* nK, uint8_t* nV) {
      wait_dma();          // tile j has landed (this wave's loads), and for every wave after the barrier,
      __syncthreads();     // which also ends all reads of the other stage
      const int j0 = j * kKeys;
      if (j + 1 < tiles) {
        kd.issue(nK, j0 + kKeys);
        vd.issue(nV, j0 + kKeys);
      }
      if (again) {
        zero_nonfinite<kD, kW>(cV);
        __syncthreads();
      }
      if (j0 < w_keys) tile_step<kD>(cK, cV, q, st, ka, va, c, j0 + kKeys > w_all, my_seen - j0);
    };
    for (int j = 0;;) {
      step(j, sK0, sV0, sK1, sV1);
      if (++j == tiles) break;
      step(j, sK1, sV1, sK0, sV0);
      if (++j == tiles) break;
    }
  };
  pass(false);
  auto non_finite = [&] {
    float top = 0.f;
#pragma unroll
    for (int b = 0; b < kD / 32; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = abs_max(top, st.o[b][r]);
    top = abs_max(top, other_half(top));
    return valid && !(top < INFINITY);
  };
  const bool bad = non_finite();
  bool done = !valid;
  if (__syncthreads_or(bad)) {
    __syncthreads();
    pass(true);
    // rows that were not finite: by plain loops, kept where the row itself sees such a value
    uint64_t todo = __ballot(bad) & 0xFFFFFFFFull;
    while (todo) {
      const int i = __ffsll((unsigned long long)todo) - 1;
      todo &= todo - 1;
      const int rr = w_first + i;
      if (plain_row<kD>(a, t.q0 + rr / G, hk * G + rr % G, hk, t.k0, limit_of(rr / G)) && (lane & 31) == i) done = true;
    }
  }
  if (done) return;
  const float l = st.l + other_half(st.l);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int64_t at = (t.q0 + token) * a.Hq + head;
  if (a.lse && half == 0) a.lse[at] = l == 0.f ? -INFINITY : (st.mc + __builtin_amdgcn_logf(l)) * kLn2;
  // two groups of 8 columns at a time: the lower half-wave ends up with the whole first group, the upper with the second
  uint16_t* out = a.out + at * kD;
#pragma unroll
  for (int b = 0; b < kD / 32; ++b)
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
      uint32_t x[2], y[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(
            f32x2_t{st.o[b][4 * g + 2 * i] * inv, st.o[b][4 * g + 2 * i + 1] * inv}, bf16x2_t));
        y[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(
            f32x2_t{st.o[b][4 * g + 4 + 2 * i] * inv, st.o[b][4 * g + 4 + 2 * i + 1] * inv}, bf16x2_t));
      }
      const auto e0 = __builtin_amdgcn_permlane32_swap(x[0], y[0], false, false);
      const auto e1 = __builtin_amdgcn_permlane32_swap(x[1], y[1], false, false);
      *reinterpret_cast<u32x4_t*>(out + 32 * b + 8 * (g + half)) = u32x4_t{e0[0], e1[0], e0[1], e1[1]};
    }
}

template <int kD, int kW>
hipError_t launch(const PromptArgs& a, hipStream_t stream) {
  // at most one ragged tile for each sequence; workgroups past the last tile exit at once
  const int64_t tiles = a.total_q * (a.Hq / a.Hkv) / (32 * kW) + min((int64_t)a.n_seqs, a.total_q);
  attn_prompt_kernel<kD, kW><<<dim3((unsigned)(tiles * a.Hkv)), dim3(64 * kW), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_prompt(const PromptArgs& a, hipStream_t stream) {
  return a.D == 64 ? launch<64, 8>(a, stream) : launch<128, 8>(a, stream);
}

}  // namespace sgt
