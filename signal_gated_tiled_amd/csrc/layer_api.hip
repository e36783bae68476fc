// Entry points of the transformer-layer operators (RMS norm, expert gate,
// prompt attention, paged decode attention): argument checks and launches.
// They take no context and keep no state: each runs on the calling thread's
// current device and on the caller's stream, and may be captured.
#include <hip/hip_runtime.h>

#include <cmath>

#include "sgt.h"
#include "api.hpp"
#include "layer.hpp"

using namespace sgt;

namespace {

constexpr int kMaxNormWidth = 65536;
constexpr int kMaxGateExperts = 1024, kMaxGateTopk = 64, kMaxGateGroups = 64;
constexpr int64_t kMaxRows = 0x7FFFFFFF;

bool is_real(int dtype) { return dtype == SGT_F32 || dtype == SGT_BF16; }

int64_t bytes_of(int dtype) { return dtype == SGT_F32 ? 4 : dtype == SGT_BF16 ? 2 : 1; }

bool aligned(const void* p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)n == 0; }

sgt_status check_heads(int Hq, int Hkv, int D) {
  if (Hq < 1 || Hkv < 1 || Hq > 1024 || Hq % Hkv)
    return fail(SGT_EINVAL, "Hq = %d, Hkv = %d (1 <= Hkv, Hq a multiple of Hkv and at most 1024)", Hq, Hkv);
  if (D != 64 && D != 128) return fail(SGT_EUNSUPPORTED, "head dimension %d (64 or 128)", D);
  return SGT_OK;
}

}  // namespace

extern "C" {

sgt_status sgt_rms_norm(const void* x, int x_dtype, int64_t x_stride, const void* residual, void* sum_out, int r_dtype,
                        const void* weight, int w_dtype, void* out, int out_dtype, float* scales, int block, int64_t T,
                        int64_t H, float eps, void* stream) {
  if (!is_real(x_dtype) || !is_real(r_dtype) || !is_real(w_dtype))
    return fail(SGT_EINVAL, "x_dtype %d, r_dtype %d, w_dtype %d (SGT_F32 or SGT_BF16)", x_dtype, r_dtype, w_dtype);
  if (!is_real(out_dtype) && out_dtype != SGT_F8E4M3) return fail(SGT_EINVAL, "out_dtype %d", out_dtype);
  if (T < 0 || T > kMaxRows || H < 1) return fail(SGT_EINVAL, "bad shape T=%lld H=%lld", (long long)T, (long long)H);
  if (H > kMaxNormWidth) return fail(SGT_EUNSUPPORTED, "H = %lld above %d", (long long)H, kMaxNormWidth);
  if (x_stride < H) return fail(SGT_EINVAL, "x_stride %lld below H = %lld", (long long)x_stride, (long long)H);
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(SGT_EINVAL, "eps must be finite and not negative");
  if (out_dtype == SGT_F8E4M3) {
    if (block != 0 && block != 128) return fail(SGT_EINVAL, "block %d (0: a scale per row, or 128)", block);
    if (!scales && T > 0) return fail(SGT_EINVAL, "8-bit output without scales");
  } else if (scales || block) {
    return fail(SGT_EINVAL, "scales and block belong to the 8-bit output");
  }
  if (T == 0) return SGT_OK;
  if (!x || !weight || !out) return fail(SGT_EINVAL, "x, weight or out is NULL");
  if (!aligned(x, bytes_of(x_dtype)) || !aligned(residual, bytes_of(r_dtype)) || !aligned(sum_out, bytes_of(r_dtype)) ||
      !aligned(weight, bytes_of(w_dtype)) || !aligned(out, bytes_of(out_dtype)) || !aligned(scales, 4))
    return fail(SGT_EINVAL, "a buffer is not aligned to its element size");
  NormArgs a{};
  a.x = x; a.residual = residual; a.weight = weight; a.sum_out = sum_out; a.out = out; a.scales = scales;
  a.T = T; a.x_stride = x_stride; a.H = (int32_t)H; a.block = block;
  a.x_dtype = x_dtype; a.r_dtype = r_dtype; a.w_dtype = w_dtype; a.out_dtype = out_dtype;
  a.eps = eps;
  HIP_TRY(launch_rms_norm(a, static_cast<hipStream_t>(stream)));
  return SGT_OK;
}

sgt_status sgt_moe_gate(const void* logits, int dtype, int64_t stride, const float* bias, int32_t* topk_ids, float* gate,
                        int64_t T, int E, int topk, int score, int n_group, int topk_group, int group_top,
                        int renormalize, float scale, void* stream) {
  if (!is_real(dtype)) return fail(SGT_EINVAL, "dtype %d (SGT_F32 or SGT_BF16)", dtype);
  if (score != SGT_SCORE_SOFTMAX && score != SGT_SCORE_SIGMOID) return fail(SGT_EINVAL, "score %d", score);
  if (T < 0 || T > kMaxRows) return fail(SGT_EINVAL, "T = %lld", (long long)T);
  if (E < 1 || E > kMaxGateExperts) return fail(SGT_EINVAL, "E = %d outside [1, %d]", E, kMaxGateExperts);
  if (topk < 1 || topk > kMaxGateTopk || topk > E)
    return fail(SGT_EINVAL, "topk = %d outside [1, min(E, %d)]", topk, kMaxGateTopk);
  if (stride < E) return fail(SGT_EINVAL, "stride %lld below E = %d", (long long)stride, E);
  if (n_group < 1 || n_group > kMaxGateGroups || E % n_group)
    return fail(SGT_EINVAL, "n_group = %d (a divisor of E, at most %d)", n_group, kMaxGateGroups);
  if (topk_group < 1 || topk_group > n_group) return fail(SGT_EINVAL, "topk_group = %d outside [1, %d]", topk_group, n_group);
  if (topk > topk_group * (E / n_group))
    return fail(SGT_EINVAL, "topk = %d above the %d experts of %d groups", topk, topk_group * (E / n_group), topk_group);
  if (group_top != 1 && group_top != 2) return fail(SGT_EINVAL, "group_top = %d (1 or 2)", group_top);
  if (n_group > 1 && group_top > E / n_group) return fail(SGT_EINVAL, "group_top = 2 with groups of one expert");
  if (!std::isfinite(scale)) return fail(SGT_EINVAL, "scale is not finite");
  if (T == 0) return SGT_OK;
  if (!logits || !topk_ids || !gate) return fail(SGT_EINVAL, "logits, topk_ids or gate is NULL");
  if (!aligned(logits, bytes_of(dtype)) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(gate, 4))
    return fail(SGT_EINVAL, "a buffer is not aligned to its element size");
  GateArgs a{};
  a.logits = logits; a.bias = bias; a.ids = topk_ids; a.gate = gate;
  a.T = T; a.stride = stride; a.E = E; a.k = topk;
  a.n_group = n_group; a.topk_group = topk_group; a.group_top = group_top;
  a.sigmoid = score == SGT_SCORE_SIGMOID; a.renormalize = renormalize != 0; a.bf16 = dtype == SGT_BF16;
  a.wide = stride % 4 == 0 && aligned(logits, 4 * bytes_of(dtype));
  a.wide_bias = aligned(bias, 16);
  a.scale = scale;
  HIP_TRY(launch_moe_gate(a, static_cast<hipStream_t>(stream)));
  return SGT_OK;
}

sgt_status sgt_attn_prompt(const void* q, int64_t q_token, int64_t q_head, const void* k, int64_t k_token, int64_t k_head,
                           const void* v, int64_t v_token, int64_t v_head, void* out, float* lse, const int32_t* cu_q,
                           const int32_t* cu_k, int n_seqs, int64_t total_q, int64_t total_k, int Hq, int Hkv, int D,
                           int causal, float scale, void* stream) {
  sgt_status st = check_heads(Hq, Hkv, D);
  if (st != SGT_OK) return st;
  if (n_seqs < 0 || total_q < 0 || total_k < 0 || total_q > kMaxRows || total_k > kMaxRows)
    return fail(SGT_EINVAL, "n_seqs=%d total_q=%lld total_k=%lld", n_seqs, (long long)total_q, (long long)total_k);
  if (!std::isfinite(scale)) return fail(SGT_EINVAL, "scale is not finite");
  const int64_t strides[] = {q_token, q_head, k_token, k_head, v_token, v_head};
  for (int64_t s : strides)
    if (s < 0 || s % 8) return fail(SGT_EINVAL, "stride %lld (elements: a multiple of 8, not negative)", (long long)s);
  // row offsets inside one head are 32-bit
  if (q_token >= (1 << 24) || k_token >= (1 << 24) || v_token >= (1 << 24))
    return fail(SGT_EUNSUPPORTED, "a token stride of 2^24 elements or more");
  if (total_q == 0) return SGT_OK;
  if (n_seqs == 0) return fail(SGT_EINVAL, "total_q = %lld tokens in no sequence", (long long)total_q);
  if (total_q * (Hq / Hkv) > kMaxRows || total_q * Hq / 32 + (int64_t)n_seqs * Hkv > kMaxRows)
    return fail(SGT_EINVAL, "too many rows (tokens x heads) for one launch");
  if (!q || !out || !cu_q || !cu_k || (total_k > 0 && (!k || !v)))
    return fail(SGT_EINVAL, "q, k, v, out, cu_q or cu_k is NULL");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16))
    return fail(SGT_EINVAL, "q, k, v and out must be 16-byte aligned");
  if (!aligned(lse, 4) || !aligned(cu_q, 4) || !aligned(cu_k, 4)) return fail(SGT_EINVAL, "lse, cu_q or cu_k misaligned");
  PromptArgs a{};
  a.q = static_cast<const uint16_t*>(q); a.k = static_cast<const uint16_t*>(k); a.v = static_cast<const uint16_t*>(v);
  a.out = static_cast<uint16_t*>(out); a.lse = lse; a.cu_q = cu_q; a.cu_k = cu_k;
  a.q_token = q_token; a.q_head = q_head; a.k_token = k_token; a.k_head = k_head; a.v_token = v_token; a.v_head = v_head;
  a.total_q = total_q; a.total_k = total_k; a.n_seqs = n_seqs; a.Hq = Hq; a.Hkv = Hkv; a.D = D;
  a.causal = causal != 0; a.scale = scale;
  HIP_TRY(launch_attn_prompt(a, static_cast<hipStream_t>(stream)));
  return SGT_OK;
}

int64_t sgt_attn_decode_workspace_bytes(int B, int Hq, int Hkv, int D) {
  if (B < 0 || (int64_t)B * Hkv > (1 << 24)) return fail(SGT_EINVAL, "B = %d", B);
  sgt_status st = check_heads(Hq, Hkv, D);
  if (st != SGT_OK) return st;
  return attn_decode_workspace();
}

sgt_status sgt_attn_decode(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache, int64_t page_stride,
                           int64_t slot_stride, int64_t head_stride, int64_t n_pages, int page_size,
                           const int32_t* block_table, int64_t table_stride, int max_pages, const int32_t* seq_lens,
                           void* out, int out_dtype, float* lse, void* workspace, int64_t workspace_bytes, int B, int Hq,
                           int Hkv, int D, float scale, void* stream) {
  const int64_t need = sgt_attn_decode_workspace_bytes(B, Hq, Hkv, D);
  if (need < 0) return (sgt_status)need;
  if (!is_real(out_dtype)) return fail(SGT_EINVAL, "out_dtype %d (SGT_F32 or SGT_BF16)", out_dtype);
  if (page_size < 1 || page_size > (1 << 20)) return fail(SGT_EINVAL, "page_size %d outside [1, 2^20]", page_size);
  if (n_pages < 0 || n_pages > kMaxRows) return fail(SGT_EINVAL, "n_pages %lld", (long long)n_pages);
  if (max_pages < 0 || table_stride < max_pages)
    return fail(SGT_EINVAL, "max_pages %d, table_stride %lld", max_pages, (long long)table_stride);
  if ((int64_t)max_pages * page_size > kMaxRows) return fail(SGT_EUNSUPPORTED, "a table of 2^31 tokens or more");
  const int64_t strides[] = {q_stride, page_stride, slot_stride, head_stride};
  for (int64_t s : strides)
    if (s < 0 || s % 8) return fail(SGT_EINVAL, "stride %lld (elements: a multiple of 8, not negative)", (long long)s);
  if (!std::isfinite(scale)) return fail(SGT_EINVAL, "scale is not finite");
  if (B == 0) return SGT_OK;
  if (!q || !out || !seq_lens || !workspace || (max_pages > 0 && !block_table) || (n_pages > 0 && (!k_cache || !v_cache)))
    return fail(SGT_EINVAL, "q, k_cache, v_cache, block_table, seq_lens, out or workspace is NULL");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(workspace, 16))
    return fail(SGT_EINVAL, "q, k_cache, v_cache, out and workspace must be 16-byte aligned");
  if (!aligned(lse, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return fail(SGT_EINVAL, "lse, block_table or seq_lens misaligned");
  if (workspace_bytes < need)
    return fail(SGT_EINVAL, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)need);
  DecodeArgs a{};
  a.q = static_cast<const uint16_t*>(q); a.k = static_cast<const uint16_t*>(k_cache);
  a.v = static_cast<const uint16_t*>(v_cache); a.table = block_table; a.lens = seq_lens; a.out = out; a.lse = lse;
  a.workspace = workspace; a.q_stride = q_stride; a.page_stride = page_stride; a.slot_stride = slot_stride;
  a.head_stride = head_stride; a.table_stride = table_stride; a.n_pages = n_pages;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.D = D; a.page_size = page_size; a.max_pages = n_pages > 0 ? max_pages : 0;
  a.out_f32 = out_dtype == SGT_F32; a.scale = scale;
  HIP_TRY(launch_attn_decode(a, static_cast<hipStream_t>(stream)));
  return SGT_OK;
}

}  // extern "C"
