// C ABI of the 4-bit key/value cache: host-side validation and launches.
#include <math.h>

#include "kv4.h"

using namespace dsv4;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
constexpr int kMaxTokens = 1 << 26, kMaxHeads = 1 << 14, kMaxBlocks = 1 << 22;

dsv4_status to_status(cudaError_t e) {
  if (e == cudaSuccess) return DSV4_OK;
  cudaGetLastError();  // clear a sticky launch-configuration error
  return DSV4_ERR_CUDA;
}

bool valid_batch(int batch, int total, const int32_t *cu, const int32_t *start) {
  return batch > 0 && batch <= 65535 && total >= 0 && total <= kMaxTokens && cu && start;
}

// (a base below 1 turns later pairs faster: 2^-16 keeps every angle, at positions below 2^32, within what cos_sin of
// kv4_heads.cu reduces)
bool valid_rope(const dsv4_rope &r, int dim) {
  return r.rope_dims >= 0 && r.rope_dims % 2 == 0 && r.rope_dims <= dim && (r.rope_dims == 0 || r.rope_base >= 1.52587890625e-5f);
}

bool valid_kv4(const dsv4_kv4_cache &c) {
  if (!c.k_codes || !c.v_codes || !c.k_scales || !c.v_scales || !c.block_table) return false;
  if (c.num_pages <= 0 || c.max_blocks <= 0 || c.max_blocks > kMaxBlocks || c.kv_heads <= 0 || c.kv_heads > kMaxHeads)
    return false;
  return c.dim > 0 && aligned16(c.k_codes) && aligned16(c.v_codes) && aligned16(c.k_scales) && aligned16(c.v_scales);
}

// rows of `heads` heads per token, 16-byte aligned, tokens `stride` elements apart (0: densely)
bool valid_rows(const void *p, int64_t stride, int heads, int dim, dsv4_dtype dt, int64_t *out) {
  *out = stride == 0 ? static_cast<int64_t>(heads) * dim : stride;
  return p && aligned16(p) && *out >= static_cast<int64_t>(heads) * dim && *out % (dt == DSV4_F32 ? 4 : 8) == 0;
}

bool row_dtype(dsv4_dtype d) { return d == DSV4_F32 || d == DSV4_BF16; }

Kv4Cache kernel_cache(const dsv4_kv4_cache &c) {
  Kv4Cache k{};
  k.k_codes = static_cast<uint8_t *>(c.k_codes);
  k.v_codes = static_cast<uint8_t *>(c.v_codes);
  k.k_scales = static_cast<uint8_t *>(c.k_scales);
  k.v_scales = static_cast<uint8_t *>(c.v_scales);
  k.block_table = c.block_table;
  k.num_pages = c.num_pages;
  k.max_blocks = c.max_blocks;
  return k;
}

// `rows`: also the query and output pointers (the workspace size needs only the sizes)
dsv4_status attention_args(const dsv4_kv4_attention_args *a, Kv4AttnLaunch *p, bool rows) {
  if (!a || !valid_batch(a->batch, a->total_tokens, a->cu_seqlens, a->start_pos) || !valid_kv4(a->cache))
    return DSV4_ERR_INVALID_ARG;
  if (a->heads <= 0 || a->heads > kMaxHeads || a->heads % a->cache.kv_heads != 0 || a->dim != a->cache.dim || a->max_new <= 0)
    return DSV4_ERR_INVALID_ARG;
  if (a->softmax_scale != a->softmax_scale || isinf(a->softmax_scale)) return DSV4_ERR_INVALID_ARG;
  if (a->dim != 64 && a->dim != 128) return DSV4_ERR_UNSUPPORTED;
  *p = Kv4AttnLaunch{};
  if (rows && a->total_tokens > 0) {
    if (!valid_rows(a->q, a->q_stride, a->heads, a->dim, DSV4_BF16, &p->q_stride)) return DSV4_ERR_INVALID_ARG;
    if (!a->out || !aligned16(a->out)) return DSV4_ERR_INVALID_ARG;
  }
  p->B = a->batch;
  p->T = a->total_tokens;
  p->Hq = a->heads;
  p->Hk = a->cache.kv_heads;
  p->D = a->dim;
  p->max_new = a->max_new;
  p->q = static_cast<const uint16_t *>(a->q);
  p->cu_seqlens = a->cu_seqlens;
  p->start_pos = a->start_pos;
  p->cache = kernel_cache(a->cache);
  p->softmax_scale = a->softmax_scale > 0.f ? a->softmax_scale : 1.f / sqrtf(static_cast<float>(a->dim));
  p->out = static_cast<uint16_t *>(a->out);
  p->lse = a->lse;
  p->d_status = a->d_status;
  return DSV4_OK;
}

}  // namespace

extern "C" {

dsv4_status dsv4_qk_norm_rope(const dsv4_qk_norm_rope_args *a, dsv4_stream stream) {
  if (!a || !valid_batch(a->batch, a->total_tokens, a->cu_seqlens, a->start_pos)) return DSV4_ERR_INVALID_ARG;
  if (a->q_heads < 0 || a->k_heads < 0 || a->q_heads > kMaxHeads || a->k_heads > kMaxHeads ||
      a->q_heads + a->k_heads == 0)
    return DSV4_ERR_INVALID_ARG;
  if (a->dim <= 0 || !valid_rope(a->rope, a->dim) || !(a->eps >= 0.f)) return DSV4_ERR_INVALID_ARG;
  if (!row_dtype(a->dtype) || !row_dtype(a->out_dtype)) return DSV4_ERR_UNSUPPORTED;
  if (a->dim != 64 && a->dim != 128 && a->dim != 256 && a->dim != 512) return DSV4_ERR_UNSUPPORTED;
  if (a->total_tokens == 0) return DSV4_OK;
  Kv4HeadsLaunch p{};
  if (a->q_heads > 0 && (!valid_rows(a->q, a->q_stride, a->q_heads, a->dim, a->dtype, &p.q_stride) || !a->q_out ||
                         !aligned16(a->q_out)))
    return DSV4_ERR_INVALID_ARG;
  if (a->k_heads > 0 && (!valid_rows(a->k, a->k_stride, a->k_heads, a->dim, a->dtype, &p.k_stride) || !a->k_out ||
                         !aligned16(a->k_out)))
    return DSV4_ERR_INVALID_ARG;
  p.B = a->batch;
  p.T = a->total_tokens;
  p.Hq = a->q_heads;
  p.Hk = a->k_heads;
  p.D = a->dim;
  p.q = a->q;
  p.k = a->k;
  p.in_dt = a->dtype;
  p.out_dt = a->out_dtype;
  p.gamma_q = a->gamma_q;
  p.gamma_k = a->gamma_k;
  p.eps = a->eps;
  p.rope_dims = a->rope.rope_dims;
  p.rope_base = a->rope.rope_base;
  p.cu_seqlens = a->cu_seqlens;
  p.start_pos = a->start_pos;
  p.q_out = a->q_out;
  p.k_out = a->k_out;
  p.d_status = a->d_status;
  return to_status(launch_kv4_heads(p, static_cast<cudaStream_t>(stream)));
}

dsv4_status dsv4_kv4_append(const dsv4_kv4_append_args *a, dsv4_stream stream) {
  if (!a || !valid_batch(a->batch, a->total_tokens, a->cu_seqlens, a->start_pos) || !valid_kv4(a->cache))
    return DSV4_ERR_INVALID_ARG;
  if (a->q_heads < 0 || a->q_heads > kMaxHeads) return DSV4_ERR_INVALID_ARG;
  if (!valid_rope(a->rope, a->cache.dim) || !(a->eps >= 0.f)) return DSV4_ERR_INVALID_ARG;
  if (!row_dtype(a->dtype) || (a->q_heads > 0 && !row_dtype(a->q_out_dtype))) return DSV4_ERR_UNSUPPORTED;
  if (a->cache.dim != 64 && a->cache.dim != 128) return DSV4_ERR_UNSUPPORTED;
  if (a->total_tokens == 0) return DSV4_OK;
  Kv4HeadsLaunch p{};
  const int Hk = a->cache.kv_heads, D = a->cache.dim;
  if (!valid_rows(a->k, a->k_stride, Hk, D, a->dtype, &p.k_stride) ||
      !valid_rows(a->v, a->v_stride, Hk, D, a->dtype, &p.v_stride))
    return DSV4_ERR_INVALID_ARG;
  if (a->q_heads > 0 && (!valid_rows(a->q, a->q_stride, a->q_heads, D, a->dtype, &p.q_stride) || !a->q_out ||
                         !aligned16(a->q_out)))
    return DSV4_ERR_INVALID_ARG;
  if (!aligned16(a->k_stored) || !aligned16(a->v_stored)) return DSV4_ERR_INVALID_ARG;
  p.B = a->batch;
  p.T = a->total_tokens;
  p.Hq = a->q_heads;
  p.Hk = Hk;
  p.D = D;
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.in_dt = a->dtype;
  p.out_dt = a->q_out_dtype;
  p.gamma_q = a->gamma_q;
  p.gamma_k = a->gamma_k;
  p.eps = a->eps;
  p.rope_dims = a->rope.rope_dims;
  p.rope_base = a->rope.rope_base;
  p.cu_seqlens = a->cu_seqlens;
  p.start_pos = a->start_pos;
  p.q_out = a->q_out;
  p.k_stored = static_cast<uint16_t *>(a->k_stored);
  p.v_stored = static_cast<uint16_t *>(a->v_stored);
  p.cache = kernel_cache(a->cache);
  p.d_status = a->d_status;
  return to_status(launch_kv4_heads(p, static_cast<cudaStream_t>(stream)));
}

size_t dsv4_kv4_attention_workspace_size(const dsv4_kv4_attention_args *a) {
  Kv4AttnLaunch p;
  if (attention_args(a, &p, false) != DSV4_OK) return 0;
  return kv4_attention_workspace_bytes(p, kv4_attention_plan(p));
}

size_t dsv4_kv4_attention_workspace_limit(const dsv4_kv4_attention_args *a) {
  Kv4AttnLaunch p;
  if (attention_args(a, &p, false) != DSV4_OK) return 0;
  return kv4_attention_workspace_limit(p);
}

dsv4_status dsv4_kv4_attention_plan(const dsv4_kv4_attention_args *a, dsv4_kv4_plan *out) {
  Kv4AttnLaunch p;
  if (!out) return DSV4_ERR_INVALID_ARG;
  const dsv4_status s = attention_args(a, &p, false);
  if (s != DSV4_OK) return s;
  const Kv4AttnPlan plan = kv4_attention_plan(p);
  const bool prompt = plan.form == DSV4_KV4_PROMPT;
  out->form = plan.form;
  out->rows = plan.rows;
  out->units = prompt ? plan.shape.row_blocks * p.B * p.Hk : 0;
  out->shared = prompt ? out->units - plan.shape.whole : 0;
  out->splits = prompt ? plan.shape.splits : 0;
  return DSV4_OK;
}

dsv4_status dsv4_kv4_attention(const dsv4_kv4_attention_args *a, void *ws, size_t ws_bytes, dsv4_stream stream) {
  Kv4AttnLaunch p;
  const dsv4_status s = attention_args(a, &p, true);
  if (s != DSV4_OK) return s;
  if (p.T == 0) return DSV4_OK;
  const Kv4AttnPlan plan = kv4_attention_plan(p);
  if (!ws || ws_bytes < kv4_attention_workspace_bytes(p, plan) || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return DSV4_ERR_INVALID_ARG;
  return to_status(launch_kv4_attention(p, plan, ws, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
