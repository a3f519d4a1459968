// C ABI of the latent-cache operators (declared in include/hisparse.h):
// argument validation and launches, under the rules of csrc/api.hip.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "hisparse.h"
#include "hs_check.h"
#include "latent.h"

using hs::aligned16;
using hs::check_layout;
using hs::from_hip;
using hs::log2i;

namespace {

constexpr int32_t kMaxRows = 1 << 20;   // heads, query rows an item, tokens, list entries

// Whether the layout's rows are 4-bit ones; HS_ERR_UNSUPPORTED where they are
// neither format.
hs_status row_format(const hs_layout* lay, bool* fp4) {
  if (lay->row_bytes != HS_ROW_FP8 && lay->row_bytes != HS_ROW_FP4) return HS_ERR_UNSUPPORTED;
  *fp4 = lay->row_bytes == HS_ROW_FP4;
  return HS_OK;
}

bool aligned4(const void* p) { return ((uintptr_t)p & 3) == 0; }

// Whether n (> 1) pieces of 64 values a stride apart overlap.
bool overlaps(int32_t n, int64_t stride) { return n > 1 && stride < 64; }

bool bad_stride(int64_t stride, int64_t multiple) { return stride < 0 || stride % multiple != 0; }

}  // namespace

extern "C" {

hs_status hs_mla_append(const hs_layout* layout, const hs_batch* batch, int32_t layer,
                        const hs_append* tokens, int32_t* row_ids, uint16_t* values,
                        hipStream_t stream) {
  hs_status s = check_layout(layout);
  if (s != HS_OK) return s;
  if (!batch || !tokens || layer < 0 || layer >= layout->num_layers)
    return HS_ERR_INVALID_ARGUMENT;
  bool fp4 = false;
  if ((s = row_format(layout, &fp4)) != HS_OK) return s;
  const hs_append& a = *tokens;
  if (a.num_tokens < 0 || a.num_heads < 0 || batch->num_reqs < 0 || batch->max_pages < 1 ||
      (a.rope_interleaved != 0 && a.rope_interleaved != 1) || a.reserved != 0)
    return HS_ERR_INVALID_ARGUMENT;
  if (a.num_heads > kMaxRows) return HS_ERR_UNSUPPORTED;
  if (a.num_tokens == 0) return HS_OK;
  if (!a.token_req || !a.positions || !a.latent || !a.rope || !a.rope_freq || !batch->kv_pool ||
      (batch->num_reqs > 0 && !batch->block_table))
    return HS_ERR_INVALID_ARGUMENT;
  if (!aligned16(batch->kv_pool) || !aligned16(a.latent) || !aligned16(values) ||
      bad_stride(a.latent_stride, 8) || bad_stride(a.rope_stride, 1))
    return HS_ERR_INVALID_ARGUMENT;
  if (a.num_heads > 0 &&
      (!a.q_rope || !a.q_out || !aligned16(a.q_rope) || !aligned16(a.q_out) ||
       bad_stride(a.q_token_stride, 8) || bad_stride(a.q_head_stride, 8) ||
       bad_stride(a.q_out_token_stride, 8) || bad_stride(a.q_out_head_stride, 8) ||
       overlaps(a.num_tokens, a.q_out_token_stride) || overlaps(a.num_heads, a.q_out_head_stride)))
    return HS_ERR_INVALID_ARGUMENT;
  hs::AppendParams p{};
  p.pool = batch->kv_pool + (int64_t)layer * layout->pool_layer_stride;
  p.pool_blocks = layout->pool_rows / layout->page_size;
  p.block_table = batch->block_table;
  p.num_reqs = batch->num_reqs;
  p.max_pages = batch->max_pages;
  p.page_shift = log2i(layout->page_size);
  p.num_tokens = a.num_tokens;
  p.num_heads = a.num_heads;
  p.token_req = a.token_req;
  p.positions = a.positions;
  p.latent = a.latent;
  p.latent_stride = a.latent_stride;
  p.rope = a.rope;
  p.rope_stride = a.rope_stride;
  p.freq = a.rope_freq;
  p.q = a.q_rope;
  p.q_token_stride = a.q_token_stride;
  p.q_head_stride = a.q_head_stride;
  p.q_out = a.q_out;
  p.q_out_token_stride = a.q_out_token_stride;
  p.q_out_head_stride = a.q_out_head_stride;
  p.row_ids = row_ids;
  p.values = values;
  if (!hs::append_fits(p)) return HS_ERR_UNSUPPORTED;
  return from_hip(hs::launch_append(p, fp4, a.rope_interleaved == 1, stream), "append launch");
}

namespace {

// Checks the workspace and the outputs of an absorbed attention call and
// enqueues it.
hs_status attend(hs::DecodeParams p, bool fp4, bool paged, int64_t keys, const void* out,
                 const void* lse, void* workspace, size_t workspace_bytes, const char* what,
                 hipStream_t stream) {
  if (!p.q || !out || !lse || !aligned16(p.q) || !aligned16(out) || !aligned4(lse))
    return HS_ERR_INVALID_ARGUMENT;
  const size_t need = hs::plan_decode(p, keys, paged);
  if (!hs::decode_fits(p)) return HS_ERR_UNSUPPORTED;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return HS_ERR_INVALID_ARGUMENT;
  return from_hip(hs::launch_decode(p, fp4, paged, workspace, stream), what);
}

}  // namespace

hs_status hs_sparse_mla_decode_fp4(const hs_layout* layout, const uint8_t* kv_layer,
                                   const int32_t* row_ids, int32_t num_tokens, int32_t top_k,
                                   const uint16_t* q, int32_t num_heads, float sm_scale,
                                   uint16_t* out, float* lse, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
  hs_status s = check_layout(layout);
  if (s != HS_OK) return s;
  if (layout->row_bytes != HS_ROW_FP4) return HS_ERR_UNSUPPORTED;
  if (num_tokens < 0 || top_k < 0 || num_heads < 1 || !std::isfinite(sm_scale))
    return HS_ERR_INVALID_ARGUMENT;
  if (num_tokens > kMaxRows || top_k > kMaxRows || num_heads > kMaxRows) return HS_ERR_UNSUPPORTED;
  if (num_tokens == 0) return HS_OK;
  if (top_k > 0 && (!kv_layer || !row_ids || !aligned16(kv_layer))) return HS_ERR_INVALID_ARGUMENT;
  hs::DecodeParams p{};
  p.kv = kv_layer;
  p.pool_rows = layout->pool_rows;
  p.row_ids = row_ids;
  p.top_k = top_k;
  p.positions = 1;
  p.heads = p.rows = num_heads;
  p.items = num_tokens;
  p.q = q;
  p.scale = sm_scale;
  p.out = out;
  p.lse = lse;
  return attend(p, true, false, top_k, out, lse, workspace, workspace_bytes,
                "4-bit sparse MLA launch", stream);
}

size_t hs_sparse_mla_fp4_workspace_bytes(int32_t num_tokens, int32_t num_heads, int32_t top_k) {
  if (num_tokens <= 0 || num_heads <= 0 || top_k <= 0) return 0;
  hs::DecodeParams p{};
  p.items = num_tokens;
  p.rows = num_heads;
  return hs::plan_decode(p, top_k, false);
}

hs_status hs_paged_mla_decode(const hs_layout* layout, const hs_batch* batch, int32_t layer,
                              const uint16_t* q, int32_t num_pos, int32_t num_heads,
                              int32_t max_ctx, float sm_scale, uint16_t* out, float* lse,
                              void* workspace, size_t workspace_bytes, hipStream_t stream) {
  hs_status s = check_layout(layout);
  if (s != HS_OK) return s;
  if (!batch || layer < 0 || layer >= layout->num_layers) return HS_ERR_INVALID_ARGUMENT;
  bool fp4 = false;
  if ((s = row_format(layout, &fp4)) != HS_OK) return s;
  if (batch->num_reqs < 0 || batch->max_pages < 1 || num_pos < 1 || num_heads < 1 || max_ctx < 0 ||
      !std::isfinite(sm_scale))
    return HS_ERR_INVALID_ARGUMENT;
  if ((int64_t)num_pos * num_heads > kMaxRows) return HS_ERR_UNSUPPORTED;
  if (batch->num_reqs == 0) return HS_OK;
  if (!batch->kv_pool || !batch->block_table || !batch->ctx_len || !aligned16(batch->kv_pool))
    return HS_ERR_INVALID_ARGUMENT;
  hs::DecodeParams p{};
  p.kv = batch->kv_pool + (int64_t)layer * layout->pool_layer_stride;
  p.pool_rows = layout->pool_rows;
  p.block_table = batch->block_table;
  p.ctx_len = batch->ctx_len;
  p.max_pages = batch->max_pages;
  p.page_shift = log2i(layout->page_size);
  const int64_t table = (int64_t)batch->max_pages << p.page_shift;
  p.max_keys = (int32_t)(table < max_ctx ? table : max_ctx);
  p.positions = num_pos;
  p.heads = num_heads;
  p.rows = num_pos * num_heads;
  p.items = batch->num_reqs;
  p.q = q;
  p.scale = sm_scale;
  p.out = out;
  p.lse = lse;
  // the launch goes by the caller's bound, whatever the table's size: the
  // workspace is a matter of the call's sizes alone
  return attend(p, fp4, true, max_ctx, out, lse, workspace, workspace_bytes, "paged MLA launch",
                stream);
}

size_t hs_paged_mla_workspace_bytes(int32_t num_reqs, int32_t num_pos, int32_t num_heads,
                                    int32_t max_ctx) {
  if (num_reqs <= 0 || num_pos <= 0 || num_heads <= 0 || max_ctx <= 0 ||
      (int64_t)num_pos * num_heads > kMaxRows)
    return 0;
  hs::DecodeParams p{};
  p.items = num_reqs;
  p.rows = num_pos * num_heads;
  return hs::plan_decode(p, max_ctx, true);
}

hs_status hs_mla_prefill(const hs_layout* layout, const hs_batch* batch, int32_t layer,
                         const int32_t* q_start, int32_t num_q, int32_t num_kv, const uint16_t* q,
                         int32_t num_heads, const uint16_t* w_kv, float sm_scale, uint16_t* out,
                         void* workspace, size_t workspace_bytes, hipStream_t stream) {
  hs_status s = check_layout(layout);
  if (s != HS_OK) return s;
  if (!batch || layer < 0 || layer >= layout->num_layers) return HS_ERR_INVALID_ARGUMENT;
  bool fp4 = false;
  if ((s = row_format(layout, &fp4)) != HS_OK) return s;
  if (batch->num_reqs < 0 || batch->max_pages < 1 || num_q < 0 || num_kv < 0 || num_heads < 1 ||
      !std::isfinite(sm_scale))
    return HS_ERR_INVALID_ARGUMENT;
  if (num_heads > kMaxRows || batch->num_reqs > kMaxRows) return HS_ERR_UNSUPPORTED;
  if (batch->num_reqs == 0 || num_q == 0) return HS_OK;
  if (!q_start || !q || !w_kv || !out || !batch->kv_pool || !batch->block_table || !batch->ctx_len)
    return HS_ERR_INVALID_ARGUMENT;
  if (!aligned16(batch->kv_pool) || !aligned16(q) || !aligned16(w_kv) || !aligned16(out) ||
      !aligned4(q_start))
    return HS_ERR_INVALID_ARGUMENT;
  hs::PrefillParams p{};
  p.kv = batch->kv_pool + (int64_t)layer * layout->pool_layer_stride;
  p.pool_rows = layout->pool_rows;
  p.block_table = batch->block_table;
  p.ctx_len = batch->ctx_len;
  p.num_reqs = batch->num_reqs;
  p.max_pages = batch->max_pages;
  p.page_shift = log2i(layout->page_size);
  p.q_start = q_start;
  p.num_q = num_q;
  p.num_kv = num_kv;
  p.q = q;
  p.heads = num_heads;
  p.w = w_kv;
  p.scale = sm_scale;
  p.out = out;
  const size_t need = hs::plan_prefill(p, workspace);
  if (!hs::prefill_fits(p)) return HS_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < need || !aligned16(workspace)) return HS_ERR_INVALID_ARGUMENT;
  return from_hip(hs::launch_prefill(p, fp4, stream), "MLA prefill launch");
}

size_t hs_mla_prefill_workspace_bytes(int32_t num_reqs, int32_t num_q, int32_t num_kv,
                                      int32_t num_heads) {
  if (num_reqs <= 0 || num_q <= 0 || num_kv < 0 || num_heads <= 0) return 0;
  hs::PrefillParams p{};
  p.num_reqs = num_reqs;
  p.num_q = num_q;
  p.num_kv = num_kv;
  p.heads = num_heads;
  return hs::plan_prefill(p, nullptr);
}

}  // extern "C"
