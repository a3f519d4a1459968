// C ABI of the latent-cache operators (declared in include/hisparse.h):
// argument validation and launches, under the rules of csrc/api.hip.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hisparse.h"
#include "hs_check.h"
#include "latent.h"

using hs::aligned16;
using hs::check_layout;
using hs::from_hip;
using hs::log2i;

namespace {

// Whether the layout's rows are 4-bit ones; HS_ERR_UNSUPPORTED where they are
// neither format.
hs_status row_format(const hs_layout* lay, bool* fp4) {
  if (lay->row_bytes != HS_ROW_FP8 && lay->row_bytes != HS_ROW_FP4) return HS_ERR_UNSUPPORTED;
  *fp4 = lay->row_bytes == HS_ROW_FP4;
  return HS_OK;
}

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
  if (a.num_heads > (1 << 20)) return HS_ERR_UNSUPPORTED;
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
       bad_stride(a.q_out_token_stride, 8) || bad_stride(a.q_out_head_stride, 8)))
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
  return from_hip(hs::launch_append(p, fp4, a.rope_interleaved == 1, stream), "append launch");
}

}  // extern "C"
