// Internal interface of the latent-cache operators: rows appended to the pool,
// attention over 4-bit rows, through the block table and in the expanded form.
#pragma once

#include "hs_internal.h"

namespace hs {

// Row formats of the latent cache, told apart by the layout's row_bytes.
constexpr int kFp8RowBytes = 656;  // 512 E4M3, 4 float32 scales, 64 bfloat16
constexpr int kFp4RowBytes = 400;  // 512 E2M1 (two a byte), 16 E8M0 scales, 64 bfloat16

// Rows written at their positions, with the rotation (append.hip).
struct AppendParams {
  uint8_t* pool;            // one layer
  int64_t pool_blocks;
  const int32_t* block_table;
  int32_t num_reqs, max_pages, page_shift;
  int32_t num_tokens, num_heads;
  const int32_t* token_req;
  const int32_t* positions;
  const uint16_t* latent;
  int64_t latent_stride;
  const uint16_t* rope;
  int64_t rope_stride;
  const double* freq;
  const uint16_t* q;
  int64_t q_token_stride, q_head_stride;
  uint16_t* q_out;
  int64_t q_out_token_stride, q_out_head_stride;
  int32_t* row_ids;         // or null
  uint16_t* values;         // or null
  int32_t heads_per_group;  // set by launch_append
};

hipError_t launch_append(AppendParams p, bool fp4, bool interleaved, hipStream_t stream);

}  // namespace hs
