// Internal interface of the latent-cache operators: rows appended to the pool,
// attention over 4-bit rows, through the block table and in the expanded form.
#pragma once

#include "hs_internal.h"

namespace hs {

// Row formats of the latent cache, told apart by the layout's row_bytes.
constexpr int kFp8RowBytes = 656;  // 512 E4M3, 4 float32 scales, 64 bfloat16
constexpr int kFp4RowBytes = 400;  // 512 E2M1 (two a byte), 16 E8M0 scales, 64 bfloat16

// Whether a launch of so many workgroups of so many threads is one that the
// device takes: a grid dimension holds less than 2^32 threads.
inline bool grid_fits(int64_t groups, int threads) {
  return groups >= 0 && groups <= (int64_t)(UINT32_MAX / (uint32_t)threads);
}

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

// Whether the launch's grid is within the device's limits.
bool append_fits(const AppendParams& p);
hipError_t launch_append(AppendParams p, bool fp4, bool interleaved, hipStream_t stream);

// Absorbed latent attention (decode.hip): M query rows an item, 576 wide, over
// the item's keys; 512-wide bfloat16 outputs.
constexpr int kDecodeSplitKeys = 2048;     // keys a split, at most: their row ids are in LDS

constexpr int kDealtReqs = 512;           // requests whose splits the kernel deals out

struct DecodeParams {
  const uint8_t* kv;        // one layer of the pool
  int64_t pool_rows;
  const int32_t* row_ids;   // sparse: [items][top_k]
  int32_t top_k;
  const int32_t* block_table;  // paged: [items][max_pages]
  const int32_t* ctx_len;      // paged: [items]
  int32_t max_pages, page_shift;
  int32_t max_keys;         // paged: keys attended to, at most (the table's, the caller's bound)
  int32_t positions;        // paged: query positions an item
  int32_t heads;
  int32_t items;            // tokens, or requests
  int32_t rows;             // M: heads, or positions * heads
  const uint16_t* q;        // [items][rows][576]
  float scale;
  uint16_t* out;            // [items][rows][512]
  float* lse;               // [items][rows]
  // set by plan_decode and launch_decode
  int32_t tile_rows, row_tiles, splits;  // query rows a workgroup; their tiles
  int32_t round;            // (item, split) places that the chip runs at once
  int64_t keys_per_split;   // a multiple of 32; at most, where part_off is there
  uint16_t* part_o;         // [items * splits][rows][512] IEEE half, normalised and scaled
  float* part_ml;           // [items * splits][rows][6]: maximum, sum, four scales
  int32_t* part_off;        // or null, for fixed splits: [items + 1] the items' first parts
};

// Sets the launch shape for items of about `keys` keys; returns the workspace's bytes.
size_t plan_decode(DecodeParams& p, int64_t keys, bool paged);
int64_t decode_grid(const DecodeParams& p);
hipError_t launch_decode_narrow(const DecodeParams& p, bool fp4, bool paged, hipStream_t stream);
// Whether a planned launch's grid is within the device's limits.
bool decode_fits(const DecodeParams& p);
hipError_t launch_decode(DecodeParams p, bool fp4, bool paged, void* workspace,
                         hipStream_t stream);

constexpr int kPrefillMaxSplits = 16;

// Expanded latent attention of chunks of new tokens (prefill.hip).
struct PrefillParams {
  const uint8_t* kv;        // one layer of the pool
  int64_t pool_rows;
  const int32_t* block_table;
  const int32_t* ctx_len;
  int32_t num_reqs, max_pages, page_shift;
  const int32_t* q_start;   // [reqs + 1]
  int32_t num_q, num_kv;    // queries; tokens of the workspace
  const uint16_t* q;        // [num_q][heads][192]
  int32_t heads;
  const uint16_t* w;        // [heads][128 key + 128 value dimensions][512]
  float scale;
  uint16_t* out;            // [num_q][heads][128]
  // set by plan_prefill
  int32_t tile_rows, max_tiles, splits;
  uint16_t* part_o;         // [splits][num_q][heads][128] IEEE half, normalised and scaled
  float* part_ml;           // [splits][num_q][heads][3]: maximum, sum, scale
  int32_t* off;             // [reqs + 1]
  int32_t* tile_off;        // [reqs + 1]
  uint8_t* flags;           // [num_kv]
  uint16_t* lat;            // [num_kv][512]
  uint16_t* rope;           // [num_kv][64]
  uint16_t* heads_kv;       // [heads][num_kv][256]

  // Request r's first query and its queries, whatever q_start holds.
  __device__ int32_t query_start(int32_t r) const {
    const int32_t s = q_start[r];
    return s < 0 ? 0 : s > num_q ? num_q : s;
  }
};

__device__ inline int32_t query_count(const PrefillParams& p, int32_t r) {
  const int32_t n = p.query_start(r + 1) - p.query_start(r);
  return n < 0 ? 0 : n;
}

// Sets the launch shape and lays out the workspace (null: sizes only); its bytes.
size_t plan_prefill(PrefillParams& p, void* workspace);
// Whether a planned launch's grid is within the device's limits.
bool prefill_fits(const PrefillParams& p);
hipError_t launch_prefill(const PrefillParams& p, bool fp4, hipStream_t stream);

}  // namespace hs
