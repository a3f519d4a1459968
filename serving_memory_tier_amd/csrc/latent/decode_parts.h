// What the two absorbed latent attention kernels share: a workgroup's share of
// the work, its row ids, and rows on their way into LDS.
#pragma once

#include "latent.h"
#include "parts.h"

namespace hs {
namespace {

constexpr int kKeys = 32;                    // rows a block
constexpr int kLatent = 512;
constexpr int kDim = 576;
constexpr int32_t kBad = -2;                 // in place of a fetched row's id: see sanitize_rows

// A (split, query row)'s floats in part_ml: its maximum, its sum, and the scales of
// its four times 128 partial outputs.
constexpr int kPartFloats = 6;

// The lists of a workgroup of ROWS query rows.
template <int ROWS>
struct Lists {
  int32_t ids[kDecodeSplitKeys];                   // row ids, -1 where there is none; kBad
  int32_t mine[ROWS];                        // keys of the split that a query row sees
  uint32_t there[kDecodeSplitKeys / 32];           // a block's keys that have a row
};

// A workgroup's share: keys [lo, lo + n) of its item for query rows from row0.
struct Share {
  int32_t item, row0;
  int64_t part;                              // its place among the partial outputs
  int64_t lo;
  int n, edge;                               // the first query row sees the fewest keys, `edge`
};

// The paged form's splits for up to kDealtReqs requests.  The launch has items *
// splits places, enough for contexts of the caller's bound; here, where the
// contexts are known, they are dealt out anew: of the rounds of the chip that the
// longest splits would take, the last is filled, and a split is the fewest blocks
// with which the requests' splits, one at least each, fit.  So ragged contexts keep
// the chip as full as equal ones, and a bound far above the contexts (a captured
// call's) costs little.  Against splits fixed by the bound: 8 requests x 4 x 128
// heads on half to all of 74,160 4-bit tokens 625 us, 799 before; 32 x 128 on half
// to all of 8,192 FP8 tokens 101 and 114; 32 x 16 heads 43 and 47; at its cost 0.6
// us.  Under a bound of 74,160, on half to all of 2,000 FP8 tokens: 64 x 128 heads
// 87 us, 168 with every place filled; 128 x 16 heads 53, 119 with fixed splits; 300
// x 128 heads on 500 201 and 631.  Place -> item, split; false past the last.
__device__ __forceinline__ bool place(const DecodeParams& p, int32_t pair, bool first, int32_t& item,
                                      int32_t& split, int64_t& per) {
  constexpr int kEach = kDealtReqs / 64;     // requests a lane, at most
  const int l = threadIdx.x & 63, slots = p.items * p.splits, each = (p.items + 63) / 64;
  int b[kEach];                              // blocks of request l * each + i, -1 past the last
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int r = l * each + i;
    b[i] = -1;
    if (i < each && r < p.items) {
      b[i] = (int)((min((int64_t)max(p.ctx_len[r], 0), (int64_t)p.max_keys) + kKeys - 1) / kKeys);
      sum += b[i];
    }
  }
  auto parts = [&](int blocks, int n) { return blocks < 0 ? 0 : max(1, (blocks + n - 1) / n); };
  auto mine = [&](int n) {                   // this lane's requests' splits of n blocks
    int x = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (i < each) x += parts(b[i], n);
    return x;
  };
  int hi = (int)(p.keys_per_split / kKeys);
  const int least = lane_of(wave_scan(mine(hi)), 63);
  const int use = min(slots, (least + p.round - 1) / p.round * p.round);
  if (pair >= use) return false;             // a loose bound's many, soonest
  // n blocks a split make at most all / n + items of them
  const int all = lane_of(wave_scan(sum), 63);
  int lo = max(1, (all + use - 1) / use);
  if (use > p.items) hi = min(hi, all / (use - p.items) + 1);
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (lane_of(wave_scan(mine(mid)), 63) <= use) hi = mid; else lo = mid + 1;
  }
  const int own = mine(lo), end = wave_scan(own), total = lane_of(end, 63);
  if (first && threadIdx.x < 64) {
    int at = end - own;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (b[i] < 0) continue;
      p.part_off[l * each + i] = at;
      at += parts(b[i], lo);
    }
    if (l == 0) p.part_off[p.items] = total;
  }
  if (pair >= total) return false;
  const int lane = __popcll(__ballot(end <= pair));
  int rest = pair - (lane > 0 ? lane_of(end, lane - 1) : 0);
  item = -1;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (i >= each || item >= 0) continue;
    const int n = parts(lane_of(b[i], lane), lo);
    if (rest < n) item = lane * each + i; else rest -= n;
  }
  split = rest;
  per = (int64_t)lo * kKeys;
  return true;
}

// Finds the workgroup's share and stages its row ids; false for a place without
// one.  Ends with a barrier.
template <bool PAGED, int ROWS>
__device__ __forceinline__ bool begin(const DecodeParams& p, Lists<ROWS>& s, Share& sh) {
  // workgroup -> (item, split, row tile): the row tiles of one (item, split)
  // are 8 workgroups apart, the XCD stride, so one's rows are in the other's L2
  const int64_t L = blockIdx.x;
  const int tile = (int)((L >> 3) % p.row_tiles);
  const int64_t pair = L / (8 * p.row_tiles) * 8 + (L & 7);
  if (pair >= (int64_t)p.items * p.splits) return false;
  int32_t split;
  int64_t per = p.keys_per_split;
  if (PAGED && p.part_off) {
    if (!place(p, (int32_t)pair, L == 0, sh.item, split, per)) return false;
    sh.part = pair;
  } else {
    sh.item = (int32_t)(pair % p.items);
    split = (int32_t)(pair / p.items);
    sh.part = (int64_t)sh.item * p.splits + split;
  }
  sh.row0 = tile * ROWS;
  sh.lo = split * per;
  const int tid = threadIdx.x, l = tid & 63;
  const int32_t rows = min(ROWS, p.rows - sh.row0);
  int64_t keys, unseen;                      // a query row sees unseen + its position of the keys
  if constexpr (PAGED) {
    const int64_t ctx = max(p.ctx_len[sh.item], 0);
    keys = min(ctx, (int64_t)p.max_keys);
    unseen = ctx - p.positions + 1;
  } else {
    keys = unseen = p.top_k;
  }
  auto seen = [&](int32_t row) {
    return (int)max((int64_t)0, min(per,
                                    min(keys, unseen + (sh.row0 + row) / p.heads) - sh.lo));
  };
  sh.n = seen(rows - 1);
  sh.edge = seen(0);
  for (int i = tid; i < ROWS; i += blockDim.x) s.mine[i] = seen(min(i, rows - 1));
  for (int k = tid; k < (sh.n + 63) / 64 * 64; k += blockDim.x) {
    int32_t id = -1;
    if (k < sh.n) {
      if constexpr (PAGED) {
        const int64_t t = sh.lo + k;
        const int32_t b = p.block_table[(int64_t)sh.item * p.max_pages + (t >> p.page_shift)];
        if (b >= 0 && b < p.pool_rows >> p.page_shift)
          id = (b << p.page_shift) | (int32_t)(t & ((1 << p.page_shift) - 1));
      } else {
        id = p.row_ids[(int64_t)sh.item * p.top_k + sh.lo + k];
        if (id >= p.pool_rows) id = -1;
      }
    }
    s.ids[k] = id;
    const uint64_t b = __ballot(id >= 0);
    if (l == 0) s.there[k >> 5] = (uint32_t)b;
    if (l == 32) s.there[k >> 5] = (uint32_t)(b >> 32);
  }
  __syncthreads();
  return true;
}

// What a key without a row reads.
__device__ __attribute__((aligned(16))) uint8_t zero_row[kFp8RowBytes];

template <bool FP4>
struct Row {
  static constexpr int kBytes = FP4 ? kFp4RowBytes : kFp8RowBytes;
  static constexpr int kPieces = kBytes / 16;
  static constexpr int kLatPieces = FP4 ? 16 : 32;
  static constexpr int kScales = FP4 ? 256 : 512;
  static constexpr int kRope = kScales + 16;
};

// A block's rows from the pool straight into LDS, 16 bytes a lane; wait_rows()
// and a barrier before they are read.
template <bool FP4, int T>
__device__ __forceinline__ void fetch_rows(const uint8_t* kv, const int32_t* ids, uint8_t* raw) {
  using R = Row<FP4>;
  const int tid = fresh_tid(), first = __builtin_amdgcn_readfirstlane(tid);
#pragma unroll
  for (int i = 0; i < (kKeys * R::kPieces + T - 1) / T; ++i) {
    const int q = tid + T * i;
    if (kKeys * R::kPieces % T != 0 && q >= kKeys * R::kPieces) continue;
    const int k = q / R::kPieces, id = ids[k];
    const uint8_t* row = id >= 0 ? kv + (int64_t)id * R::kBytes : zero_row;
    // the wave's lanes fill 64 consecutive pieces from the first lane's
    load_to_lds(row + 16 * (q - k * R::kPieces), raw + 16 * (first + T * i));
  }
}

// Rows from `from` on are seen by some query rows and masked for others, where
// a probability of 0 times a NaN or an infinity would be NaN: pieces that hold
// one become zeros and their row's id, no longer needed, kBad: its scores are
// NaN for the query rows that see it.  On the pieces that this thread loaded
// and waited for.
template <bool FP4, int T>
__device__ __forceinline__ void sanitize_rows(uint8_t* raw, int32_t* ids, int from) {
  using R = Row<FP4>;
  for (int q = threadIdx.x; q < kKeys * R::kPieces; q += T) {
    const int k = q / R::kPieces, pc = q - k * R::kPieces;
    if (k < from) continue;
    u32x4* at = reinterpret_cast<u32x4*>(raw + 16 * q);
    const u32x4 w = *at;
    bool nan = false;
    if (pc < R::kLatPieces) {
      if (!FP4) {
#pragma unroll
        for (int j = 0; j < 16; ++j) nan |= ((w[j / 4] >> (8 * (j % 4))) & 0x7fu) == 0x7fu;
      }
    } else if (pc == R::kLatPieces) {
      if (FP4) {
#pragma unroll
        for (int j = 0; j < 16; ++j) nan |= ((w[j / 4] >> (8 * (j % 4))) & 0xffu) == 0xffu;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) nan |= (w[j] & 0x7f800000u) == 0x7f800000u;
      }
    } else {
      nan = bad_bf16(w);
    }
    if (!nan) continue;
    *at = u32x4{0u, 0u, 0u, 0u};
    ids[k] = kBad;
  }
}

}  // namespace
}  // namespace hs
