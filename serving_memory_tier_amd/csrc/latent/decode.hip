// Latent attention in the absorbed form: the sparse decode over 4-bit rows and
// the dense decode through the block table (FP8 or 4-bit rows).
//
// For a query row q (576) and the latent rows c_j (512) with their rope parts:
//   s_j = scale <q, [c_j, rope_j]>,  out = sum_j softmax(s)_j c_j,
//   lse = log sum_j exp(s_j).
// Keys and values are one vector, so a block of rows is brought to LDS once
// and read twice: as it lies for the scores, transposed for the values.
//
// Work split.  An item (a token of the sparse form, a request of the paged
// one) has M query rows: its heads, for each of its positions.  A workgroup of
// 8 waves takes 128 of them and one range of the item's keys.  Four wave pairs
// take 32 rows each; a pair's waves take the two halves of the latent
// dimensions for both products, so a wave reads only its half of a block:
//   S^T (32 keys x 32 rows), 18 MFMAs 32x32x16 over 256 latent and 32 rope
//     dimensions; the halves' sums are exchanged through LDS;
//   the online softmax (a lane holds 16 keys of one row), in both waves alike;
//   O^T (256 dimensions x 32 rows) += V^T P^T, 16 MFMAs; the probabilities are
//     the B operand from registers, the values come from the row-major block
//     through the transposing LDS read (ds_read_b64_tr_b16).
// That keeps a wave's queries (72 registers) and output (128) within 256
// registers, two waves a SIMD, with 32 x 32 tiles: half the LDS bytes a FLOP of
// 16-row tiles.
//
// Blocks of 32 rows are converted to bfloat16 once as they enter LDS, exactly:
// E4M3 values as they are (their float32 scales, one per 128 values, multiply
// the partial scores and the probabilities), E2M1 values times their E8M0
// scale.  Two blocks are resident, the one after them is in registers.  Two
// barriers a block: after the partial scores (the other buffer is free, the
// scores are complete) and after the values (the next block is complete).
//
// Row strides in LDS: 1104 bytes (latent) and 144 (rope), 5 and 9 sixteen-byte
// units modulo the banks: 16 consecutive rows' fragments fall on distinct
// banks, and so do the transposing reads' 64-byte pieces, two deep.
//
// Rounding: scores, softmax and outputs in float32; the probabilities times
// the value scales are rounded to bfloat16 for the MFMAs (2^-8 half steps that
// average over the keys); key splits hand over their normalised outputs in
// half precision (2^-11), merged in float32; out is rounded to bfloat16.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "latent.h"

namespace hs {
namespace {

constexpr int kKeys = 32;                    // rows a block
constexpr int kLatent = 512;
constexpr int kDim = 576;
constexpr int kLatStride = 1072;             // bytes between latent rows in LDS
constexpr int kRopeStride = 144;
constexpr int kQuerySteps = 5;               // of a wave's 18 query fragments, in LDS (the rope's first)
constexpr int kQueryRegs = 18 - kQuerySteps;
constexpr int kSplitKeys = 2048;             // keys a split, at most: their row ids are in LDS
constexpr int32_t kBad = -2;                 // in place of a fetched row's id: see Fetch::store
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kStaleMax = 8.f;             // log2 of the largest unnormalised probability

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

struct Block {
  uint8_t lat[kKeys * kLatStride];
  uint8_t rope[kKeys * kRopeStride];
  float scale[4][kKeys];                     // FP8: the rows' scales, by latent tile
};

template <int NP>
struct Lds {
  Block blk[2];
  f32x4 xs[2 * NP][4][64];                   // a wave's partial scores
  bf16x8 qs[2 * NP][kQuerySteps][64];        // a wave's queries that are not in registers
  int32_t ids[kSplitKeys];                     // row ids, -1 where there is none
  int32_t mine[32 * NP];                     // keys of the split that a query row sees
  uint32_t there[kSplitKeys / 32];         // a block's keys that have one
};

// Within each 16 lanes, lane c receives element c % 4 of the 8-byte vectors at
// the addresses of lanes 4 j + c / 4, j = 0..3.
__device__ __forceinline__ u32x2 tr16_read(const uint8_t* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (lds_s16x4*)(const_cast<uint8_t*>(p))));
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

template <bool HI>
__device__ __forceinline__ uint32_t fp8_pair(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}

// The thread's number, opaque to the compiler: what it addresses with it is
// computed where it is used instead of held in registers over the loop.
__device__ __forceinline__ int fresh_tid() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// A block on its way from the pool to LDS: the latent pieces (16 bytes: 16
// E4M3 values, or the 32 E2M1 values of one scale) in whole rounds of the
// workgroup, then the rest of the rows (FP8: scales and rope, 9 pieces a row;
// 4-bit: rope, 8).
template <bool FP4, int T>
struct Fetch {
  static constexpr int kLat = FP4 ? 16 : 32;                   // latent pieces a row
  static constexpr int kRest = FP4 ? 8 : 9;
  static constexpr int kRow = FP4 ? kFp4RowBytes : kFp8RowBytes;
  static constexpr int kRestOffset = FP4 ? 272 : 512;
  static constexpr int kLatRounds = kKeys * kLat / T;
  static constexpr int kRestRounds = (kKeys * kRest + T - 1) / T;
  static_assert(kKeys * kLat % T == 0, "whole rounds");

  u32x4 lat[kLatRounds];
  u32x4 rest[kRestRounds];
  uint32_t scale[FP4 ? kLatRounds : 1];
  uint32_t there;                                              // bit a piece: its row is there

  __device__ __forceinline__ void load(const uint8_t* kv, const int32_t* ids) {
    const int tid = fresh_tid();
    int32_t id[kLatRounds + kRestRounds];
#pragma unroll
    for (int i = 0; i < kLatRounds; ++i) id[i] = ids[(tid + T * i) / kLat];
#pragma unroll
    for (int i = 0; i < kRestRounds; ++i) {
      const int q = tid + T * i;
      id[kLatRounds + i] = q < kKeys * kRest ? ids[q / kRest] : -1;
    }
    there = 0;
#pragma unroll
    for (int i = 0; i < kLatRounds; ++i) {
      // a key without a row reads row 0 and is stored as zeros
      const uint8_t* row = kv + (int64_t)max(id[i], 0) * kRow;
      const int pc = (tid + T * i) % kLat;
      lat[i] = *reinterpret_cast<const u32x4*>(row + 16 * pc);
      if constexpr (FP4) scale[i] = row[256 + pc];
      there |= (id[i] >= 0 ? 1u : 0u) << i;
    }
#pragma unroll
    for (int i = 0; i < kRestRounds; ++i) {
      const int q = tid + T * i;
      const uint8_t* row = kv + (int64_t)max(id[kLatRounds + i], 0) * kRow;
      if (q < kKeys * kRest)
        rest[i] = *reinterpret_cast<const u32x4*>(row + kRestOffset + 16 * (q % kRest));
      there |= (id[kLatRounds + i] >= 0 ? 1u : 0u) << (kLatRounds + i);
    }
  }

  // sanitize: rows from `from` on are seen by some query rows and masked for
  // others, where a probability of 0 times a NaN or an infinity would be NaN:
  // pieces that hold one are stored as zeros and their row's id, no longer
  // needed, becomes kBad: its scores are NaN for the query rows that see it.
  __device__ __forceinline__ void store(Block& b, int32_t* ids, bool sanitize, int from) {
    const int tid = fresh_tid();
#pragma unroll
    for (int i = 0; i < kLatRounds; ++i) {
      const int q = tid + T * i, k = q / kLat, pc = q % kLat;
      u32x4 w = (there >> i) & 1 ? lat[i] : u32x4{0u, 0u, 0u, 0u};
      uint8_t* dst = b.lat + k * kLatStride + pc * (FP4 ? 64 : 32);
      if constexpr (FP4) {
        uint32_t sb = (there >> i) & 1 ? scale[i] : 127u;
        if (sanitize && k >= from && sb == 255u) {
          ids[k] = kBad;
          w = u32x4{0u, 0u, 0u, 0u};
          sb = 127u;
        }
        const float s = __builtin_bit_cast(float, sb << 23);   // 255: infinity, whose product is NaN
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4 v = {
              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 0)),
              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 1)),
              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 2)),
              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 3))};
          *reinterpret_cast<u32x4*>(dst + 16 * j) = v;
        }
      } else {
        if (sanitize && k >= from) {
          bool nan = false;
#pragma unroll
          for (int j = 0; j < 16; ++j) nan |= ((w[j / 4] >> (8 * (j % 4))) & 0x7fu) == 0x7fu;
          if (nan) {
            ids[k] = kBad;
            w = u32x4{0u, 0u, 0u, 0u};
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<u32x4*>(dst + 16 * j) =
              u32x4{fp8_pair<false>(w[2 * j]), fp8_pair<true>(w[2 * j]),
                    fp8_pair<false>(w[2 * j + 1]), fp8_pair<true>(w[2 * j + 1])};
      }
    }
#pragma unroll
    for (int i = 0; i < kRestRounds; ++i) {
      const int q = tid + T * i;
      if (q >= kKeys * kRest) continue;
      const int k = q / kRest, pc = q % kRest;
      u32x4 w = (there >> (kLatRounds + i)) & 1 ? rest[i] : u32x4{0u, 0u, 0u, 0u};
      const bool scales = !FP4 && pc == 0;
      if (sanitize && k >= from) {
        bool nan = false;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          nan |= (w[j] & 0x7f800000u) == 0x7f800000u ||
                 (!scales && (w[j] & 0x7f80u) == 0x7f80u);
        if (nan) {
          ids[k] = kBad;
          w = u32x4{0u, 0u, 0u, 0u};
        }
      }
      if (scales) {
#pragma unroll
        for (int t = 0; t < 4; ++t) b.scale[t][k] = __builtin_bit_cast(float, w[t]);
      } else {
        *reinterpret_cast<u32x4*>(b.rope + k * kRopeStride + 16 * (FP4 ? pc : pc - 1)) = w;
      }
    }
  }
};

template <bool FP4, bool PAGED, int NP>
__global__ void __launch_bounds__(128 * NP) decode_kernel(DecodeParams p) {
  constexpr int T = 128 * NP;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
  Lds<NP>& s = *reinterpret_cast<Lds<NP>*>(lds_raw);
  // workgroup -> (item, split, row tile): the row tiles of one (item, split)
  // are 8 workgroups apart, the XCD stride, so one's rows are in the other's L2
  const int64_t L = blockIdx.x;
  const int tile = (int)((L >> 3) % p.row_tiles);
  const int64_t pair = L / (8 * p.row_tiles) * 8 + (L & 7);
  if (pair >= (int64_t)p.items * p.splits) return;     // the grid's rounding: the whole workgroup
  const int32_t item = (int32_t)(pair % p.items), split = (int32_t)(pair / p.items);
  const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, hi = l >> 5, half = w / NP;
  const int32_t row0 = tile * 32 * NP;
  // the keys of this workgroup: [lo, lo + n); the first query row sees the
  // fewest of them, `edge`
  const int64_t lo = (int64_t)split * p.keys_per_split;
  int n, edge;
  {
    const int64_t most = p.keys_per_split;
    const int32_t rows = min(32 * NP, p.rows - row0);
    int64_t keys, unseen;                      // a query row sees unseen + its position of the keys
    if constexpr (PAGED) {
      const int64_t ctx = max(p.ctx_len[item], 0);
      keys = min(ctx, (int64_t)p.max_keys);
      unseen = ctx - p.positions + 1;
    } else {
      keys = unseen = p.top_k;
    }
    auto seen = [&](int32_t row) {
      return (int)max((int64_t)0, min(most, min(keys, unseen + (row0 + row) / p.heads) - lo));
    };
    n = seen(rows - 1);
    edge = seen(0);
    if (tid < 32 * NP) s.mine[tid] = seen(min(tid, rows - 1));
  }

  // a lane past the last row takes row 0's queries; it writes nothing
  auto query_row = [&](int t) {
    const int32_t m = row0 + (t >> 6) % NP * 32 + (t & 31);
    return m < p.rows ? m : -1;
  };
  bf16x8 qb[kQueryRegs];
  {
    const uint16_t* q = p.q + ((int64_t)item * p.rows + max(query_row(tid), 0)) * kDim;
#pragma unroll
    for (int ks = 0; ks < 18; ++ks) {
      const int at = ks < 16 ? half * 256 + ks * 16 + 8 * hi
                             : kLatent + half * 32 + (ks - 16) * 16 + 8 * hi;
      const bf16x8 v = *reinterpret_cast<const bf16x8*>(q + at);
      if (ks < kQueryRegs)
        qb[ks] = v;
      else
        s.qs[w][ks - kQueryRegs][l] = v;
    }
  }
  f32x16 o[8];                                 // O^T: dimensions 256 half + 32 dt + row, by column
#pragma unroll
  for (int dt = 0; dt < 8; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[dt][i] = 0.f;
  float m_run = -INFINITY, l_run = 0.f;        // l_run: this lane's keys only
  const float qk_scale = p.scale * kLog2e;

  const int blocks = (n + kKeys - 1) / kKeys;
  for (int k = tid; k < (n + 63) / 64 * 64; k += T) {
    int32_t id = -1;
    if (k < n) {
      if constexpr (PAGED) {
        const int64_t t = lo + k;
        const int32_t b = p.block_table[(int64_t)item * p.max_pages + (t >> p.page_shift)];
        if (b >= 0 && b < p.pool_rows >> p.page_shift)
          id = (b << p.page_shift) | (int32_t)(t & ((1 << p.page_shift) - 1));
      } else {
        id = p.row_ids[(int64_t)item * p.top_k + lo + k];
        if (id >= p.pool_rows) id = -1;
      }
    }
    s.ids[k] = id;
    const uint64_t b = __ballot(id >= 0);
    if (l == 0) s.there[k >> 5] = (uint32_t)b;
    if (l == 32) s.there[k >> 5] = (uint32_t)(b >> 32);
  }
  __syncthreads();
  Fetch<FP4, T> f;
  if (blocks > 0) {
    f.load(p.kv, s.ids);
    f.store(s.blk[0], s.ids, PAGED && kKeys > edge, edge);
    if (blocks > 1) f.load(p.kv, s.ids + kKeys);
  }
  __syncthreads();
  for (int bi = 0; bi < blocks; ++bi) {
    Block& cb = s.blk[bi & 1];
    const int tid = fresh_tid(), w = tid >> 6, l = tid & 63;
    const int col = l & 31, hi = l >> 5, duo = w % NP, half = w / NP;
    auto query = [&](int ks) { return ks < kQueryRegs ? qb[ks] : s.qs[w][ks - kQueryRegs][l]; };
    // ---- this half's share of S^T: row (key) col of A is row `col` of the block
    f32x16 sc;
#pragma unroll
    for (int i = 0; i < 16; ++i) sc[i] = 0.f;
    const uint8_t* krow = cb.lat + col * kLatStride + half * 512 + 16 * hi;
    const uint8_t* rrow = cb.rope + col * kRopeStride + half * 64 + 16 * hi;
    if constexpr (FP4) {
#pragma unroll
      for (int ks = 0; ks < 16; ++ks)
        sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            *reinterpret_cast<const bf16x8*>(krow + 32 * ks), query(ks), sc, 0, 0, 0);
    } else {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x16 acc;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              *reinterpret_cast<const bf16x8*>(krow + 32 * (8 * t + ks)), query(8 * t + ks),
              acc, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 k4 = *reinterpret_cast<const f32x4*>(&cb.scale[2 * half + t][8 * i + 4 * hi]);
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[4 * i + j] += k4[j] * acc[4 * i + j];
        }
      }
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          *reinterpret_cast<const bf16x8*>(rrow + 32 * ks), query(16 + ks), sc, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s.xs[w][i][l] = f32x4{sc[4 * i], sc[4 * i + 1], sc[4 * i + 2], sc[4 * i + 3]};
    __syncthreads();
    // ---- the other half's share (a sum of two: alike in both waves)
    const int other = w < NP ? w + NP : w - NP;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 v = s.xs[other][i][l];
#pragma unroll
      for (int j = 0; j < 4; ++j) sc[4 * i + j] = (sc[4 * i + j] + v[j]) * qk_scale;
    }
    if (bi + 1 < blocks) {
      f.store(s.blk[(bi + 1) & 1], s.ids + (bi + 1) * kKeys, PAGED && (bi + 2) * kKeys > edge, edge - (bi + 1) * kKeys);
      if (bi + 2 < blocks) f.load(p.kv, s.ids + (bi + 2) * kKeys);
    }
    // ---- masks: keys without a row, and keys this row does not see
    const uint32_t there = s.there[bi];
    if (there != 0xffffffffu || (bi + 1) * kKeys > edge) {
      const int left = s.mine[duo * 32 + col] - bi * kKeys;
      uint32_t seen = left >= kKeys ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
      seen = (seen & there) >> (4 * hi);
#pragma unroll
      for (int i = 0; i < 16; ++i) {           // key 8 (i / 4) + 4 hi + i % 4
        if (PAGED && s.ids[bi * kKeys + 4 * hi + 8 * (i / 4) + i % 4] == kBad)
          sc[i] = __builtin_nanf("");
        if (!(seen & (1u << (8 * (i / 4) + i % 4)))) sc[i] = -INFINITY;
      }
    }
    // ---- online softmax; the maximum is renewed only when it grows by 2^8
    float mb = sc[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) mb = fmaxf(mb, sc[i]);
    mb = fmaxf(mb, __shfl_xor(mb, 32));
    const bool grow = mb > m_run + kStaleMax;
    const float m_new = grow ? mb : m_run;
    const float alpha = grow ? __builtin_amdgcn_exp2f(m_run - m_new) : 1.f;
    const float base = m_new == -INFINITY ? 0.f : m_new;    // nothing seen yet: exp2(-inf) = 0
    float pr[16], ls = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      pr[i] = __builtin_amdgcn_exp2f(sc[i] - base);
      ls += pr[i];
    }
    l_run = l_run * alpha + ls;
    m_run = m_new;
    if (__any(grow)) {
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) o[dt] *= alpha;
    }
    // ---- O^T += V^T P^T.  Step ks covers keys 16 ks + 4 hi + {0..3, 8..11},
    // the ones this lane holds; lane c of a 16-lane group supplies row c / 4
    // and 4 dimensions of each transposing read
    const uint8_t* vrow = cb.lat + (4 * hi + ((l & 15) >> 2)) * kLatStride + half * 512 +
                          32 * ((l >> 4) & 1) + 8 * (l & 3);
#pragma unroll
    for (int t = 0; t < (FP4 ? 1 : 2); ++t) {
      bf16x8 pb[2];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x[4];
          if constexpr (FP4) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = pr[8 * ks + 4 * i + j];
          } else {
            const f32x4 k4 = *reinterpret_cast<const f32x4*>(
                &cb.scale[2 * half + t][16 * ks + 8 * i + 4 * hi]);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = pr[8 * ks + 4 * i + j] * k4[j];
          }
          v[2 * i] = bf16_pair(x[0], x[1]);
          v[2 * i + 1] = bf16_pair(x[2], x[3]);
        }
        pb[ks] = __builtin_bit_cast(bf16x8, v);
      }
#pragma unroll
      for (int d = 0; d < (FP4 ? 8 : 4); ++d) {
        const int dt = 4 * t + d;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const u32x2 a = tr16_read(vrow + 16 * ks * kLatStride + 64 * dt);
          const u32x2 b = tr16_read(vrow + (16 * ks + 8) * kLatStride + 64 * dt);
          o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]}), pb[ks], o[dt], 0, 0, 0);
        }
      }
    }
    __syncthreads();
  }

  const int32_t m = query_row(fresh_tid());
  if (m < 0) return;
  l_run += __shfl_xor(l_run, 32);              // the same query row
  const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
  const int d0 = half * 256 + 4 * hi;
  const int64_t mrow = (int64_t)item * p.rows + m;
  if (p.splits == 1) {
    uint16_t* out = p.out + mrow * kLatent + d0;
#pragma unroll
    for (int dt = 0; dt < 8; ++dt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<u32x2*>(out + 32 * dt + 8 * i) =
            u32x2{bf16_pair(o[dt][4 * i] * inv, o[dt][4 * i + 1] * inv),
                  bf16_pair(o[dt][4 * i + 2] * inv, o[dt][4 * i + 3] * inv)};
    if (half == 0 && hi == 0)
      p.lse[mrow] = l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) / kLog2e;
    return;
  }
  const int64_t ps = ((int64_t)item * p.splits + split) * p.rows + m;
  if (half == 0 && hi == 0) {
    p.part_ml[2 * ps] = m_run;
    p.part_ml[2 * ps + 1] = l_run;
  }
  if (l_run == 0.f) return;                    // the merge does not read it
  uint16_t* po = p.part_o + ps * kLatent + d0;
#pragma unroll
  for (int dt = 0; dt < 8; ++dt)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<f16x4*>(po + 32 * dt + 8 * i) =
          f16x4{(_Float16)(o[dt][4 * i] * inv), (_Float16)(o[dt][4 * i + 1] * inv),
                (_Float16)(o[dt][4 * i + 2] * inv), (_Float16)(o[dt][4 * i + 3] * inv)};
}

// Merges the key splits of a query row, one wave a row: with w_s = 2^(m_s - M)
// l_s, out = sum_s w_s out_s / sum_s w_s.  Lane s reads the maximum and sum of
// splits s, s + 64, ...; then each lane sums 8 dimensions over the splits.
__global__ void __launch_bounds__(256) decode_merge_kernel(DecodeParams p) {
  const int l = threadIdx.x & 63;
  const int64_t mrow = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (mrow >= (int64_t)p.items * p.rows) return;
  const int64_t item = mrow / p.rows, m = mrow - item * p.rows;
  const int64_t ps0 = item * p.splits * p.rows + m;
  float M = -INFINITY;
  for (int sp = l; sp < p.splits; sp += 64) {
    const int64_t ps = ps0 + (int64_t)sp * p.rows;
    if (p.part_ml[2 * ps + 1] != 0.f) M = fmaxf(M, p.part_ml[2 * ps]);
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) M = fmaxf(M, __shfl_xor(M, d));
  float sum = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < p.splits; s0 += 64) {
    float wgt = 0.f;
    if (s0 + l < p.splits) {
      const int64_t ps = ps0 + (int64_t)(s0 + l) * p.rows;
      const float ls = p.part_ml[2 * ps + 1];
      if (ls != 0.f) wgt = exp2f(p.part_ml[2 * ps] - M) * ls;     // NaN stays NaN
    }
    for (int j = 0; j < min(64, p.splits - s0); ++j) {
      const float x = __shfl(wgt, j);
      if (x == 0.f) continue;                  // nothing seen there: not written
      sum += x;
      const f16x8 h = *reinterpret_cast<const f16x8*>(
          p.part_o + (ps0 + (int64_t)(s0 + j) * p.rows) * kLatent + 8 * l);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += x * (float)h[i];
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<u32x4*>(p.out + mrow * kLatent + 8 * l) =
      u32x4{bf16_pair(acc[0] * inv, acc[1] * inv), bf16_pair(acc[2] * inv, acc[3] * inv),
            bf16_pair(acc[4] * inv, acc[5] * inv), bf16_pair(acc[6] * inv, acc[7] * inv)};
  if (l == 0) p.lse[mrow] = sum == 0.f ? -INFINITY : (M + log2f(sum)) / kLog2e;
}

int64_t grid_of(const DecodeParams& p) {
  return ((int64_t)p.items * p.splits + 7) / 8 * 8 * p.row_tiles;
}

template <bool FP4, bool PAGED, int NP>
hipError_t launch(const DecodeParams& p, hipStream_t stream) {
  auto fn = decode_kernel<FP4, PAGED, NP>;
  static std::atomic<uint64_t> raised{0};
  hipError_t e = allow_full_lds(reinterpret_cast<const void*>(fn), raised);
  if (e != hipSuccess) return e;
  return launch_kernel(fn, dim3((uint32_t)grid_of(p)), dim3(128 * NP), sizeof(Lds<NP>), stream, p);
}

}  // namespace

// The workgroups of a launch to aim for: one round of the chip's 256 units.
constexpr int64_t kDecodeGroups = 256;
constexpr int64_t kDecodeMaxSplits = 64;   // below the splits that kSplitKeys asks for

size_t plan_decode(DecodeParams& p, int64_t keys) {
  p.row_tiles = (p.rows + kDecodeRows - 1) / kDecodeRows;
  const int64_t base = (int64_t)p.items * p.row_tiles;
  const int64_t blocks = (keys + kKeys - 1) / kKeys;
  int64_t splits = base > 0 ? (kDecodeGroups + base - 1) / base : 1;
  splits = min(splits, kDecodeMaxSplits);
  splits = max(splits, (blocks * kKeys + kSplitKeys - 1) / kSplitKeys);
  splits = max((int64_t)1, min(splits, blocks));
  const int64_t per = (blocks + splits - 1) / splits;          // blocks a split, at most kSplitKeys
  p.splits = (int32_t)(per > 0 ? (blocks + per - 1) / per : 1);
  p.keys_per_split = per * kKeys;
  // per (item, split, row): 512 half-precision values and two floats
  return p.splits > 1 ? (size_t)p.items * p.splits * p.rows * (kLatent * 2 + 2 * 4) : 0;
}

bool decode_fits(const DecodeParams& p) {
  return grid_of(p) <= INT32_MAX && (int64_t)p.items * p.rows <= 4 * (int64_t)INT32_MAX;
}

hipError_t launch_decode(DecodeParams p, bool fp4, bool paged, void* workspace,
                         hipStream_t stream) {
  if (p.items == 0 || p.rows == 0) return hipSuccess;
  if (p.splits > 1) {
    p.part_o = static_cast<uint16_t*>(workspace);
    p.part_ml = reinterpret_cast<float*>(p.part_o + (size_t)p.items * p.splits * p.rows * kLatent);
  }
  hipError_t e = paged ? (fp4 ? launch<true, true, 4>(p, stream) : hipErrorNotSupported)
                       : launch<true, false, 4>(p, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t rows = (int64_t)p.items * p.rows;
  return launch_kernel(decode_merge_kernel, dim3((uint32_t)((rows + 3) / 4)), dim3(256), 0, stream,
                       p);
}

}  // namespace hs
