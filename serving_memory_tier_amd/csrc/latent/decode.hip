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
// 8 waves takes 128 of them and one range of the item's keys, in blocks of 32.
// Four wave pairs take 32 rows each; a pair's waves take the two halves of the
// latent dimensions for both products, so a wave reads only its half of a block:
//   S^T (32 keys x 32 rows), 18 MFMAs 32x32x16 over 256 latent and 32 rope
//     dimensions; the halves' sums are exchanged through LDS;
//   the online softmax (a lane holds 16 keys of one row), in both waves alike;
//   O^T (256 dimensions x 32 rows) += V^T P^T, 16 MFMAs; the probabilities are
//     the B operand from registers, the values come from the row-major block
//     through the transposing LDS reads.
// That keeps a wave's queries (72 registers) and output (128) within 256
// registers, two waves a SIMD, with 32 x 32 tiles: half the LDS bytes a FLOP of
// 16-row tiles.
//
// The two row formats meet LDS in different ways:
//   4-bit rows are converted to bfloat16 once as they enter LDS (E2M1 values
//     times their E8M0 scale, exactly): a scale spans 32 dimensions of one
//     key, and the transposed operand pairs keys, so scaling there would take
//     a multiplication and a packing of every probability for each 32
//     dimensions.  Two blocks are resident, the one after is in registers; two
//     barriers a block.  The two waves of a SIMD run half a block apart, so that
//     one's scores meet the other's softmax and value products.
//   FP8 rows go from the pool into LDS as they are, with no register between
//     (three blocks resident, two barriers a block), and are converted at each
//     use, exactly; their float32 scales, one per 128 values, copied beside the
//     rows once a block, multiply the partial scores and the probabilities.
//     Converted copies beside the scales' accumulators would not fit the
//     registers.
//
// Bound: a block's LDS reads (18 KB of keys and 16 KB of values a wave, the
// transposing reads at half the rate of the others), its MFMAs and the steps
// between them, which two waves a SIMD overlap in part (no LDS bank conflict is
// left over 4-bit rows).  512 tokens x 128 heads x 2,048 4-bit rows: 338 us, 846
// TFLOP/s, 39 % of what a loop of these MFMAs alone reaches (2,170); a large matrix
// product of the library reaches 1,210 to 1,330.  32 x 128 x 2,048 takes 45 us, of
// it the merge 8 (eight splits, 34 MB written and read); 8 requests x 4 positions x
// 128 heads on half to all of 74,160 4-bit tokens 625 us (810 TFLOP/s); 32 x 128
// heads on half to all of 8,192 FP8 tokens 100 us (551 TFLOP/s: the conversions at
// use).
//
// Rounding: scores, softmax and outputs in float32; the probabilities times
// the FP8 scales are rounded to bfloat16 for the MFMAs (half steps of 2^-8 that
// average over the keys); key splits hand over their normalised outputs in half
// precision, brought into its range by a power of two for each wave's dimensions
// of a row (half steps of 2^-11, against bfloat16's 2^-8 at the same bytes),
// merged in float32; out is rounded to bfloat16.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "decode_parts.h"

namespace hs {
namespace {

// Waves w and w + 4 share a SIMD; they take different pairs, in opposite phases.
__device__ __forceinline__ int duo_of(int w) { return (w & 1) + 2 * (w >> 2); }
__device__ __forceinline__ int half_of(int w) { return (w >> 1) & 1; }

// Thread t's query row of the item, or -1 past the last.
template <int NP>
__device__ __forceinline__ int32_t query_row(const DecodeParams& p, const Share& sh, int t) {
  const int32_t m = sh.row0 + duo_of(t >> 6) * 32 + (t & 31);
  return m < p.rows ? m : -1;
}

// Masks a block's scores (keys without a row, and keys the row does not see)
// where it has any to mask.
template <bool PAGED, int NP>
__device__ __forceinline__ void mask(const Lists<32 * NP>& s, const Share& sh, int bi, int row, int hi,
                                     f32x16& sc) {
  const uint32_t there = s.there[bi];
  if (there == 0xffffffffu && (bi + 1) * kKeys <= sh.edge) return;
  const int left = s.mine[row] - bi * kKeys;
  uint32_t seen = left >= kKeys ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
  seen = (seen & there) >> (4 * hi);
#pragma unroll
  for (int i = 0; i < 16; ++i) {             // key 8 (i / 4) + 4 hi + i % 4
    if (PAGED && s.ids[bi * kKeys + 4 * hi + 8 * (i / 4) + i % 4] == kBad)
      sc[i] = __builtin_nanf("");
    if (!(seen & (1u << (8 * (i / 4) + i % 4)))) sc[i] = -INFINITY;
  }
}

// One block of the online softmax: scores, which qk_scale > 0 brings to log2
// units, to probabilities.  The maximum is renewed, and the output rescaled, only
// when it grows by 2^8.
__device__ __forceinline__ void softmax(f32x16& sc, float qk_scale, float& m_run, float& l_run,
                                        f32x16 (&o)[8]) {
  float mb = sc[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) mb = fmaxf(mb, sc[i]);
  mb = max_halves(mb) * qk_scale;
  const bool grow = mb > m_run + kStaleMax;
  const float m_new = grow ? mb : m_run;
  const float alpha = grow ? __builtin_amdgcn_exp2f(m_run - m_new) : 1.f;
  const float base = m_new == -INFINITY ? 0.f : m_new;    // nothing seen yet: exp2(-inf) = 0
  float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    sc[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], qk_scale, -base));
    ls[i % 4] += sc[i];
  }
  l_run = l_run * alpha + ((ls[0] + ls[1]) + (ls[2] + ls[3]));
  m_run = m_new;
  if (__any(grow)) {
#pragma unroll
    for (int dt = 0; dt < 8; ++dt) o[dt] *= alpha;
  }
}

// Writes this lane's 128 output values and, once a row, its log sum: the
// result, or the split's share of it.
template <int NP>
__device__ __forceinline__ void finish(const DecodeParams& p, const Share& sh, const f32x16 (&o)[8],
                                       float m_run, float l_run) {
  const int tid = fresh_tid(), hi = (tid & 63) >> 5, half = half_of(tid >> 6);
  const int32_t m = query_row<NP>(p, sh, tid);
  if (m < 0) return;
  l_run += __shfl_xor(l_run, 32);              // the same query row
  const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
  const int d0 = half * 256 + 4 * hi;
  const int64_t mrow = (int64_t)sh.item * p.rows + m;
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
  const int64_t ps = sh.part * p.rows + m;
  float* ml = p.part_ml + kPartFloats * ps;
  if (half == 0 && hi == 0) *reinterpret_cast<f32x2*>(ml) = f32x2{m_run, l_run};
  if (l_run == 0.f) return;                    // the merge does not read it
  float most = 0.f;
#pragma unroll
  for (int dt = 0; dt < 8; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(o[dt][i]));
  const int e = half_exponent(max_halves(most) * inv);
  if (hi == 0) *reinterpret_cast<f32x2*>(ml + 2 + 2 * half) = f32x2{ldexpf(1.f, e), ldexpf(1.f, e)};
  const float f = ldexpf(inv, -e);
  uint16_t* po = p.part_o + ps * kLatent + d0;
#pragma unroll
  for (int dt = 0; dt < 8; ++dt)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<f16x4*>(po + 32 * dt + 8 * i) = half4(
          o[dt][4 * i] * f, o[dt][4 * i + 1] * f, o[dt][4 * i + 2] * f, o[dt][4 * i + 3] * f);
}

// ------------------------------------------------------------ 4-bit rows

// Converted rows in LDS: 1072 bytes apart (3 sixteen-byte units modulo the 16 of
// the banks), rope rows 144 (9).  Within a row, unit u = 4 pc + j (piece pc's j-th,
// 8 values) lies at unit 16 j + (pc ^ 4 j): the 16 lanes that write one j of a
// row's pieces, the 16 rows of a key fragment and the 4 rows x 4 units of a
// transposing read each fall on distinct banks.
constexpr int kLatStride = 1072;
constexpr int kRopeStride = 144;
// Of a wave's 18 query fragments, the last are kept in LDS.
constexpr int kQuerySteps = 5;
constexpr int kQueryRegs = 18 - kQuerySteps;

struct Block4 {
  uint8_t lat[kKeys * kLatStride];
  uint8_t rope[kKeys * kRopeStride];
};

template <int NP>
struct Lds4 {
  Block4 blk[2];
  f32x4 xs[2 * NP][4][64];                   // a wave's partial scores
  bf16x8 qs[2 * NP][kQuerySteps][64];
  Lists<32 * NP> lists;
};

// A block on its way from the pool to LDS: 16 latent pieces a row (16 bytes,
// the 32 values of one scale), then its 8 rope pieces.
template <int T>
struct Fetch4 {
  static constexpr int kLat = 16, kRope = 8;
  static constexpr int kLatRounds = kKeys * kLat / T;
  static constexpr int kRopeRounds = (kKeys * kRope + T - 1) / T;
  static_assert(kKeys * kLat % T == 0, "whole rounds");

  u32x4 lat[kLatRounds];
  u32x4 rope[kRopeRounds];
  uint32_t scale[kLatRounds];
  uint32_t there;                                              // bit a piece: its row is there
  int32_t id[kLatRounds + kRopeRounds];

  __device__ __forceinline__ void load_ids(const int32_t* ids) {
    const int tid = fresh_tid();
#pragma unroll
    for (int i = 0; i < kLatRounds; ++i) id[i] = ids[(tid + T * i) / kLat];
#pragma unroll
    for (int i = 0; i < kRopeRounds; ++i) {
      const int q = tid + T * i;
      id[kLatRounds + i] = ids[q < kKeys * kRope ? q / kRope : 0];
    }
  }

  __device__ __forceinline__ void load(const uint8_t* kv) {
    const int tid = fresh_tid();
    there = 0;
#pragma unroll
    for (int i = 0; i < kLatRounds; ++i) {
      // a key without a row reads row 0 and is stored as zeros
      const uint8_t* row = kv + (int64_t)max(id[i], 0) * kFp4RowBytes;
      const int pc = (tid + T * i) % kLat;
      lat[i] = *reinterpret_cast<const u32x4*>(row + 16 * pc);
      // the word that holds the scale: a byte's load would be widened, and waited
      // for, right here
      scale[i] = *reinterpret_cast<const uint32_t*>(row + 256 + (pc & ~3));
      there |= (id[i] >= 0 ? 1u : 0u) << i;
    }
#pragma unroll
    for (int i = 0; i < kRopeRounds; ++i) {
      const int q = tid + T * i;
      const uint8_t* row = kv + (int64_t)max(id[kLatRounds + i], 0) * kFp4RowBytes;
      if (q < kKeys * kRope)
        rope[i] = *reinterpret_cast<const u32x4*>(row + 272 + 16 * (q % kRope));
      there |= (id[kLatRounds + i] >= 0 ? 1u : 0u) << (kLatRounds + i);
    }
  }

  // sanitize: rows from `from` on are seen by some query rows and masked for
  // others, where a probability of 0 times a NaN or an infinity would be NaN:
  // pieces that hold one are stored as zeros and their row's id, no longer
  // needed, becomes kBad: its scores are NaN for the query rows that see it.
  __device__ __forceinline__ void store(Block4& b, int32_t* ids, bool sanitize, int from) {
    const int tid = fresh_tid();
#pragma unroll
    for (int i = 0; i < kLatRounds; ++i) {
      const int q = tid + T * i, k = q / kLat, pc = q % kLat;
      u32x4 w = (there >> i) & 1 ? lat[i] : u32x4{0u, 0u, 0u, 0u};
      uint32_t sb = (there >> i) & 1 ? (scale[i] >> (8 * (pc & 3))) & 255u : 127u;
      if (sanitize && k >= from && bad_fp4(w, sb)) {
        ids[k] = kBad;
        w = u32x4{0u, 0u, 0u, 0u};
        sb = 127u;
      }
      const float s = __builtin_bit_cast(float, sb << 23);     // 255: infinity, whose product is NaN
      uint8_t* dst = b.lat + k * kLatStride;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<u32x4*>(dst + 256 * j + ((16 * pc) ^ (64 * j))) = u32x4{
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 0)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 1)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 2)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 3))};
    }
#pragma unroll
    for (int i = 0; i < kRopeRounds; ++i) {
      const int q = tid + T * i;
      if (q >= kKeys * kRope) continue;
      const int k = q / kRope;
      u32x4 w = (there >> (kLatRounds + i)) & 1 ? rope[i] : u32x4{0u, 0u, 0u, 0u};
      if (sanitize && k >= from && bad_bf16(w)) {
        ids[k] = kBad;
        w = u32x4{0u, 0u, 0u, 0u};
      }
      *reinterpret_cast<u32x4*>(b.rope + k * kRopeStride + 16 * (q % kRope)) = w;
    }
  }
};

template <bool PAGED, int NP>
__global__ void __launch_bounds__(128 * NP) decode_fp4_kernel(DecodeParams p) {
  constexpr int T = 128 * NP;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
  Lds4<NP>& s = *reinterpret_cast<Lds4<NP>*>(lds_raw);
  Share sh;
  if (!begin<PAGED, 32 * NP>(p, s.lists, sh)) return;       // the whole workgroup
  int32_t* ids = s.lists.ids;
  const int blocks = (sh.n + kKeys - 1) / kKeys;
  Fetch4<T> f;
  if (blocks > 0) {                            // before the queries: waited for first
    f.load_ids(ids);
    f.load(p.kv);
  }
  bf16x8 qb[kQueryRegs];
  {
    // a lane past the last row takes row 0's queries; it writes nothing
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, hi = l >> 5, half = half_of(w);
    const uint16_t* q =
        p.q + ((int64_t)sh.item * p.rows + max(query_row<NP>(p, sh, tid), 0)) * kDim;
#pragma unroll
    for (int ks = 0; ks < 18; ++ks) {
      const int at = ks < 16 ? half * 256 + ks * 16 + 8 * hi
                             : kLatent + half * 32 + (ks - 16) * 16 + 8 * hi;
      const bf16x8 v = signed_query(q + at, p.scale);
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
  const float qk_scale = positive_scale(p.scale);
  if (blocks > 0) {
    f.store(s.blk[0], ids, PAGED && kKeys > sh.edge, sh.edge);
    if (blocks > 1) {
      f.load_ids(ids + kKeys);
      f.load(p.kv);
    }
  }
  __syncthreads();
  const bool late = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) != 0;
  if (late) __syncthreads();
  for (int bi = 0; bi < blocks; ++bi) {
    const Block4& cb = s.blk[bi & 1];
    const int tid = fresh_tid(), w = tid >> 6, l = tid & 63;
    const int col = l & 31, hi = l >> 5, duo = duo_of(w), half = half_of(w);
    auto query = [&](int ks) { return ks < kQueryRegs ? qb[ks] : s.qs[w][ks - kQueryRegs][l]; };
    auto next = [&]() {
      if (bi + 1 < blocks) {
        if (bi + 2 < blocks) f.load_ids(ids + (bi + 2) * kKeys);
        f.store(s.blk[(bi + 1) & 1], ids + (bi + 1) * kKeys, PAGED && (bi + 2) * kKeys > sh.edge,
                sh.edge - (bi + 1) * kKeys);
        if (bi + 2 < blocks) f.load(p.kv);
      }
    };
    if (late) next();
    // ---- this half's share of S^T: row (key) col of A is row `col` of the block
    f32x16 sc;
#pragma unroll
    for (int i = 0; i < 16; ++i) sc[i] = 0.f;
    // step ks reads unit 32 half + 2 ks + hi: ks = 8 a + 2 t + b
    const uint8_t* krow = cb.lat + col * kLatStride + 256 * hi;
    const uint8_t* rrow = cb.rope + col * kRopeStride + half * 64 + 16 * hi;
    const uint8_t* kbase[2][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) kbase[a][b] = krow + 512 * b + 128 * (half ^ b) + 64 * (hi ^ a);
    constexpr int kC = 4;                      // steps whose fragments are read under the last ones' products
    bf16x8 kf[2][kC];
    auto read_keys = [&](int c) {
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        const int ks = kC * c + j;
        if (ks < 18)
          kf[c & 1][j] = *reinterpret_cast<const bf16x8*>(ks < 16 ? kbase[ks >> 3][ks & 1] + 16 * ((ks >> 1) & 3)
                                                         : rrow + 32 * (ks - 16));
      }
    };
    read_keys(0);
#pragma unroll
    for (int c = 0; c < (18 + kC - 1) / kC; ++c) {
      if (kC * (c + 1) < 18) read_keys(c + 1);
#pragma unroll
      for (int j = 0; j < kC; ++j)
        if (kC * c + j < 18)
          sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[c & 1][j], query(kC * c + j), sc, 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s.xs[w][i][l] = f32x4{sc[4 * i], sc[4 * i + 1], sc[4 * i + 2], sc[4 * i + 3]};
    __syncthreads();
    // ---- the other half's share (a sum of two: alike in both waves)
    const int other = w ^ 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 v = s.xs[other][i][l];
#pragma unroll
      for (int j = 0; j < 4; ++j) sc[4 * i + j] += v[j];
    }
    if (!late) next();
    mask<PAGED, NP>(s.lists, sh, bi, duo * 32 + col, hi, sc);
    softmax(sc, qk_scale, m_run, l_run, o);
    // ---- O^T += V^T P^T.  Step ks covers keys 16 ks + 4 hi + {0..3, 8..11},
    // the ones this lane holds; lane c of a 16-lane group supplies row c / 4
    // and 4 dimensions of each transposing read
    // of row c / 4, unit 32 half + 4 dt + j
    const int j = (l >> 3 & 2) + (l >> 1 & 1);
    const uint8_t* vrow = cb.lat + (4 * hi + ((l & 15) >> 2)) * kLatStride + 256 * j +
                          128 * (half ^ (j >> 1)) + 8 * (l & 1);
    const uint8_t* vbase[2] = {vrow + 64 * (j & 1), vrow + 64 * (~j & 1)};
    bf16x8 pb[2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      pb[ks] = __builtin_bit_cast(
          bf16x8, u32x4{bf16_pair(sc[8 * ks], sc[8 * ks + 1]), bf16_pair(sc[8 * ks + 2], sc[8 * ks + 3]),
                        bf16_pair(sc[8 * ks + 4], sc[8 * ks + 5]),
                        bf16_pair(sc[8 * ks + 6], sc[8 * ks + 7])});
    u32x2 vf[3][4];
    auto read_values = [&](int dt) {
#pragma unroll
      for (int j = 0; j < 4; ++j) vf[dt % 3][j] = tr16_read(vbase[dt >> 2] + 8 * j * kLatStride + 16 * (dt & 3));
    };
    read_values(0);
    read_values(1);
#pragma unroll
    for (int dt = 0; dt < 8; ++dt) {
      if (dt + 2 < 8) read_values(dt + 2);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const u32x2 a = vf[dt % 3][2 * ks], b = vf[dt % 3][2 * ks + 1];
        o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]}), pb[ks], o[dt], 0, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
  }
  if (!late) __syncthreads();
  finish<NP>(p, sh, o, m_run, l_run);
}

// -------------------------------------------------------------- FP8 rows

constexpr int kScales = 512, kRope = 528;    // offsets in a row

constexpr int kQuerySteps8 = 7;              // query fragments in LDS, the last

// Rows lie in LDS as in the pool, 656 bytes apart (an odd number of 16-byte
// units: rows' fragments on distinct banks).
template <int NP>
struct Lds8 {
  uint8_t blk[3][kKeys * kFp8RowBytes];
  float scale[2][4][kKeys];                  // the rows' scales, by latent tile
  f32x4 xs[2 * NP][4][64];                   // a wave's partial scores
  bf16x8 qs[2 * NP][kQuerySteps8][64];
  Lists<32 * NP> lists;
};

// The scales of a block in LDS, by latent tile, so that a lane's keys' are read
// four at a time.
__device__ __forceinline__ void copy_scales(const uint8_t* blk, float (&scale)[4][kKeys]) {
  const int tid = fresh_tid();
  if (tid < 4 * kKeys)
    scale[tid & 3][tid >> 2] =
        *reinterpret_cast<const float*>(blk + (tid >> 2) * kFp8RowBytes + kScales + 4 * (tid & 3));
}

template <int NP>
__global__ void __launch_bounds__(128 * NP) decode_fp8_kernel(DecodeParams p) {
  constexpr int T = 128 * NP;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
  Lds8<NP>& s = *reinterpret_cast<Lds8<NP>*>(lds_raw);
  Share sh;
  if (!begin<true, 32 * NP>(p, s.lists, sh)) return;        // the whole workgroup
  const int blocks = (sh.n + kKeys - 1) / kKeys;
  if (blocks > 0) fetch_rows<false, T>(p.kv, s.lists.ids, s.blk[0]);
  if (blocks > 1) fetch_rows<false, T>(p.kv, s.lists.ids + kKeys, s.blk[1]);
  bf16x8 qb[18 - kQuerySteps8];
  {
    // in the order in which the keys are read: 16 values a lane for two steps
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, hi = l >> 5, half = half_of(w);
    const uint16_t* q =
        p.q + ((int64_t)sh.item * p.rows + max(query_row<NP>(p, sh, tid), 0)) * kDim;
#pragma unroll
    for (int ks = 0; ks < 18; ++ks) {
      const int at = ks < 16 ? half * 256 + (ks / 2) * 32 + 16 * hi + 8 * (ks % 2)
                             : kLatent + half * 32 + (ks - 16) * 16 + 8 * hi;
      const bf16x8 v = signed_query(q + at, p.scale);
      if (ks < 18 - kQuerySteps8)
        qb[ks] = v;
      else
        s.qs[w][ks - 18 + kQuerySteps8][l] = v;
    }
  }
  f32x16 o[8];                                 // O^T: dimensions 256 half + 32 dt + row, by column
#pragma unroll
  for (int dt = 0; dt < 8; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[dt][i] = 0.f;
  float m_run = -INFINITY, l_run = 0.f;        // l_run: this lane's keys only
  const float qk_scale = positive_scale(p.scale);
  wait_rows();
  if (blocks > 0 && kKeys > sh.edge) sanitize_rows<false, T>(s.blk[0], s.lists.ids, sh.edge);
  __syncthreads();
  copy_scales(s.blk[0], s.scale[0]);
  __syncthreads();
  int cur = 0;
  for (int bi = 0; bi < blocks; ++bi) {
    uint8_t* cb = s.blk[cur];
    const int tid = fresh_tid(), w = tid >> 6, l = tid & 63;
    const int col = l & 31, hi = l >> 5, duo = duo_of(w), half = half_of(w);
    auto query = [&](int ks) {
      return ks < 18 - kQuerySteps8 ? qb[ks] : s.qs[w][ks - 18 + kQuerySteps8][l];
    };
    // ---- this half's share of S^T: row (key) col of A is row `col` of the block
    const uint8_t* krow = cb + col * kFp8RowBytes + half * 256 + 16 * hi;
    const uint8_t* rrow = cb + col * kFp8RowBytes + kRope + half * 64 + 16 * hi;
    f32x16 sc;
#pragma unroll
    for (int i = 0; i < 16; ++i) sc[i] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          *reinterpret_cast<const bf16x8*>(rrow + 32 * ks), query(16 + ks), sc, 0, 0, 0);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      f32x16 acc;
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const u32x4 k = *reinterpret_cast<const u32x4*>(krow + 128 * t + 32 * c);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fp8x8(k[0], k[1]), query(8 * t + 2 * c), acc,
                                                      0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fp8x8(k[2], k[3]), query(8 * t + 2 * c + 1), acc,
                                                      0, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 k4 =
            *reinterpret_cast<const f32x4*>(&s.scale[bi & 1][2 * half + t][8 * i + 4 * hi]);
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[4 * i + j] += acc[4 * i + j] * k4[j];
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s.xs[w][i][l] = f32x4{sc[4 * i], sc[4 * i + 1], sc[4 * i + 2], sc[4 * i + 3]};
    // past this barrier: the scores and the next block's rows are complete, and
    // every wave is done with the block before, whose buffer is filled next
    wait_rows();
    const int nxt = cur == 2 ? 0 : cur + 1;
    if (bi + 1 < blocks && (bi + 2) * kKeys > sh.edge)
      sanitize_rows<false, T>(s.blk[nxt], s.lists.ids + (bi + 1) * kKeys,
                              sh.edge - (bi + 1) * kKeys);
    lds_barrier();
    copy_scales(s.blk[nxt], s.scale[(bi + 1) & 1]);    // (past the last block: for nobody)
    if (bi + 2 < blocks)
      fetch_rows<false, T>(p.kv, s.lists.ids + (bi + 2) * kKeys, s.blk[nxt == 2 ? 0 : nxt + 1]);
    // ---- the other half's share (a sum of two: alike in both waves)
    const int other = w ^ 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 v = s.xs[other][i][l];
#pragma unroll
      for (int j = 0; j < 4; ++j) sc[4 * i + j] += v[j];
    }
    mask<true, NP>(s.lists, sh, bi, duo * 32 + col, hi, sc);
    softmax(sc, qk_scale, m_run, l_run, o);
    // ---- O^T += V^T P'^T, P' = p * scale of the latent tile.  Step ks covers
    // keys 16 ks + 4 hi + {0..3, 8..11}, the ones this lane holds; lane c of a
    // 16-lane group supplies row c / 2 of those and 8 dimensions
    const int j8 = (l & 15) >> 1;
    const uint8_t* vrow = cb + (4 * hi + j8 + (j8 < 4 ? 0 : 4)) * kFp8RowBytes + half * 256 +
                          16 * ((l >> 4) & 1) + 8 * (l & 1);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      bf16x8 pb[2];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const f32x4 k4 = *reinterpret_cast<const f32x4*>(
              &s.scale[bi & 1][2 * half + t][16 * ks + 8 * i + 4 * hi]);
          const int e = 8 * ks + 4 * i;
          v[2 * i] = bf16_pair(sc[e] * k4[0], sc[e + 1] * k4[1]);
          v[2 * i + 1] = bf16_pair(sc[e + 2] * k4[2], sc[e + 3] * k4[3]);
        }
        pb[ks] = __builtin_bit_cast(bf16x8, v);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const u32x2 a = tr8_read(vrow + 16 * ks * kFp8RowBytes + 32 * (4 * t + d));
          o[4 * t + d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fp8x8(a[0], a[1]), pb[ks],
                                                                 o[4 * t + d], 0, 0, 0);
        }
    }
    cur = nxt;
    lds_barrier();                             // the scores are read
  }
  finish<NP>(p, sh, o, m_run, l_run);
}

// Merges the key splits of a query row, one wave a row: with w_s = 2^(m_s - M)
// l_s, out = sum_s w_s out_s / sum_s w_s.  Lane s reads the maximum and sum of
// splits s, s + 64, ...; then each lane sums 8 dimensions over the splits.
__global__ void __launch_bounds__(256) decode_merge_kernel(DecodeParams p) {
  const int l = threadIdx.x & 63;
  const int64_t mrow = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (mrow >= (int64_t)p.items * p.rows) return;
  const int64_t item = mrow / p.rows, m = mrow - item * p.rows;
  const int64_t part0 = p.part_off ? p.part_off[item] : item * p.splits;
  const int32_t splits = p.part_off ? p.part_off[item + 1] - (int32_t)part0 : p.splits;
  const int64_t ps0 = part0 * p.rows + m;
  // eight splits' outputs at a time, the first ones beside the sums; one that saw
  // nothing was not written, and has no weight
  f16x8 h[8];
  float scale[8];
  auto read = [&](int sp) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t ps = ps0 + (int64_t)min(sp + j, splits - 1) * p.rows;
      h[j] = *reinterpret_cast<const f16x8*>(p.part_o + ps * kLatent + 8 * l);
      scale[j] = p.part_ml[kPartFloats * ps + 2 + (l >> 4)];
    }
  };
  auto sums = [&](int sp) {
    return sp < splits
               ? *reinterpret_cast<const f32x2*>(p.part_ml + kPartFloats * (ps0 + (int64_t)sp * p.rows))
               : f32x2{-INFINITY, 0.f};
  };
  f32x2 ml = sums(l);
  read(0);
  float M = ml[1] != 0.f ? ml[0] : -INFINITY;
  for (int sp = l + 64; sp < splits; sp += 64) {
    const f32x2 v = sums(sp);
    if (v[1] != 0.f) M = fmaxf(M, v[0]);
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) M = fmaxf(M, __shfl_xor(M, d));
  float sum = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < splits; s0 += 64) {
    if (s0 > 0) ml = sums(s0 + l);
    const float wgt = ml[1] != 0.f ? exp2f(ml[0] - M) * ml[1] : 0.f;    // NaN stays NaN
    for (int j0 = 0; j0 < min(64, splits - s0); j0 += 8) {
      if (s0 + j0 > 0) read(s0 + j0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = __shfl(wgt, j0 + j);   // 0 past the last split
        if (x == 0.f) continue;
        sum += x;
        const float y = x * scale[j];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += y * (float)h[j][i];
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<u32x4*>(p.out + mrow * kLatent + 8 * l) =
      u32x4{bf16_pair(acc[0] * inv, acc[1] * inv), bf16_pair(acc[2] * inv, acc[3] * inv),
            bf16_pair(acc[4] * inv, acc[5] * inv), bf16_pair(acc[6] * inv, acc[7] * inv)};
  if (l == 0) p.lse[mrow] = sum == 0.f ? -INFINITY : (M + log2f(sum)) / kLog2e;
}

hipError_t launch(void (*fn)(DecodeParams), int threads, size_t lds, std::atomic<uint64_t>& raised,
                  const DecodeParams& p, hipStream_t stream) {
  hipError_t e = allow_full_lds(reinterpret_cast<const void*>(fn), raised);
  if (e != hipSuccess) return e;
  return launch_kernel(fn, dim3((uint32_t)decode_grid(p)), dim3((uint32_t)threads), lds, stream, p);
}

template <int NP>
hipError_t launch_wide(const DecodeParams& p, bool fp4, bool paged, hipStream_t stream) {
  constexpr int T = 128 * NP;
  static std::atomic<uint64_t> raised[3];
  return !paged ? launch(decode_fp4_kernel<false, NP>, T, sizeof(Lds4<NP>), raised[0], p, stream)
         : fp4  ? launch(decode_fp4_kernel<true, NP>, T, sizeof(Lds4<NP>), raised[1], p, stream)
                : launch(decode_fp8_kernel<NP>, T, sizeof(Lds8<NP>), raised[2], p, stream);
}

}  // namespace

// In block times (about 2 us): a workgroup's start and end, a merge's launch, the
// splits that it takes one over, and the rows whose partial outputs (2 KB written
// and read) take one.
constexpr int kStartBlocks = 4, kMergeBlocks = 2, kMergeSplits = 12;
constexpr double kMergeRows = 7000;

int64_t decode_grid(const DecodeParams& p) {
  return ((int64_t)p.items * p.splits + 7) / 8 * 8 * p.row_tiles;
}

// Whether the kernel deals out the splits by the contexts: where they are of more
// than the least, one block.
static bool dealt_out(const DecodeParams& p, bool paged) {
  return paged && p.items <= kDealtReqs && p.splits > 1 && p.keys_per_split > kKeys;
}

size_t plan_decode(DecodeParams& p, int64_t keys, bool paged) {
  // The least tile that holds the rows: up to 32 the narrow kernel, up to 64 this
  // file's with two wave pairs.  Measured with tiles of 16, 32, 64 and 128 rows, 32
  // requests on up to 8,192 FP8 tokens (splits by the bound): 16 heads 47, 59, 99 and 107 us; 32 heads
  // 79, 63, 101 and 111; 64 heads 146, 109, 106 and 117; 128 heads 277, 202, 193
  // and 125
  p.tile_rows = p.rows <= 16 ? 16 : p.rows <= 32 ? 32 : p.rows <= 64 ? 64 : 128;
  p.row_tiles = (p.rows + p.tile_rows - 1) / p.tile_rows;
  // Key splits: the fewest block times over the rounds of the chip that the
  // workgroups take (256 units, two narrow workgroups each), with some block
  // times a workgroup for its start and end, and a merge's launch and traffic.
  // 5 tokens x 16 heads x 1,000 rows with 8, 16 and 32 splits: 13.8, 11.8, 12.7 us;
  // 32 x 128 x 2,048 with 2, 4 and 8: 95, 63, 50; one request of 16 heads on 8,192
  // tokens with 16, 32 and 64: 35, 24, 21
  const int64_t base = (int64_t)p.items * p.row_tiles;
  const int64_t blocks = (keys + kKeys - 1) / kKeys;
  const int64_t slots = p.tile_rows >= 64 ? 256 : 512;
  p.round = (int32_t)(slots / p.row_tiles > 0 ? slots / p.row_tiles : 1);
  const int64_t least = (blocks * kKeys + kDecodeSplitKeys - 1) / kDecodeSplitKeys;
  int64_t best = 1;
  double best_t = 1e300;
  const int64_t full = base * least / slots;   // rounds that the fewest splits fill
  // as few as may be; as many as fill up to four rounds more; a half and a quarter
  // of the blocks
  for (int r = 0; r <= 6; ++r) {
    int64_t n = r > 4 ? blocks / (2 * (r - 4)) : r > 0 && base > 0 ? (full + r) * slots / base : 1;
    n = n < least ? least : n;
    n = n > blocks ? blocks : n;
    if (n < 1) n = 1;
    const int64_t per = (blocks + n - 1) / n;
    if (per > 0) n = (blocks + per - 1) / per;
    const double t = (double)((base * n + slots - 1) / slots) * (per + kStartBlocks) +
                     (n > 1 ? kMergeBlocks + (double)n / kMergeSplits +
                                  (double)p.items * p.rows * n / kMergeRows
                            : 0.0);
    if (t < best_t) {
      best_t = t;
      best = n;
    }
  }
  const int64_t per = (blocks + best - 1) / best;              // blocks a split
  p.splits = (int32_t)(per > 0 ? (blocks + per - 1) / per : 1);
  p.keys_per_split = per * kKeys;
  if (p.splits == 1) return 0;
  return (size_t)p.items * p.splits * p.rows * (kLatent * 2 + kPartFloats * 4) +
         (dealt_out(p, paged) ? (p.items + 1) * sizeof(int32_t) : 0);
}

bool decode_fits(const DecodeParams& p) {
  return grid_fits(decode_grid(p), 512) && grid_fits(((int64_t)p.items * p.rows + 3) / 4, 256);
}

hipError_t launch_decode(DecodeParams p, bool fp4, bool paged, void* workspace,
                         hipStream_t stream) {
  if (p.items == 0 || p.rows == 0) return hipSuccess;
  if (p.splits > 1) {
    p.part_o = static_cast<uint16_t*>(workspace);
    const size_t parts = (size_t)p.items * p.splits * p.rows;
    p.part_ml = reinterpret_cast<float*>(p.part_o + parts * kLatent);
    if (dealt_out(p, paged))
      p.part_off = reinterpret_cast<int32_t*>(p.part_ml + parts * kPartFloats);
  }
  const hipError_t e = p.tile_rows == 128  ? launch_wide<4>(p, fp4, paged, stream)
                       : p.tile_rows == 64 ? launch_wide<2>(p, fp4, paged, stream)
                                           : launch_decode_narrow(p, fp4, paged, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t rows = (int64_t)p.items * p.rows;
  return launch_kernel(decode_merge_kernel, dim3((uint32_t)((rows + 3) / 4)), dim3(256), 0, stream,
                       p);
}

}  // namespace hs
