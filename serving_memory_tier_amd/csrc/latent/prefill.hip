// Latent attention in the expanded form, for a chunk of new tokens against the
// cached context: keys and values of every head from the latent rows,
//   k_j = [W^K_h c_j, rope_j] (128 + 64),  v_j = W^V_h c_j (128),
// then causal attention of 192-wide queries.  For n new tokens the absorbed
// form costs 2 * 1088 FLOPs a (query, key, head), this one 2 * 320 and, once a
// key and head, 2 * 512 * 256: it wins from some 350 new tokens on.
//
// Launches: the rows, brought out of the paged pool as bfloat16 [token][512] and
// [token][64] (with the offsets of the requests' tokens); the expansion, a matrix
// product to [head][token][128 + 128]; the attention; and a merge where it
// splits the keys.
//
// Rounding: latent values are exact in bfloat16 where a row's scales are powers
// of two (as hs_mla_append writes them), rounded once otherwise; products and
// sums in float32; the expanded keys and values, the probabilities and the
// output are rounded to bfloat16, as a model that stores them would; key splits'
// normalised outputs to half precision, brought into its range by a power of two
// a row.
//
// Bound: the matrix cores, less what feeds them.  One request's 2,048 new tokens
// on 8,192, 128 heads, FP8 rows: 1,525 us, 969 TFLOP/s, where a large matrix
// product of the library reaches 1,210 to 1,330 (rows 7 us; expansion 341, of it
// 537 MB written; attention 1,215 to 1,300, 925 TFLOP/s, 43 % of a loop of MFMAs
// alone).  Four requests of up to 753 on 4,849, 64 heads, 4-bit rows: 740 us.
// Three of up to 130 on 500, 16 heads: 33.5 us, three dependent launches.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "latent.h"
#include "parts.h"

namespace hs {
namespace {

constexpr int kNope = 128, kRopeDim = 64, kVal = 128;
constexpr int kQ = kNope + kRopeDim;         // 192
constexpr int kHeadRow = kNope + kVal;       // 256 values a (head, token)
constexpr int kPartFloats = 3;               // a split's, a row: maximum, sum, the values' scale

// ------------------------------------------------------------- offsets

// off[r]: the first workspace row of request r's tokens (its context, cut to
// the table and to what num_kv leaves); tile_off[r]: its first query tile.  Up to
// 64 requests, the rows' kernel finds them itself (a wave's lanes a request each)
// and writes them for the launches behind it; more have a launch of their own.
constexpr int kInlineReqs = 64;

__device__ __forceinline__ int64_t context(const PrefillParams& p, int32_t r) {
  return min((int64_t)max(p.ctx_len[r], 0), (int64_t)p.max_pages << p.page_shift);
}

__device__ __forceinline__ int64_t query_tiles(const PrefillParams& p, int32_t r) {
  return (query_count(p, r) + p.tile_rows - 1) / p.tile_rows;
}

__device__ __forceinline__ int64_t wave_sums(int64_t n) {      // of this lane and those before
  const int l = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t a = __shfl_up(n, d);
    if (l >= d) n += a;
  }
  return n;
}

__global__ void __launch_bounds__(1024) prefill_plan_kernel(PrefillParams p) {
  __shared__ int64_t sums[2][1024];
  __shared__ int64_t base[2];
  const int tid = threadIdx.x;
  if (tid < 2) base[tid] = 0;
  for (int32_t r0 = 0; r0 < p.num_reqs; r0 += 1024) {
    const int32_t r = r0 + tid;
    int64_t n = 0, tiles = 0;
    if (r < p.num_reqs) {
      n = context(p, r);
      tiles = query_tiles(p, r);
    }
    sums[0][tid] = n;
    sums[1][tid] = tiles;
    __syncthreads();
    for (int d = 1; d < 1024; d *= 2) {
      const int64_t a = tid >= d ? sums[0][tid - d] : 0, b = tid >= d ? sums[1][tid - d] : 0;
      __syncthreads();
      sums[0][tid] += a;
      sums[1][tid] += b;
      __syncthreads();
    }
    if (r < p.num_reqs) {
      p.off[r + 1] = (int32_t)min((int64_t)p.num_kv, base[0] + sums[0][tid]);
      p.tile_off[r + 1] = (int32_t)min((int64_t)p.max_tiles, base[1] + sums[1][tid]);
    }
    __syncthreads();
    if (tid < 2) base[tid] += sums[tid][1023];
    __syncthreads();
  }
  if (tid == 0) p.off[0] = p.tile_off[0] = 0;
}

// The last r with off[r] <= i, off ascending from 0 over n requests.
__device__ __forceinline__ int32_t find(const int32_t* off, int32_t n, int32_t i) {
  int32_t lo = 0, hi = n - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) / 2;
    if (off[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// ---------------------------------------------------------------- rows

// One wave a token: its row's latent values and rope values as bfloat16.  A
// token without a row, or whose row holds a NaN or an infinity, gets zeros and
// a flag (1: none, 2: not finite): a value that some queries must not see
// cannot reach them through a product with a probability of 0.
template <bool FP4>
__global__ void __launch_bounds__(256) prefill_rows_kernel(PrefillParams p) {
  const int l = threadIdx.x & 63;
  const int32_t i = (int32_t)(blockIdx.x * 4 + (threadIdx.x >> 6));
  int32_t r, t;
  if (p.num_reqs <= kInlineReqs) {
    const int64_t end = min((int64_t)p.num_kv, wave_sums(l < p.num_reqs ? context(p, l) : 0));
    if (blockIdx.x == 0 && threadIdx.x < 64) {
      const int64_t tiles = min((int64_t)p.max_tiles,
                                wave_sums(l < p.num_reqs ? query_tiles(p, l) : 0));
      if (l < p.num_reqs) {
        p.off[l + 1] = (int32_t)end;
        p.tile_off[l + 1] = (int32_t)tiles;
      }
      if (l == 0) p.off[0] = p.tile_off[0] = 0;
    }
    const uint64_t past = __ballot(l < p.num_reqs && end > i);
    if (past == 0) return;
    r = __ffsll((unsigned long long)past) - 1;
    t = i - (r == 0 ? 0 : (int32_t)__shfl((int)end, r - 1));
  } else {
    if (i >= p.off[p.num_reqs]) return;
    r = find(p.off, p.num_reqs, i);
    t = i - p.off[r];
  }
  const int32_t b = p.block_table[(int64_t)r * p.max_pages + (t >> p.page_shift)];
  const bool there = b >= 0 && b < p.pool_rows >> p.page_shift;
  u32x4 v = {0u, 0u, 0u, 0u}, rope = {0u, 0u, 0u, 0u};
  bool bad = false;
  if (there) {
    const int32_t id = (b << p.page_shift) | (t & ((1 << p.page_shift) - 1));
    if constexpr (FP4) {
      const uint8_t* row = p.kv + (int64_t)id * kFp4RowBytes;
      const uint32_t w = *reinterpret_cast<const uint32_t*>(row + 4 * l);
      const uint32_t sb = row[256 + l / 4];
      const float s = __builtin_bit_cast(float, sb << 23);
      bad = sb == 255u;
      v = u32x4{
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
      if (l < 8) rope = *reinterpret_cast<const u32x4*>(row + 272 + 16 * l);
    } else {
      const uint8_t* row = p.kv + (int64_t)id * kFp8RowBytes;
      const u32x2 w = *reinterpret_cast<const u32x2*>(row + 8 * l);
      const float s = *reinterpret_cast<const float*>(row + 512 + 4 * (l / 16));
      const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[0], false);
      const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[0], true);
      const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[1], false);
      const f32x2 e = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[1], true);
      v = u32x4{bf16_pair(a[0] * s, a[1] * s), bf16_pair(c[0] * s, c[1] * s),
                bf16_pair(d[0] * s, d[1] * s), bf16_pair(e[0] * s, e[1] * s)};
      if (l < 8) rope = *reinterpret_cast<const u32x4*>(row + 528 + 16 * l);
    }
    bad |= bad_bf16(v) || bad_bf16(rope);
    bad = __any(bad);
  }
  if (!there || bad) v = rope = u32x4{0u, 0u, 0u, 0u};
  *reinterpret_cast<u32x4*>(p.lat + (int64_t)i * 512 + 8 * l) = v;
  if (l < 8) *reinterpret_cast<u32x4*>(p.rope + (int64_t)i * kRopeDim + 8 * l) = rope;
  if (l == 0) p.flags[i] = !there ? 1 : bad ? 2 : 0;
}

// ----------------------------------------------------------- expansion

// [token][512] x [head][256][512]^T -> [head][token][256], a workgroup of 2 MW
// waves a tile of 64 MW tokens x one head's 256 dimensions, a wave 64 x 128 of
// it; the contraction in 8 chunks of 64.  Chunks go straight into LDS, one
// computed and one on its way, one barrier a chunk; 16-byte pieces of a row are
// exchanged by bits 1 to 3 of its number, which puts 16 rows' fragments on
// distinct banks.  The grid runs over heads first: an XCD sees every eighth head,
// whose weights (256 KB) stay in its L2 over the tokens' tiles.
constexpr int kGemmN = 256, kGemmK = 64;

template <int MW>
struct GemmLds {
  union {
    struct {
      uint8_t a[64 * MW * 2 * kGemmK];
      uint8_t w[kGemmN * 2 * kGemmK];
    } chunk[2];
    uint16_t out[64 * MW][kGemmN + 8];
  };
};

__device__ __forceinline__ int gemm_slot(int row, int piece) {
  return row * 128 + 16 * (piece ^ ((row >> 1) & 7));
}

// 16-byte pieces of ROWS rows of 64 values, from src rows row_bytes apart.
template <int ROWS, int T>
__device__ __forceinline__ void gemm_fetch(const uint8_t* src, int64_t row_bytes, int32_t last,
                                           uint8_t* dst) {
  const int tid = threadIdx.x, first = __builtin_amdgcn_readfirstlane(tid);
#pragma unroll
  for (int i = 0; i < ROWS * 8 / T; ++i) {
    const int q = tid + T * i, row = q >> 3;
    const int piece = (q & 7) ^ ((row >> 1) & 7);
    load_to_lds(src + (int64_t)min(row, last) * row_bytes + 16 * piece, dst + 16 * (first + T * i));
  }
}

template <int MW>
__global__ void __launch_bounds__(128 * MW, 2) prefill_expand_kernel(PrefillParams p) {
  constexpr int T = 128 * MW, kGemmM = 64 * MW;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
  GemmLds<MW>& s = *reinterpret_cast<GemmLds<MW>*>(lds_raw);
  const int head = blockIdx.x;
  const int32_t m0 = (int32_t)blockIdx.y * kGemmM;
  const int32_t total = p.off[p.num_reqs];
  if (m0 >= total) return;
  const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, col = l & 31, hi = l >> 5;
  const int wm = (w % MW) * 64, wn = (w / MW) * 128;
  const uint8_t* a = reinterpret_cast<const uint8_t*>(p.lat + (int64_t)m0 * 512);
  const uint8_t* b = reinterpret_cast<const uint8_t*>(p.w + (int64_t)head * kGemmN * 512);
  const int32_t last = min(kGemmM, total - m0) - 1;
  auto fetch = [&](int c) {
    gemm_fetch<kGemmM, T>(a + c * 128, 1024, last, s.chunk[c & 1].a);
    gemm_fetch<kGemmN, T>(b + c * 128, 1024, kGemmN - 1, s.chunk[c & 1].w);
  };
  f32x16 acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.f;
  fetch(0);
#pragma unroll 2
  for (int c = 0; c < 512 / kGemmK; ++c) {
    wait_rows();
    lds_barrier();                             // chunk c is complete, chunk c - 1 left
    if (c + 1 < 512 / kGemmK) fetch(c + 1);
    const uint8_t* ca = s.chunk[c & 1].a;
    const uint8_t* cw = s.chunk[c & 1].w;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      bf16x8 fa[2], fb[4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        fa[i] = *reinterpret_cast<const bf16x8*>(ca + gemm_slot(wm + 32 * i + col, 2 * ks + hi));
#pragma unroll
      for (int j = 0; j < 4; ++j)
        fb[j] = *reinterpret_cast<const bf16x8*>(cw + gemm_slot(wn + 32 * j + col, 2 * ks + hi));
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
  }
  // (W A^T): column = token, rows = dimensions 4 hi + 8 i + 0..3; through LDS so
  // that the stores are whole rows
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<u32x2*>(&s.out[wm + 32 * i + col][wn + 32 * j + 8 * k + 4 * hi]) =
            u32x2{bf16_pair(acc[i][j][4 * k], acc[i][j][4 * k + 1]),
                  bf16_pair(acc[i][j][4 * k + 2], acc[i][j][4 * k + 3])};
  __syncthreads();
  uint16_t* out = p.heads_kv + ((int64_t)head * p.num_kv + m0) * kHeadRow;
  for (int q = tid; q < kGemmM * 32; q += T) {
    const int row = q >> 5, pc = q & 31;
    if (row <= last)
      *reinterpret_cast<u32x4*>(out + (int64_t)row * kHeadRow + 8 * pc) =
          *reinterpret_cast<const u32x4*>(&s.out[row][8 * pc]);
  }
}

// ----------------------------------------------------------- attention

// A workgroup of NW waves takes 32 NW queries of one request and head, a wave
// 32, and one of `splits` shares of the keys that they see (more than one where
// the tiles and heads alone leave the chip idle); keys in tiles of 64, two resident
// in LDS, the next on its way while one is computed; one barrier a tile.  S^T (64
// keys x 32 queries) is 24 MFMAs 32x32x16 a wave, O^T (128 x 32) += V^T P^T 16; the
// probabilities are the B operand from registers, V^T comes through the transposing
// LDS read.
// The grid runs over heads first (an XCD sees every eighth head's keys), and
// the last tiles, which see the most keys, come first.
constexpr int kTile = 64;

struct TileLds {
  uint8_t nope[kTile * 256];                 // 16-byte piece c of row r at place c ^ (r & 15)
  uint8_t rope[kTile * 128];                 // at c ^ (r / 2 & 7)
  uint8_t val[kTile * 256];                  // at c ^ (r & 3) * 4
};

template <int NW>
__device__ __forceinline__ void fetch_tile(const PrefillParams& p, const uint8_t* hkv,
                                           const uint8_t* rope, int32_t k0, int32_t n, TileLds& s) {
  constexpr int T = 64 * NW;
  const int tid = threadIdx.x, first = __builtin_amdgcn_readfirstlane(tid);
  // keys past the request's last one read the last: masked, and finite
#pragma unroll
  for (int i = 0; i < kTile * 16 / T; ++i) {
    const int q = tid + T * i, row = q >> 4, c = q & 15;
    const uint8_t* src = hkv + (int64_t)min(k0 + row, n - 1) * (kHeadRow * 2);
    load_to_lds(src + 16 * (c ^ (row & 15)), s.nope + 16 * (first + T * i));
    load_to_lds(src + 256 + 16 * (c ^ ((row & 3) * 4)), s.val + 16 * (first + T * i));
  }
#pragma unroll
  for (int i = 0; i < kTile * 8 / T; ++i) {
    const int q = tid + T * i, row = q >> 3, c = q & 7;
    load_to_lds(rope + (int64_t)min(k0 + row, n - 1) * 128 + 16 * (c ^ ((row >> 1) & 7)),
                s.rope + 16 * (first + T * i));
  }
}

template <int NW>
__global__ void __launch_bounds__(64 * NW, 2) prefill_attend_kernel(PrefillParams p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
  TileLds* s = reinterpret_cast<TileLds*>(lds_raw);
  const int head = blockIdx.x;
  const int32_t tiles_all = p.tile_off[p.num_reqs];
  const int32_t split = (int32_t)(blockIdx.y % p.splits);
  const int32_t ti = tiles_all - 1 - (int32_t)(blockIdx.y / p.splits);
  if (ti < 0) return;
  const int32_t r = find(p.tile_off, p.num_reqs, ti);
  const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, col = l & 31, hi = l >> 5;
  const int32_t nq = query_count(p, r);
  const int32_t q0 = (ti - p.tile_off[r]) * (32 * NW);          // first query of the tile
  const int32_t n = p.off[r + 1] - p.off[r];                    // tokens at hand
  const int32_t unseen = max(p.ctx_len[r], 0) - nq;             // query i sees i + 1 + unseen
  auto sees = [&](int32_t i) { return max(0, min(n, unseen + i + 1)); };
  const int32_t wq = q0 + 32 * w;                               // this wave's first query
  const int32_t limit = sees(min(wq + col, nq - 1));
  const int32_t keys = sees(min(q0 + 32 * NW, nq) - 1);         // of the workgroup
  const int32_t mine = wq < nq ? sees(min(wq + 32, nq) - 1) : 0;  // of the wave
  const int32_t least = wq < nq ? sees(wq) : 0;
  const int64_t qrow = p.query_start(r) + min(wq + col, nq - 1);

  bf16x8 qb[12];
  {
    const uint16_t* q = p.q + (qrow * p.heads + head) * kQ;
#pragma unroll
    for (int ks = 0; ks < 12; ++ks)
      qb[ks] = signed_query(q + 16 * ks + 8 * hi, p.scale);
  }
  f32x16 o[4];
#pragma unroll
  for (int dt = 0; dt < 4; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[dt][i] = 0.f;
  float m_run = -INFINITY, l_run = 0.f;
  const float qk_scale = positive_scale(p.scale);
  const int64_t at = p.off[r];
  const uint8_t* hkv =
      reinterpret_cast<const uint8_t*>(p.heads_kv + ((int64_t)head * p.num_kv + at) * kHeadRow);
  const uint8_t* rope = reinterpret_cast<const uint8_t*>(p.rope + at * kRopeDim);
  const uint8_t* flags = p.flags + at;
  // this split's tiles: [lo, count)
  const int32_t all = (keys + kTile - 1) / kTile, per = (all + p.splits - 1) / p.splits;
  const int32_t lo = min(all, split * per), count = min(all, lo + per);
  auto flag_of = [&](int32_t k) { return k < n ? flags[k] : (uint8_t)1; };
  uint8_t next_flag = 1;
  if (count > lo) {
    next_flag = flag_of(lo * kTile + l);
    fetch_tile<NW>(p, hkv, rope, lo * kTile, n, s[lo & 1]);
  }
  for (int32_t j = lo; j < count; ++j) {
    const int32_t k0 = j * kTile;
    wait_rows();
    lds_barrier();                             // tile j is complete, tile j - 1 left
    const uint8_t flag = next_flag;
    if (j + 1 < count) {
      next_flag = flag_of(k0 + kTile + l);     // (before the tile: waiting for it waits for no row)
      fetch_tile<NW>(p, hkv, rope, k0 + kTile, n, s[(j + 1) & 1]);
    }
    if (k0 >= mine) continue;                  // the wave's queries see nothing here
    const TileLds& t = s[j & 1];
    f32x16 sc[2];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[kt][i] = 0.f;
      const int row = 32 * kt + col;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        sc[kt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            *reinterpret_cast<const bf16x8*>(t.nope + 256 * row + 16 * ((2 * ks + hi) ^ (row & 15))),
            qb[ks], sc[kt], 0, 0, 0);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        sc[kt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            *reinterpret_cast<const bf16x8*>(t.rope + 128 * row +
                                             16 * ((2 * ks + hi) ^ ((row >> 1) & 7))),
            qb[8 + ks], sc[kt], 0, 0, 0);
    }
    // ---- masks: keys without a row, keys past the query
    const uint64_t gone = __ballot(flag == 1), bad = __ballot(flag == 2);
    if (gone != 0 || bad != 0 || k0 + kTile > least) {
      const int32_t left = limit - k0;
      uint64_t seen = left >= kTile ? ~0ull : left <= 0 ? 0ull : (1ull << left) - 1ull;
      seen &= ~gone;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        const uint32_t see = (uint32_t)(seen >> (32 * kt)) >> (4 * hi);
        const uint32_t nan = (uint32_t)(bad >> (32 * kt)) >> (4 * hi);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t bit = 1u << (8 * (i / 4) + i % 4);
          if (nan & bit) sc[kt][i] = __builtin_nanf("");
          if (!(see & bit)) sc[kt][i] = -INFINITY;
        }
      }
    }
    // ---- online softmax; the maximum is renewed only when it grows by 2^8
    float mb = sc[0][0];
#pragma unroll
    for (int i = 1; i < 32; ++i) mb = fmaxf(mb, sc[i / 16][i % 16]);
    mb = max_halves(mb) * qk_scale;
    const bool grow = mb > m_run + kStaleMax;
    const float m_new = grow ? mb : m_run;
    const float alpha = grow ? __builtin_amdgcn_exp2f(m_run - m_new) : 1.f;
    const float base = m_new == -INFINITY ? 0.f : m_new;
    float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      sc[i / 16][i % 16] =
          __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i / 16][i % 16], qk_scale, -base));
      ls[i % 4] += sc[i / 16][i % 16];
    }
    l_run = l_run * alpha + ((ls[0] + ls[1]) + (ls[2] + ls[3]));
    m_run = m_new;
    if (__any(grow)) {
#pragma unroll
      for (int dt = 0; dt < 4; ++dt) o[dt] *= alpha;
    }
    // ---- O^T += V^T P^T: step ks covers keys 16 ks + 4 hi + {0..3, 8..11}
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const f32x16& x = sc[ks / 2];
      const int e = 8 * (ks % 2);
      const bf16x8 pb = __builtin_bit_cast(
          bf16x8, u32x4{bf16_pair(x[e], x[e + 1]), bf16_pair(x[e + 2], x[e + 3]),
                        bf16_pair(x[e + 4], x[e + 5]), bf16_pair(x[e + 6], x[e + 7])});
      const int sub = (l & 15) >> 2;           // the row this lane supplies: + 4 hi, and 8 on
      const uint8_t* v0 = t.val + 256 * (16 * ks + 4 * hi + sub);
#pragma unroll
      for (int dt = 0; dt < 4; ++dt) {
        const int c = (4 * dt + 2 * ((l >> 4) & 1) + ((l & 3) >> 1)) ^ (sub * 4);
        const u32x2 a = tr16_read(v0 + 16 * c + 8 * (l & 1));
        const u32x2 b = tr16_read(v0 + 8 * 256 + 16 * c + 8 * (l & 1));
        o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]}), pb, o[dt], 0, 0, 0);
      }
    }
  }
  if (wq + col >= nq) return;
  l_run += __shfl_xor(l_run, 32);
  const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
  const int64_t row = qrow * p.heads + head;
  if (p.splits == 1) {
    uint16_t* out = p.out + row * kVal + 4 * hi;
#pragma unroll
    for (int dt = 0; dt < 4; ++dt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<u32x2*>(out + 32 * dt + 8 * i) =
            u32x2{bf16_pair(o[dt][4 * i] * inv, o[dt][4 * i + 1] * inv),
                  bf16_pair(o[dt][4 * i + 2] * inv, o[dt][4 * i + 3] * inv)};
    return;
  }
  const int64_t ps = (int64_t)split * p.num_q * p.heads + row;
  float most = 0.f;
#pragma unroll
  for (int dt = 0; dt < 4; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(o[dt][i]));
  const int e = half_exponent(max_halves(most) * inv);
  if (hi == 0) {
    p.part_ml[kPartFloats * ps] = m_run;
    p.part_ml[kPartFloats * ps + 1] = l_run;
    p.part_ml[kPartFloats * ps + 2] = ldexpf(1.f, e);
  }
  if (l_run == 0.f) return;                    // the merge does not read it
  const float f = ldexpf(inv, -e);
  uint16_t* po = p.part_o + ps * kVal + 4 * hi;
#pragma unroll
  for (int dt = 0; dt < 4; ++dt)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<f16x4*>(po + 32 * dt + 8 * i) = half4(
          o[dt][4 * i] * f, o[dt][4 * i + 1] * f, o[dt][4 * i + 2] * f, o[dt][4 * i + 3] * f);
}

// Merges the key splits of a (query, head), 16 lanes 8 dimensions each: with
// w_s = 2^(m_s - M) l_s, out = sum_s w_s out_s / sum_s w_s.
__global__ void __launch_bounds__(256) prefill_merge_kernel(PrefillParams p) {
  const int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4), rows = (int64_t)p.num_q * p.heads;
  if (row >= rows) return;
  const int32_t q = (int32_t)(row / p.heads);
  // a query of no request: not written, left as it was
  if (q < p.query_start(0) || q >= p.query_start(p.num_reqs)) return;
  const int c = threadIdx.x & 15;
  float M = -INFINITY;
  for (int sp = 0; sp < p.splits; ++sp) {
    const int64_t ps = (int64_t)sp * rows + row;
    if (p.part_ml[kPartFloats * ps + 1] != 0.f) M = fmaxf(M, p.part_ml[kPartFloats * ps]);
  }
  float sum = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int sp = 0; sp < p.splits; ++sp) {
    const int64_t ps = (int64_t)sp * rows + row;
    const float* ml = p.part_ml + kPartFloats * ps;
    if (ml[1] == 0.f) continue;                // nothing seen there: not written
    const float x = exp2f(ml[0] - M) * ml[1];  // NaN stays NaN
    sum += x;
    const float y = x * ml[2];
    const f16x8 h = *reinterpret_cast<const f16x8*>(p.part_o + ps * kVal + 8 * c);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += y * (float)h[i];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<u32x4*>(p.out + row * kVal + 8 * c) =
      u32x4{bf16_pair(acc[0] * inv, acc[1] * inv), bf16_pair(acc[2] * inv, acc[3] * inv),
            bf16_pair(acc[4] * inv, acc[5] * inv), bf16_pair(acc[6] * inv, acc[7] * inv)};
}

template <int MW>
hipError_t launch_expand(const PrefillParams& p, hipStream_t stream) {
  static std::atomic<uint64_t> raised{0};
  const auto fn = prefill_expand_kernel<MW>;
  const hipError_t e = allow_full_lds(reinterpret_cast<const void*>(fn), raised);
  if (e != hipSuccess) return e;
  return launch_kernel(fn,
                       dim3((uint32_t)p.heads, (uint32_t)((p.num_kv + 64 * MW - 1) / (64 * MW))),
                       dim3(128 * MW), sizeof(GemmLds<MW>), stream, p);
}

constexpr size_t kAlign = 256;
size_t up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

}  // namespace

size_t plan_prefill(PrefillParams& p, void* workspace) {
  // Tiles of 256 queries (8 waves, one workgroup a unit) where the queries fill
  // them and the chip, else of 128 (4 waves, two a unit): 2,048 on 8,192 with 128
  // heads 1,320 us against 1,471, four requests of 753 on 4,849 with 64 heads 669
  // against 696; 512 on 1,024 with 64 heads 43 against 35.  Then as many key splits
  // as give the fewest key-tile times (about 1.4 us, 2 for 4 waves) over the
  // rounds of the chip, a workgroup's start and end and the merge counted in them:
  // 2,048 on 8,192 with 8 heads takes 90 us in four splits, 264 in one
  const int64_t R = p.num_reqs > 0 ? p.num_reqs : 1, nq = p.num_q;
  p.tile_rows = nq >= 256 * R && (nq / 256 + R) * p.heads >= 256 ? 256 : 128;
  p.max_tiles = (int32_t)min((int64_t)INT32_MAX, nq / p.tile_rows + p.num_reqs);
  const int64_t slots = p.tile_rows == 256 ? 256 : 512;
  const int64_t base = (nq + p.tile_rows - 1) / p.tile_rows * p.heads;
  const int64_t tiles = (p.num_kv / R + kTile - 1) / kTile;
  p.splits = 1;
  double best = 1e300;
  for (int n = 1; n <= kPrefillMaxSplits && n <= (tiles > 1 ? tiles : 1); n *= 2) {
    const double t = (double)((base * n + slots - 1) / slots) * ((tiles + n - 1) / n + 3) +
                     (n > 1 ? 3 + (double)nq * p.heads * n / 10000 : 0.0);
    if (t < best) {
      best = t;
      p.splits = n;
    }
  }
  uint8_t* at = static_cast<uint8_t*>(workspace);
  size_t n = 0;
  auto take = [&](size_t bytes) {
    uint8_t* q = at ? at + n : nullptr;
    n += up(bytes);
    return q;
  };
  const size_t kv = p.num_kv, H = p.heads;
  p.off = reinterpret_cast<int32_t*>(take((p.num_reqs + (size_t)1) * 4));
  p.tile_off = reinterpret_cast<int32_t*>(take((p.num_reqs + (size_t)1) * 4));
  p.flags = take(kv);
  p.lat = reinterpret_cast<uint16_t*>(take(kv * 512 * 2));
  p.rope = reinterpret_cast<uint16_t*>(take(kv * kRopeDim * 2));
  p.heads_kv = reinterpret_cast<uint16_t*>(take(H * kv * kHeadRow * 2));
  if (p.splits > 1) {
    p.part_o = reinterpret_cast<uint16_t*>(take((size_t)p.splits * nq * H * kVal * 2));
    p.part_ml = reinterpret_cast<float*>(take((size_t)p.splits * nq * H * kPartFloats * 4));
  }
  return n;
}

bool prefill_fits(const PrefillParams& p) {
  // tiles are a grid's second dimension
  return (int64_t)p.max_tiles * p.splits <= 65535 && ((int64_t)p.num_kv + 127) / 128 <= 65535 &&
         grid_fits(p.heads, 512) && grid_fits(((int64_t)p.num_q * p.heads + 15) / 16, 256);
}

hipError_t launch_prefill(const PrefillParams& p, bool fp4, hipStream_t stream) {
  if (p.num_reqs == 0 || p.num_q == 0) return hipSuccess;
  hipError_t e = hipSuccess;
  if (p.num_reqs > kInlineReqs) {
    e = launch_kernel(prefill_plan_kernel, dim3(1), dim3(1024), 0, stream, p);
    if (e != hipSuccess) return e;
  }
  // (at least one workgroup: the offsets)
  {
    e = launch_kernel(fp4 ? prefill_rows_kernel<true> : prefill_rows_kernel<false>,
                      dim3((uint32_t)((p.num_kv + 3) / 4 > 0 ? (p.num_kv + 3) / 4 : 1)), dim3(256), 0,
                      stream, p);
    if (e != hipSuccess) return e;
  }
  if (p.num_kv > 0) {
    // Tiles of 256 tokens (one workgroup a unit) read the weights half as often as
    // tiles of 128 (two a unit) and are taken where they fill the chip: 128 heads
    // of 8,192 tokens 405 us against 501, 8 of 8,192 (256 tiles) 24.1 against 28.9;
    // 16 of 2,048 (128 tiles) 19.3 against 14.9
    const int64_t tiles = ((int64_t)p.num_kv + 255) / 256 * p.heads;
    e = tiles >= 256 ? launch_expand<4>(p, stream) : launch_expand<2>(p, stream);
    if (e != hipSuccess) return e;
  }
  static std::atomic<uint64_t> raised[2];
  const bool big = p.tile_rows == 256;
  auto fn = big ? prefill_attend_kernel<8> : prefill_attend_kernel<4>;
  e = allow_full_lds(reinterpret_cast<const void*>(fn), raised[big]);
  if (e != hipSuccess) return e;
  e = launch_kernel(fn, dim3((uint32_t)p.heads, (uint32_t)(p.max_tiles * p.splits)),
                    dim3((uint32_t)p.tile_rows * 2), 2 * sizeof(TileLds), stream, p);
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t rows = (int64_t)p.num_q * p.heads;
  return launch_kernel(prefill_merge_kernel, dim3((uint32_t)((rows + 15) / 16)), dim3(256), 0, stream,
                       p);
}

}  // namespace hs
