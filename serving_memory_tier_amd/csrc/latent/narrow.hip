// Latent attention in the absorbed form for items of few query rows (at most 32:
// a tensor-parallel rank's heads): see decode.hip for the formulas and rounding.
//
// With 16 or 32 query rows a row's 656 or 400 bytes carry a fifth or less of the
// FLOPs that the matrix cores do meanwhile, so the aim is to keep rows coming.
// Work split: a workgroup of 4 waves takes all of an item's query rows and one
// range of its keys; each wave takes a quarter of the latent dimensions (and the
// first two half the rope's) for both products, 16x16x32 MFMAs:
//   S^T (32 keys x 16 rows a tile): the four shares are exchanged through LDS,
//     and every wave computes the softmax alike;
//   O^T (128 dimensions x 16 rows) += V^T P'^T, P' = p * scale.
// A wave then needs few registers (16 for queries and 32 for outputs a row tile),
// and each byte of a row is read from LDS by one wave for each product.
// Rows go from the pool into LDS as they are and are converted at use, exactly;
// two barriers a block (rows complete; shares complete), two workgroups a unit.
//
// Bound: with enough requests the rows' bytes (32 requests x 16 heads on half to
// all of 8,192 FP8 tokens, 129 MB: 43 us with the merge, 3.0 TB/s over all; 4-bit
// rows 44 us, 32 heads 58 and 59 us, bound by the conversions and the softmax that
// four waves repeat); with few requests a block's chain of barriers, LDS and MFMAs,
// 1.5 us: 3 requests x 16 heads on up to 500 tokens 13.3 us, of it the merge 4.8.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "decode_parts.h"

namespace hs {
namespace {

// Masks a block's scores (keys without a row, and keys the row does not see)
// where it has any to mask.  A lane's score 4 mt + r is key 16 mt + 4 g + r.
template <bool PAGED, int ROWS>
__device__ __forceinline__ void mask8(const Lists<ROWS>& s, const Share& sh, int bi, int row, int g,
                                     float (&sc)[8]) {
  const uint32_t there = s.there[bi];
  if (there == 0xffffffffu && (bi + 1) * kKeys <= sh.edge) return;
  const int left = s.mine[row] - bi * kKeys;
  uint32_t seen = left >= kKeys ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
  seen = (seen & there) >> (4 * g);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = 16 * (i / 4) + i % 4;
    if (PAGED && s.ids[bi * kKeys + 4 * g + at] == kBad) sc[i] = __builtin_nanf("");
    if (!(seen & (1u << at))) sc[i] = -INFINITY;
  }
}

// One block of the online softmax of a lane's 8 keys: scores, which qk_scale > 0
// brings to log2 units, to probabilities.  The maximum is renewed, and the output to be rescaled by the
// returned factor, only when it grows by 2^8.
__device__ __forceinline__ float softmax8(float (&sc)[8], float qk_scale, float& m_run,
                                         float& l_run) {
  float mb = sc[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mb = fmaxf(mb, sc[i]);
  mb = fmaxf(mb, __shfl_xor(mb, 16));
  mb = fmaxf(mb, __shfl_xor(mb, 32)) * qk_scale;
  const bool grow = mb > m_run + kStaleMax;
  const float m_new = grow ? mb : m_run;
  const float alpha = grow ? __builtin_amdgcn_exp2f(m_run - m_new) : 1.f;
  const float base = m_new == -INFINITY ? 0.f : m_new;    // nothing seen yet: exp2(-inf) = 0
  float ls = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sc[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], qk_scale, -base));
    ls += sc[i];
  }
  l_run = l_run * alpha + ls;
  m_run = m_new;
  return alpha;
}

constexpr int kWaves = 4, kThreads = 256;

template <bool FP4, int RT>
struct Lds {
  static constexpr int kBufs = !FP4 && RT == 2 ? 2 : 3;    // two workgroups a unit
  uint8_t raw[kBufs][kKeys * Row<FP4>::kBytes];
  f32x4 xs[kWaves][RT][2][64];  // partial scores: [wave][row tile][key tile]
  Lists<16 * RT> lists;
};

template <bool FP4, bool PAGED, int RT>
__global__ void __launch_bounds__(kThreads, 2) decode_narrow_kernel(DecodeParams p) {
  using R = Row<FP4>;
  using L = Lds<FP4, RT>;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
  L& s = *reinterpret_cast<L*>(lds_raw);
  Share sh;
  if (!begin<PAGED, 16 * RT>(p, s.lists, sh)) return;  // the whole workgroup
  int32_t* ids = s.lists.ids;
  const int blocks = (sh.n + kKeys - 1) / kKeys;
#pragma unroll
  for (int b = 0; b + 1 < L::kBufs; ++b)
    if (b < blocks) fetch_rows<FP4, kThreads>(p.kv, ids + b * kKeys, s.raw[b]);
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // the wave's 128 latent dimensions, and of the rope's 64 the first two waves 32
  // each.  A step's place 8 g + j of the contraction is a dimension that the keys
  // are read by: FP8 16 consecutive values a lane for two steps, 4-bit rows the
  // 32 values of one scale for all four
  bf16x8 qb[RT][5];
  {
    const int l = threadIdx.x & 63, g = l >> 4;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      // a lane past the last row takes the last row's queries; it writes nothing
      const int32_t m = min(sh.row0 + 16 * rt + (l & 15), p.rows - 1);
      const uint16_t* q = p.q + ((int64_t)sh.item * p.rows + m) * kDim;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        qb[rt][i] = signed_query(
            q + 128 * w + (FP4 ? 32 * g + 8 * i : 64 * (i / 2) + 16 * g + 8 * (i % 2)), p.scale);
      qb[rt][4] = signed_query(q + kLatent + 32 * (w & 1) + 8 * g, p.scale);
    }
  }
  // O^T of the wave's dimensions, by column (row of the tile): tile dt's rows are
  // dimensions 16 dt + 4 g + r; 4-bit rows: the even, then the odd dimensions of
  // each 32
  f32x4 o[RT][8];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int dt = 0; dt < 8; ++dt) o[rt][dt] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m_run[RT], l_run[RT];            // l_run: this lane's keys only
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    m_run[i] = -INFINITY;
    l_run[i] = 0.f;
  }
  const float qk_scale = positive_scale(p.scale);
  int cur = 0;                                 // bi modulo the buffers
  for (int bi = 0; bi < blocks; ++bi) {
    uint8_t* raw = s.raw[cur];
    const int l = fresh_tid() & 63, col = l & 15, g = l >> 4;
    wait_rows();                               // this block's, asked for a block or two ago
    if (PAGED && (bi + 1) * kKeys > sh.edge)
      sanitize_rows<FP4, kThreads>(raw, ids + bi * kKeys, sh.edge - bi * kKeys);
    lds_barrier();                             // complete; and the block before is done with
    const int ahead = L::kBufs - 1;
    if (bi + ahead < blocks)
      fetch_rows<FP4, kThreads>(p.kv, ids + (bi + ahead) * kKeys,
                                s.raw[cur + ahead >= L::kBufs ? cur - 1 : cur + ahead]);
    cur = cur + 1 == L::kBufs ? 0 : cur + 1;
    // ---- this wave's share of S^T: two tiles of 16 keys
    f32x4 sc[RT][2];
    float ks[8];                               // FP8: the scales of this lane's keys, this tile's
    uint32_t ks4[8];                           // 4-bit: four scales each
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint8_t* at = raw + (16 * (i / 4) + 4 * g + i % 4) * R::kBytes + R::kScales + 4 * w;
      if constexpr (FP4)
        ks4[i] = *reinterpret_cast<const uint32_t*>(at);
      else
        ks[i] = *reinterpret_cast<const float*>(at);
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const uint8_t* row = raw + (16 * mt + col) * R::kBytes;
      bf16x8 kf[4];
      if constexpr (FP4) {
        const u32x4 k = *reinterpret_cast<const u32x4*>(row + 64 * w + 16 * g);
        const float sf = __builtin_bit_cast(float, (uint32_t)row[R::kScales + 4 * w + g] << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i) kf[i] = fp4x8(k[i], sf);
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const u32x4 k = *reinterpret_cast<const u32x4*>(row + 128 * w + 64 * c + 16 * g);
          kf[2 * c] = fp8x8(k[0], k[1]);
          kf[2 * c + 1] = fp8x8(k[2], k[3]);
        }
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) sc[rt][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          sc[rt][mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[i], qb[rt][i], sc[rt][mt], 0, 0, 0);
      if constexpr (!FP4) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int r = 0; r < 4; ++r) sc[rt][mt][r] *= ks[4 * mt + r];
      }
      if (w < 2) {
        const bf16x8 rope = *reinterpret_cast<const bf16x8*>(row + R::kRope + 64 * w + 16 * g);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          sc[rt][mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(rope, qb[rt][4], sc[rt][mt], 0, 0, 0);
      }
    }
    // ---- the shares are exchanged; a fixed order of the sum
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) s.xs[w][rt][mt][l] = sc[rt][mt];
    lds_barrier();
    float x[RT][8];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < kWaves; ++v)
          sum += s.xs[v][i][mt][l];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[i][4 * mt + r] = sum[r];
      }
      mask8<PAGED, 16 * RT>(s.lists, sh, bi, 16 * i + col, g, x[i]);
      const float alpha = softmax8(x[i], qk_scale, m_run[i], l_run[i]);
      if (__any(alpha != 1.f)) {
#pragma unroll
        for (int dt = 0; dt < 8; ++dt) o[i][dt] *= alpha;
      }
    }
    // ---- O^T += V^T P'^T over the 32 keys, P' = p * scale: place 8 g + 4 mt + r
    // of the contraction is key 16 mt + 4 g + r, which this lane holds; lane c of
    // a 16-lane group supplies row c / 2 of those eight and 8 bytes
    const int j = col >> 1;
    const uint8_t* vrow = raw + ((j < 4 ? 0 : 12) + 4 * g + j) * R::kBytes + (FP4 ? 64 : 128) * w +
                          8 * (col & 1);
    bf16x8 pb[RT];
    auto weigh = [&](const float (&k)[8]) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = x[rt][i] * k[i];
        pb[rt] = __builtin_bit_cast(bf16x8, u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]),
                                                  bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])});
      }
    };
    if constexpr (FP4) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float k[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          k[i] = __builtin_bit_cast(float, ((ks4[i] >> (8 * q)) & 255u) << 23);
        weigh(k);
        // bytes of two dimensions: the even and the odd ones make two operands
        const u32x2 v = tr8_read(vrow + 16 * q);
        uint32_t e[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          e[4 * h] = fp4_pair<0>(v[h]);
          e[4 * h + 1] = fp4_pair<1>(v[h]);
          e[4 * h + 2] = fp4_pair<2>(v[h]);
          e[4 * h + 3] = fp4_pair<3>(v[h]);
        }
        u32x4 even, odd;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          even[h] = __builtin_amdgcn_perm(e[2 * h + 1], e[2 * h], 0x05040100u);
          odd[h] = __builtin_amdgcn_perm(e[2 * h + 1], e[2 * h], 0x07060302u);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          o[rt][2 * q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, even),
                                                                 pb[rt], o[rt][2 * q], 0, 0, 0);
          o[rt][2 * q + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, odd), pb[rt], o[rt][2 * q + 1], 0, 0, 0);
        }
      }
    } else {
      weigh(ks);
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) {
        const u32x2 v = tr8_read(vrow + 16 * dt);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          o[rt][dt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8x8(v[0], v[1]), pb[rt], o[rt][dt],
                                                              0, 0, 0);
      }
    }
  }

  // ---- the rows' sums, then this wave's 128 dimensions of every row
  const int l = fresh_tid() & 63, col = l & 15, g = l >> 4;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    l_run[i] += __shfl_xor(l_run[i], 16);
    l_run[i] += __shfl_xor(l_run[i], 32);
    const int32_t m = sh.row0 + 16 * i + col;
    if (w == 0 && g == 0 && m < p.rows) {
      if (p.splits == 1) {
        p.lse[(int64_t)sh.item * p.rows + m] =
            l_run[i] == 0.f ? -INFINITY : (m_run[i] + log2f(l_run[i])) / kLog2e;
      } else {
        const int64_t ps = sh.part * p.rows + m;
        *reinterpret_cast<f32x2*>(p.part_ml + kPartFloats * ps) = f32x2{m_run[i], l_run[i]};
      }
    }
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int32_t m = sh.row0 + 16 * rt + col;
    if (m >= p.rows) continue;
    const float sum = l_run[rt];
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t mrow = (int64_t)sh.item * p.rows + m;
    const int64_t ps = sh.part * p.rows + m;
    if (p.splits > 1 && sum == 0.f) continue;  // the merge does not read it
    float f = inv;
    if (p.splits > 1) {
      float most = 0.f;                        // of the row's 128 dimensions: four lanes'
#pragma unroll
      for (int dt = 0; dt < 8; ++dt)
#pragma unroll
        for (int r = 0; r < 4; ++r) most = fmaxf(most, fabsf(o[rt][dt][r]));
      most = fmaxf(most, __shfl_xor(most, 16));
      most = fmaxf(most, __shfl_xor(most, 32));
      const int e = half_exponent(most * inv);
      if (g == 0) p.part_ml[kPartFloats * ps + 2 + w] = ldexpf(1.f, e);
      f = ldexpf(inv, -e);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // FP8: 16 (2 q) + 4 g + r, then 16 more; 4-bit: 32 q + 8 g + 2 r, even and odd
      const f32x4 a = o[rt][2 * q] * f, b = o[rt][2 * q + 1] * f;
      const int at = 128 * w + 32 * q + (FP4 ? 8 : 4) * g;
      if (p.splits == 1) {
        uint16_t* out = p.out + mrow * kLatent + at;
        if constexpr (FP4) {
          *reinterpret_cast<u32x4*>(out) = u32x4{bf16_pair(a[0], b[0]), bf16_pair(a[1], b[1]),
                                                 bf16_pair(a[2], b[2]), bf16_pair(a[3], b[3])};
        } else {
          *reinterpret_cast<u32x2*>(out) = u32x2{bf16_pair(a[0], a[1]), bf16_pair(a[2], a[3])};
          *reinterpret_cast<u32x2*>(out + 16) = u32x2{bf16_pair(b[0], b[1]), bf16_pair(b[2], b[3])};
        }
      } else {
        uint16_t* po = p.part_o + ps * kLatent + at;
        if constexpr (FP4) {
          *reinterpret_cast<f16x4*>(po) = half4(a[0], b[0], a[1], b[1]);
          *reinterpret_cast<f16x4*>(po + 4) = half4(a[2], b[2], a[3], b[3]);
        } else {
          *reinterpret_cast<f16x4*>(po) = half4(a[0], a[1], a[2], a[3]);
          *reinterpret_cast<f16x4*>(po + 16) = half4(b[0], b[1], b[2], b[3]);
        }
      }
    }
  }
}

template <int RT>
hipError_t launch_rows(const DecodeParams& p, bool fp4, bool paged, hipStream_t stream) {
  static std::atomic<uint64_t> raised[3];
  const int n = !paged ? 0 : fp4 ? 1 : 2;
  auto fn = n == 0 ? decode_narrow_kernel<true, false, RT>
            : n == 1 ? decode_narrow_kernel<true, true, RT> : decode_narrow_kernel<false, true, RT>;
  const hipError_t e = allow_full_lds(reinterpret_cast<const void*>(fn), raised[n]);
  if (e != hipSuccess) return e;
  const size_t lds = fp4 ? sizeof(Lds<true, RT>) : sizeof(Lds<false, RT>);
  return launch_kernel(fn, dim3((uint32_t)decode_grid(p)), dim3(kThreads), lds, stream, p);
}

}  // namespace

hipError_t launch_decode_narrow(const DecodeParams& p, bool fp4, bool paged, hipStream_t stream) {
  return p.tile_rows == 16 ? launch_rows<1>(p, fp4, paged, stream) : launch_rows<2>(p, fp4, paged, stream);
}

}  // namespace hs
