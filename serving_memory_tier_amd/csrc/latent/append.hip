// Appending rows to the paged latent cache, with the position rotation on the
// way: the writer of the rows that the resolver, the gather, the offload and
// the attention read.
//
// Token i of request r at position n has the pool row
//   block_table[r][n / page] * page + n % page.
// Its 64 rope values are rotated by the angles n * freq[j], j < 32, its 512
// latent values quantised by groups, and the row stored in the layout's
// format; the same launch rotates the rope part of the token's queries.
//
// Scales.  A group's scale is the smallest power of two 2^e, e >= -126, with
//   max |x| <= 1.75 * 2^(e + E):  E = 8 for E4M3 (its largest value is 448),
//   E = 2 for E2M1 (7, which rounds to its largest value, 6),
// so no value saturates by more than half a step, and x / 2^e is exact: the
// only rounding is to the code.  Both formats are floating point, so a scale
// that is no power of two would gain nothing but the partly used top binade.
// A group with a NaN or an infinity stores a NaN scale: it reads back as NaN.
//
// Angles are formed and reduced in float64 (a position of a million times a
// frequency of 1 loses 2^-4 of a radian in float32).  The cached key is
// rotated in float64 and rounded to float32, then bfloat16 (the bytes do not
// depend on the order of float32 operations); the queries' sines and cosines
// are rounded to float32 and the rotation, in float32, to bfloat16.
//
// Work split: one workgroup of 4 waves per (token, head range).  Wave 0's
// first 32 lanes make the sines and cosines, which the others read from LDS;
// wave 1 quantises the latent values, 8 a lane (16 lanes an E4M3 group, 4 an
// E2M1 group: the largest value by lane exchanges); wave 2 rotates the key;
// then all rotate queries, 8 values a thread, their loads issued before the
// barrier.  Bound: HBM, 256 bytes a query head (12,048 tokens x 128 heads, FP8 rows:
// 430.6 MB in 92.5 us, 4.65 TB/s, 93 % of a large copy's rate); a launch of few
// tokens by its latency, the sines and two dependent loads for the row (32 tokens x
// 128 heads: 4.1 us).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "latent.h"
#include "parts.h"

namespace hs {
namespace {

constexpr int kThreads = 256;
constexpr int kLatent = 512;
constexpr int kPairs = 32;                     // rope pairs
constexpr int kHeadsPerRound = kThreads / 8;   // a thread rotates 8 values of a head
constexpr int kRounds = 4;                     // query loads in flight a thread

// Quantises lane l's eight latent values (wave-wide) into the row, and writes
// the values that the codes stand for.
template <bool FP4>
__device__ __forceinline__ void store_latent(u32x4 x, int l, uint8_t* row, uint16_t* values) {
  // bfloat16 magnitudes order as integers, NaN and infinity above the rest
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    most = max(most, x[i] & 0x7fffu);
    most = max(most, (x[i] >> 16) & 0x7fffu);
  }
  constexpr int kLanes = FP4 ? 4 : 16;         // lanes a group
#pragma unroll
  for (int d = 1; d < kLanes; d *= 2) most = max(most, (uint32_t)__shfl_xor((int)most, d));
  const bool bad = most >= 0x7f80u;
  int e = (int)(most >> 7) - 127 - (FP4 ? 2 : 8) + ((most & 127u) > 96u ? 1 : 0);
  e = most == 0 ? 0 : max(e, -126);
  const float up = __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
  const float down = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = bad ? 0.f : bf16_lo(x[i]) * down;
    y[2 * i + 1] = bad ? 0.f : bf16_hi(x[i]) * down;
  }
  const float scale = bad ? __builtin_nanf("") : up;
  u32x4 v;
  if constexpr (FP4) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[0], y[1], 1.f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], 1.f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[4], y[5], 1.f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[6], y[7], 1.f, 3);
    *reinterpret_cast<uint32_t*>(row + 4 * l) = w;
    if (l % kLanes == 0) row[256 + l / kLanes] = bad ? 255 : (uint8_t)(e + 127);
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 3);
    v = u32x4{bf16_pair(a[0] * scale, a[1] * scale), bf16_pair(b[0] * scale, b[1] * scale),
              bf16_pair(c[0] * scale, c[1] * scale), bf16_pair(d[0] * scale, d[1] * scale)};
  } else {
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
    *reinterpret_cast<u32x2*>(row + 8 * l) = u32x2{(uint32_t)lo, (uint32_t)hi};
    if (l % kLanes == 0) *reinterpret_cast<float*>(row + kLatent + 4 * (l / kLanes)) = scale;
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(lo, false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(lo, true);
    const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8(hi, false);
    const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8(hi, true);
    v = u32x4{bf16_pair(a[0] * scale, a[1] * scale), bf16_pair(b[0] * scale, b[1] * scale),
              bf16_pair(c[0] * scale, c[1] * scale), bf16_pair(d[0] * scale, d[1] * scale)};
  }
  if (values) *reinterpret_cast<u32x4*>(values + 8 * l) = v;
}

template <bool FP4, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendParams p) {
  __shared__ double cs[2][kPairs];
  __shared__ __attribute__((aligned(16))) float csf[2][kPairs];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  const int32_t r = p.token_req[t], n = p.positions[t];
  int32_t id = r < 0 ? -1 : -3;
  if (r >= 0 && r < p.num_reqs && n >= 0 && (n >> p.page_shift) < p.max_pages) {
    const int32_t b = p.block_table[(int64_t)r * p.max_pages + (n >> p.page_shift)];
    if (b >= 0 && b < p.pool_blocks)
      id = (b << p.page_shift) | (n & ((1 << p.page_shift) - 1));   // < pool_rows < 2^31
  }
  if (blockIdx.y == 0 && tid == 0 && p.row_ids) p.row_ids[t] = id;
  if (id < 0) return;                          // the whole workgroup: one token

  // this thread's query pieces: 8 values (4 pairs) of heads h0 + 32 i
  const int pc = tid & 7;
  const int32_t h0 = (int32_t)blockIdx.y * p.heads_per_group;
  const int32_t h1 = min(p.num_heads, h0 + p.heads_per_group);
  const uint16_t* q = p.q + t * p.q_token_stride;
  uint16_t* qo = p.q_out + t * p.q_out_token_stride;
  u32x4 v[kRounds];
  auto load = [&](int32_t base) {
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int32_t h = base + kHeadsPerRound * i + (tid >> 3);
      if (h >= h1) continue;
      const uint16_t* s = q + (int64_t)h * p.q_head_stride;
      if constexpr (INTERLEAVED) {
        v[i] = *reinterpret_cast<const u32x4*>(s + 8 * pc);
      } else {                                 // pairs (j, j + 32), j = 4 pc ..
        const u32x2 a = *reinterpret_cast<const u32x2*>(s + 4 * pc);
        const u32x2 b = *reinterpret_cast<const u32x2*>(s + kPairs + 4 * pc);
        v[i] = u32x4{a[0], a[1], b[0], b[1]};
      }
    }
  };
  load(h0);
  uint8_t* row = p.pool + (int64_t)id * (FP4 ? kFp4RowBytes : kFp8RowBytes);
  uint16_t* values = p.values ? p.values + t * (kLatent + 2 * kPairs) : nullptr;
  if (tid < kPairs) {
    double s, c;
    sincos((double)n * p.freq[tid], &s, &c);
    cs[0][tid] = c;
    cs[1][tid] = s;
    csf[0][tid] = (float)c;
    csf[1][tid] = (float)s;
  } else if (tid >= 64 && tid < 128 && blockIdx.y == 0) {
    const int l = tid - 64;
    store_latent<FP4>(*reinterpret_cast<const u32x4*>(p.latent + t * p.latent_stride + 8 * l), l,
                      row, values);
  }
  __syncthreads();
  if (tid >= 128 && tid < 128 + kPairs && blockIdx.y == 0) {
    const int j = tid - 128;
    const int ia = INTERLEAVED ? 2 * j : j, ib = INTERLEAVED ? 2 * j + 1 : j + kPairs;
    const uint16_t* s = p.rope + t * p.rope_stride;
    const double a = bf16_lo(s[ia]), b = bf16_lo(s[ib]);
    const double c = cs[0][j], sn = cs[1][j];
    float fu = (float)(a * c - b * sn), fw = (float)(a * sn + b * c);
    asm("" : "+v"(fu), "+v"(fw));              // both roundings, not one folded from float64
    const __bf16 u = (__bf16)fu, w = (__bf16)fw;
    __bf16* dst = reinterpret_cast<__bf16*>(row + (FP4 ? 256 + 16 : kLatent + 16));
    dst[ia] = u;
    dst[ib] = w;
    if (values) {
      __bf16* dv = reinterpret_cast<__bf16*>(values + kLatent);
      dv[ia] = u;
      dv[ib] = w;
    }
  }
  float c[4], s[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    c[j] = csf[0][4 * pc + j];
    s[j] = csf[1][4 * pc + j];
  }
  for (int32_t base = h0; base < h1; base += kRounds * kHeadsPerRound) {
    if (base > h0) load(base);
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int32_t h = base + kHeadsPerRound * i + (tid >> 3);
      if (h >= h1) continue;
      uint16_t* d = qo + (int64_t)h * p.q_out_head_stride;
      if constexpr (INTERLEAVED) {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a = bf16_lo(v[i][j]), b = bf16_hi(v[i][j]);
          w[j] = bf16_pair(a * c[j] - b * s[j], a * s[j] + b * c[j]);
        }
        *reinterpret_cast<u32x4*>(d + 8 * pc) = w;
      } else {
        float a[4] = {bf16_lo(v[i][0]), bf16_hi(v[i][0]), bf16_lo(v[i][1]), bf16_hi(v[i][1])};
        float b[4] = {bf16_lo(v[i][2]), bf16_hi(v[i][2]), bf16_lo(v[i][3]), bf16_hi(v[i][3])};
        float x[4], y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = a[j] * c[j] - b[j] * s[j];
          y[j] = a[j] * s[j] + b[j] * c[j];
        }
        *reinterpret_cast<u32x2*>(d + 4 * pc) = u32x2{bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3])};
        *reinterpret_cast<u32x2*>(d + kPairs + 4 * pc) =
            u32x2{bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3])};
      }
    }
  }
}

}  // namespace

bool append_fits(const AppendParams& p) {
  return grid_fits(p.num_tokens, kThreads) && p.num_heads <= 65535 * kHeadsPerRound * kRounds;
}

hipError_t launch_append(AppendParams p, bool fp4, bool interleaved, hipStream_t stream) {
  if (p.num_tokens == 0) return hipSuccess;
  p.heads_per_group = kHeadsPerRound * kRounds;
  const int32_t gy = p.num_heads > 0
                         ? (p.num_heads + p.heads_per_group - 1) / p.heads_per_group : 1;
  const dim3 grid((uint32_t)p.num_tokens, (uint32_t)gy);
  auto fn = fp4 ? (interleaved ? append_kernel<true, true> : append_kernel<true, false>)
                : (interleaved ? append_kernel<false, true> : append_kernel<false, false>);
  return launch_kernel(fn, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace hs
