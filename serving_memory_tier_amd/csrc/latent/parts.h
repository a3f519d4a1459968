// Pieces that the latent attention kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hs {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kStaleMax = 8.f;             // log2 of the largest unnormalised probability

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(2))) int i32x2;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;

// Within each 16 lanes, lane c receives element c % 4 of the 8-byte vectors at
// the addresses of lanes 4 j + c / 4, j = 0..3.
__device__ __forceinline__ u32x2 tr16_read(const uint8_t* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (lds_s16x4*)(const_cast<uint8_t*>(p))));
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// Within each 16 lanes, lane c receives byte c % 8 of the 8-byte vectors at the
// addresses of lanes 2 j + c / 8, j = 0..7.
__device__ __forceinline__ u32x2 tr8_read(const uint8_t* p) {
  return __builtin_bit_cast(
      u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)(const_cast<uint8_t*>(p))));
}

// Whether any of eight bfloat16 values is a NaN or an infinity.
__device__ __forceinline__ bool bad_bf16(u32x4 w) {
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    bad |= (w[j] & 0x7f800000u) == 0x7f800000u || (w[j] & 0x7f80u) == 0x7f80u;
  return bad;
}

template <bool HI>
__device__ __forceinline__ uint32_t fp8_pair(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}

// Eight E4M3 bytes as bfloat16, exactly.
__device__ __forceinline__ bf16x8 fp8x8(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(
      bf16x8, u32x4{fp8_pair<false>(a), fp8_pair<true>(a), fp8_pair<false>(b), fp8_pair<true>(b)});
}

// The two E2M1 values of byte B of a word times a power of two, as bfloat16,
// exactly (an infinite scale: NaN).
template <int B>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t w, float scale = 1.f) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, B));
}

// Eight E2M1 values times a power of two.
__device__ __forceinline__ bf16x8 fp4x8(uint32_t w, float scale) {
  return __builtin_bit_cast(bf16x8, u32x4{fp4_pair<0>(w, scale), fp4_pair<1>(w, scale),
                                          fp4_pair<2>(w, scale), fp4_pair<3>(w, scale)});
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) {
  return __builtin_bit_cast(float, w & 0xffff0000u);
}

// Whether 32 E2M1 values times their E8M0 scale hold a NaN, or one past the
// range of bfloat16: 2 and up times 2^127, 4 and up times 2^126.
__device__ __forceinline__ bool bad_fp4(u32x4 w, uint32_t scale) {
  if (scale < 253u) return false;
  uint32_t big = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) big |= scale == 253u ? w[j] & (w[j] << 1) : w[j];
  return scale == 255u || (big & 0x44444444u) != 0;
}

// The larger of a lane's value and that of the lane 32 away.
__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x),
                                                  __builtin_bit_cast(uint32_t, x), false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}

// Scores stay as the products give them and are scaled in the exponent, so the
// scale has to be positive: a negative one turns the queries' signs instead, zero
// becomes the least that keeps a masked score -infinity.
__device__ __forceinline__ float positive_scale(float scale) {
  const float s = fmaxf(fabsf(scale) * kLog2e, 1e-38f);
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, s)));
}

__device__ __forceinline__ bf16x8 signed_query(const uint16_t* q, float scale) {
  return __builtin_bit_cast(
      bf16x8, *reinterpret_cast<const u32x4*>(q) ^ (scale < 0.f ? 0x80008000u : 0u));
}

// The power of two (its exponent) that brings values of magnitude `most` at the
// largest to [1, 2), where half precision keeps 11 bits of them.
__device__ __forceinline__ int half_exponent(float most) {
  // (no further than what the factor 2^-e allows)
  return most > 0.f && most < INFINITY ? max(__builtin_amdgcn_frexp_expf(most) - 1, -120) : 0;
}

__device__ __forceinline__ f16x4 half4(float a, float b, float c, float d) {
  return f16x4{(_Float16)a, (_Float16)b, (_Float16)c, (_Float16)d};
}

// The sums of x over this lane and those before it; all 64 lanes take part.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);    // within 16 lanes:
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);    // 1, 2, 4, 8 lanes up
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);   // lane 15 to the next 16
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);   // lane 31 to the upper 32
  return x;
}

__device__ __forceinline__ int lane_of(int x, int l) { return __builtin_amdgcn_readlane(x, l); }

// The thread's number, opaque to the compiler: what it addresses with it is
// computed where it is used instead of held in registers over the loop.
__device__ __forceinline__ int fresh_tid() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// 16 bytes a lane from the pool straight into LDS: a wave's lanes fill 1024
// consecutive bytes from `base`, which is the same in all of them.  Written out
// because the compiler waits for its own form of this load before every
// transposing LDS read that follows; here wait_rows() and a barrier order them.
// It has no register output, and the compiler's waits for its other loads only
// become longer by loads that it does not count.  (M0 has no other user here: LDS
// accesses need none, and no register array is indexed at run time.)
__device__ __forceinline__ void load_to_lds(const uint8_t* src, uint8_t* base) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)base;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(__builtin_amdgcn_readfirstlane(at)), "v"(src)
               : "memory");
}

// A barrier that leaves loads into LDS on their way (__syncthreads would wait
// for all of them); this wave's other LDS accesses are done.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Waits for this wave's loads into LDS (and its others: the compiler knows this
// wait and adds none behind it); a barrier makes them every wave's.
__device__ __forceinline__ void wait_rows() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0f70);          // vmcnt(0), the other counters at their largest
  asm volatile("" ::: "memory");
}

}  // namespace
}  // namespace hs
