// The 8-bit activation checkpoint format, shared by every kernel that writes or reads it.
//
// A row of K values is cut into blocks of 32 (the last may hold 16).  A block stores E4M3
// codes and one byte s for the power of two 2^(s - 127) they are multiplied by: the
// smallest power, between 2^-110 and 2^120, that brings the block's largest finite
// magnitude to 448 or below.  A power of two keeps E4M3's three significand bits, so
// code * scale is exact in bf16 (the matrix cores' operand type) and packing rounds once,
// by at most 2^-4 of the value (2^-10 of the block's scale below 2^-6 of it).  Infinities
// and NaN become NaN codes and do not enter the scale; a zero block takes 2^-110.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

constexpr int kCkBlock = 32;
constexpr int kCkMinExp = -110, kCkMaxExp = 120;

// Largest finite magnitude of 16 values, as its bits.
__device__ __forceinline__ uint32_t ck_amax_bits(const float (&v)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t a = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    m = max(m, a < 0x7F800000u ? a : 0u);
  }
  return m;
}

// Block exponent: 448 = 1.75 * 2^8, so a magnitude 1.f * 2^q needs 2^(q - 8), or twice
// that when 1.f > 1.75.
__device__ __forceinline__ int ck_exponent(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 135 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kCkMinExp), kCkMaxExp);
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// 16 values to E4M3 codes under exponent e.  The hardware conversion rounds to nearest
// even; the scaled finite values never exceed 448.
__device__ __forceinline__ uint4 ck_encode16(const float (&v)[16], int e) {
  const float s = pow2f(-e);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int t = __builtin_amdgcn_cvt_pk_fp8_f32(__fmul_rn(v[4 * i], s), __fmul_rn(v[4 * i + 1], s), 0, false);
    t = __builtin_amdgcn_cvt_pk_fp8_f32(__fmul_rn(v[4 * i + 2], s), __fmul_rn(v[4 * i + 3], s), t, true);
    w[i] = (uint32_t)t;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Lane pairs (2i, 2i + 1) hold the two 16-value halves of a block (zeros where the row
// has none): the codes of this lane's half and the block's scale byte.  Every lane of the
// wave takes part (a shuffle).
__device__ __forceinline__ uint4 ck_pack16(const float (&v)[16], uint32_t& scale_byte) {
  uint32_t m = ck_amax_bits(v);
  m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
  const int e = ck_exponent(m);
  scale_byte = (uint32_t)(e + 127);
  return ck_encode16(v, e);
}

// 16 codes back to fp32 values (exact).
__device__ __forceinline__ void ck_decode16(const uint4& c, uint32_t scale_byte, float (&v)[16]) {
  const float s = pow2f((int)scale_byte - 127);
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
    v[4 * i] = __fmul_rn(lo[0], s);
    v[4 * i + 1] = __fmul_rn(lo[1], s);
    v[4 * i + 2] = __fmul_rn(hi[0], s);
    v[4 * i + 3] = __fmul_rn(hi[1], s);
  }
}

}  // namespace nvfp4
