// The 8-bit block format, shared by every kernel that writes it.
//
// A row of K values is cut into blocks of 128 (the last may be shorter); a weight into tiles
// of 128 x 128.  A block stores E4M3 codes and one fp32 scale:
//   a = largest finite magnitude, at least 448 * 2^-110,
//   scale = fp32(a / 448),   code = E4M3_nearest_even(fp32(v * fp32(448 / a))).
// The floor keeps both quotients finite and normal: a block of zeros, or of values that tiny,
// has zero codes.  a * fp32(448 / a) is within 2^-23 of 448, so finite values never leave
// E4M3's range; infinities and NaN become NaN codes and do not enter the scale.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "checkpoint_device.h"

namespace nvfp4 {

constexpr int kFp8Block = 128;

// The scale of a block from its largest finite magnitude (as bits), and the factor that
// brings its values to codes.
__device__ __forceinline__ float fp8_scale(uint32_t amax_bits, float& factor) {
  const float a = fmaxf(__uint_as_float(amax_bits), 448.0f * 0x1p-110f);
  factor = __fdiv_rn(448.0f, a);
  return __fdiv_rn(a, 448.0f);
}

// 16 values to codes.
__device__ __forceinline__ uint4 fp8_encode16(const float (&v)[16], float factor) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int t = __builtin_amdgcn_cvt_pk_fp8_f32(__fmul_rn(v[4 * i], factor), __fmul_rn(v[4 * i + 1], factor), 0, false);
    t = __builtin_amdgcn_cvt_pk_fp8_f32(__fmul_rn(v[4 * i + 2], factor), __fmul_rn(v[4 * i + 3], factor), t, true);
    w[i] = (uint32_t)t;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight consecutive lanes hold a row's block, 16 values each (zeros past the row's end): the
// codes of this lane's values and the block's scale.  Every lane of the wave takes part.
__device__ __forceinline__ uint4 fp8_block16(const float (&v)[16], float& scale) {
  uint32_t m = ck_amax_bits(v);
  // lane ^ 1, lane ^ 2, and 7 - lane of the eight, by the vector unit's lane moves
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, true));
  float factor;
  scale = fp8_scale(m, factor);
  return fp8_encode16(v, factor);
}

}  // namespace nvfp4
