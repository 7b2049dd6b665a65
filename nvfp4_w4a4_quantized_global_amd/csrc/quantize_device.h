// 16-value loads and stores and the NVFP4 encoding of one 128-wide K tile, shared by the
// quantizer (quantize.hip) and the RMS norm (norm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.h"
#include "nvfp4_device.h"

namespace nvfp4 {

// 16 consecutive fp32 values (64 bytes, 16-byte aligned).
__device__ __forceinline__ void load16_f32(const float* __restrict__ p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 t = reinterpret_cast<const float4*>(p)[i];
    v[4 * i] = t.x; v[4 * i + 1] = t.y; v[4 * i + 2] = t.z; v[4 * i + 3] = t.w;
  }
}

// Stores 16 values that are already bf16-exact as bf16.
__device__ __forceinline__ void store16_bf16(uint16_t* __restrict__ p, const float (&v)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = (__float_as_uint(v[2 * i]) >> 16) | (__float_as_uint(v[2 * i + 1]) & 0xFFFF0000u);
  uint4* d = reinterpret_cast<uint4*>(p);
  d[0] = make_uint4(w[0], w[1], w[2], w[3]);
  d[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// One lane's share of a quantize unit (row, 128-wide K tile): lane j of the unit's eight
// owns 16-block j.  v holds its 16 input values (zeros past the end); the block is
// rotated (all lanes of the wave take part), quantized under global scale gsf, and its
// codes (and, with a16, its fp16 operand form) stored; the unit's 8 scale bytes are
// gathered into lane j == 0 and written as one 8-byte word.
template <bool kRotate>
__device__ __forceinline__ void quantize_unit(float (&v)[16], int64_t row, int64_t kt, int j, int64_t m_rows,
                                              int64_t k, int group, float inv_sqrt_g, float gsf,
                                              uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                              uint16_t* __restrict__ a16) {
  if (kRotate) rotate16_bf16(v, group, inv_sqrt_g);
  const int64_t blk = kt * 8 + j;
  const bool in_row = row < m_rows;
  const bool valid = in_row && blk < k / kBlock;
  uint32_t w0, w1;
  const uint32_t s8 = quantize_block16(v, gsf, valid, w0, w1);
  if (valid) *reinterpret_cast<uint2*>(codes + row * (k / 2) + blk * 8) = make_uint2(w0, w1);
  if (a16 != nullptr && valid) {
    // the block's values in the GEMMs' operand form: fp16 code * scale * 2^-8, exact
    const gemm::half2_t sc = gemm::as_half2((s8 << 7) | (s8 << 23));
    uint4* d = reinterpret_cast<uint4*>(a16 + row * k + blk * kBlock);
    d[0] = __builtin_bit_cast(uint4, gemm::dequant8(w0, sc));
    d[1] = __builtin_bit_cast(uint4, gemm::dequant8(w1, sc));
  }
  uint32_t lo = j < 4 ? s8 << (8 * j) : 0u;
  uint32_t hi = j >= 4 ? s8 << (8 * (j - 4)) : 0u;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo |= __shfl_xor(lo, o, 64);
    hi |= __shfl_xor(hi, o, 64);
  }
  if (j == 0 && in_row) *reinterpret_cast<uint2*>(scales + (kt * m_rows + row) * 8) = make_uint2(lo, hi);
}

}  // namespace nvfp4
