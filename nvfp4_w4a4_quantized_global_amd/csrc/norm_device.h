// What the RMS norm (norm.hip) and the layer norm (layernorm.hip) share: how rows are laid out
// over lanes and workgroups, and a lane's 16 values as loaded, rounded and stored.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <numeric>

#include "nvfp4_device.h"
#include "nvfp4_launch.h"
#include "quantize_device.h"

namespace nvfp4 {

constexpr int kGroupThreads = 256;   // workgroup of the several-rows form

// Lanes per row and threads per workgroup for rows of k values.
struct RowShape {
  int lanes, threads;
};
inline RowShape row_shape(int64_t k) {
  const int chunks = (int)(k / kBlock);
  if (chunks <= 64) {
    int l = 8;
    while (l < chunks) l *= 2;
    return {l, kGroupThreads};
  }
  const int t = (chunks + 63) / 64 * 64;
  return {t, t};
}

// 16 values as loaded (8 words of bf16 pairs or 16 of fp32), expanded where used: a load
// can be in flight while other work goes on.
template <bool kF32>
struct Raw16 {
  uint4 raw[kF32 ? 4 : 2];
  __device__ __forceinline__ void load(const void* w, int64_t off) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(w) + off * (kF32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (kF32 ? 4 : 2); ++i) raw[i] = p[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (kF32 ? 4 : 2); ++i) raw[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float get(int i) const {
    const uint4& q = raw[kF32 ? i / 4 : i / 8];
    const int e = kF32 ? i & 3 : (i >> 1) & 3;
    const uint32_t u = e == 0 ? q.x : e == 1 ? q.y : e == 2 ? q.z : q.w;
    return kF32 ? __uint_as_float(u) : __uint_as_float((i & 1) ? u & 0xFFFF0000u : u << 16);
  }
};

template <bool kF32>
__device__ __forceinline__ void load_stream16(const void* p, int64_t off, float (&v)[16]) {
  if constexpr (kF32) load16_f32(static_cast<const float*>(p) + off, v);
  else load16_bf16(static_cast<const uint16_t*>(p) + off, v);
}

__device__ __forceinline__ void round_bf16(float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = gemm::pack_bf16x2(v[2 * i], v[2 * i + 1]);
    v[2 * i] = __uint_as_float(w << 16);
    v[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
  }
}

// v already rounded to the stream's type.
template <bool kF32>
__device__ __forceinline__ void store_stream16(void* p, int64_t off, const float (&v)[16]) {
  if constexpr (kF32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
    store16_bf16(static_cast<uint16_t*>(p) + off, v);
  }
}

__device__ __forceinline__ double sum_squares(const float (&v)[16]) {
  double a = 0.0, b = 0.0;
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    a = fma((double)v[i], (double)v[i], a);
    b = fma((double)v[i + 1], (double)v[i + 1], b);
  }
  return a + b;
}

__device__ __forceinline__ float row_scale(double sum, int64_t k, double eps) {
  return (float)(1.0 / sqrt(sum / (double)k + eps));
}

// Sum over the `lanes` lanes of a row (a power of two within a wave).
template <typename T>
__device__ __forceinline__ T group_sum(T v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// y = bf16((r * s) * w), over r.
template <bool kWF32>
__device__ __forceinline__ void normalize16(float (&v)[16], float s, const Raw16<kWF32>& w) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], s), w.get(i));
  round_bf16(v);
}

// Workgroups of the row-walking kernels, whose results are joined afterwards: two for each
// compute unit where they have four waves or more, about ten waves a unit where fewer.
// Gradient, both kernels: 4096 x 5120 (five waves) with 256 / 512 / 768 workgroups 48 / 36 /
// 44 us, 16384 x 1040 (two waves) with 512 / 1024 / 1280 75 / 44 / 41.  Statistics and second
// pass of the dynamic scale: 4096 x 5120 with 256 / 512 / 768 / 1024 48.9 / 39.4 / 39.7 / 41.1,
// 16384 x 5120 201 / 149 / 150 / 165, 16384 x 1040 with 512 / 1280 71 / 45.
inline int64_t walking_blocks(int64_t rows, const RowShape& s) {
  const int64_t per = s.threads / s.lanes;
  const int64_t most = s.threads >= 256 ? 512 : 2560 * 64 / s.threads;
  static_assert(2560 * 64 / 128 <= kNormPartials, "rows longer than 1024 take two waves at least");
  return std::min<int64_t>((rows + per - 1) / per, most);
}

constexpr int kNormQThreads = 256;   // workgroup of a dynamic scale's second pass

// Second-pass workgroups: a whole number of rows' tiles (at most 128) between a lane's
// units, so that its tile of the weight stays the same.
inline int64_t quantize_blocks(int64_t rows, int64_t k) {
  const int64_t kt = (k + kScaleTileK - 1) / kScaleTileK;
  const int64_t want = std::min<int64_t>((rows * kt + kNormQThreads / 8 - 1) / (kNormQThreads / 8), 2048);
  const int64_t unit = kt / std::gcd(kt, (int64_t)(kNormQThreads / 8));
  return std::max<int64_t>(want / unit, 1) * unit;
}

}  // namespace nvfp4
