// 8-bit block codes (fp8_device.h) on gfx950: activations in blocks of 128 values of a row,
// weights in tiles of 128 x 128 (with their transposed copy for the input's gradient), and back.
// All of it is bound by HBM traffic (a 1 GiB copy: 5.06 TB/s): 4096 x 5120 from bf16 11.4 us
// (5.5 TB/s, from the last-level cache in part), with column sums 13.3 + 3.9, with the checkpoint
// 15.1 to 17.6 (4.8 to 5.6; in two calls 27); the SwiGLU product of 4096 x 25600 139 us (131 to 152; 3.8
// TB/s; fewer and longer workgroups are slower); a weight 25600 x 5120 from fp32 123 us (5.3), with the
// transposed copy 150 (5.3), that from bf16 104 (5.0); back to bf16 70 us (5.6).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "fp8_device.h"
#include "gemm_common.h"
#include "nvfp4_device.h"
#include "nvfp4_launch.h"
#include "quantize_device.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kQBlocks = 4, kQRows = 8;   // blocks of a row, and rows, a workgroup holds at a time

// Activation rows to codes [rows][k] and scales [ceil(k / 128)][rows].  Eight lanes own a block;
// a workgroup takes four neighbouring blocks (1 KB of bf16) of eight rows, so that loads come in
// long runs and the scales of a block in runs of eight rows.  kSwiglu: the input is the SwiGLU
// product of x (gate) and up.  kSum: the workgroup walks down the rows and writes one partial row
// of column sums (partials [gridDim.y][k]).  kCheckpoint: x's 8-bit checkpoint from the same read.
template <bool kSwiglu, bool kSum, bool kCheckpoint>
__global__ void __launch_bounds__(kThreads) fp8_quantize_kernel(const uint16_t* __restrict__ x,
                                                                const uint16_t* __restrict__ up, int64_t rows,
                                                                int64_t k, uint8_t* __restrict__ codes,
                                                                float* __restrict__ scales,
                                                                float* __restrict__ partials,
                                                                uint8_t* __restrict__ ck_codes,
                                                                uint8_t* __restrict__ ck_scales) {
  __shared__ float sums[kSum ? kThreads * 16 : 1];
  const int t = threadIdx.x;
  const int unit = t >> 3, j = t & 7;
  const int rl = unit / kQBlocks;
  const int64_t blk = (int64_t)blockIdx.x * kQBlocks + unit % kQBlocks;
  const int64_t col = blk * kFp8Block + j * 16;
  const bool in_k = col < k;
  float sum[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) sum[i] = 0.0f;
  for (int64_t row0 = (int64_t)blockIdx.y * kQRows; row0 < rows; row0 += (int64_t)gridDim.y * kQRows) {
    const int64_t row = row0 + rl;
    const bool valid = in_k && row < rows;
    float v[16];
    if (valid) {
      load16_bf16(x + row * k + col, v);
      if constexpr (kSwiglu) {
        float u[16];
        load16_bf16(up + row * k + col, u);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = swiglu_bf16(v[i], u[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    }
    if constexpr (kSum) {
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[i] += v[i];
    }
    float scale;
    const uint4 c = fp8_block16(v, scale);
    if (valid) {
      *reinterpret_cast<uint4*>(codes + row * k + col) = c;
      if (j == 0) scales[blk * rows + row] = scale;
    }
    if constexpr (kCheckpoint) {
      uint32_t byte;
      const uint4 q = ck_pack16(v, byte);
      if (valid) {
        *reinterpret_cast<uint4*>(ck_codes + row * k + col) = q;
        if ((j & 1) == 0) ck_scales[row * ((k + kCkBlock - 1) / kCkBlock) + col / kCkBlock] = (uint8_t)byte;
      }
    }
  }
  if constexpr (kSum) {
    // the eight rows' sums side by side, added in row order
#pragma unroll
    for (int i = 0; i < 16; ++i) sums[t * 16 + i] = sum[i];
    __syncthreads();
    if (rl == 0 && in_k) {
      for (int r = 1; r < kQRows; ++r)
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[i] += sums[(t + r * 8 * kQBlocks) * 16 + i];
      float* d = partials + (int64_t)blockIdx.y * k + col;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(d)[i] = make_float4(sum[4 * i], sum[4 * i + 1], sum[4 * i + 2], sum[4 * i + 3]);
    }
  }
}

// out[j] = sum of n partial rows: 32 columns per workgroup, 32 interleaved row sets added in order.
__global__ void __launch_bounds__(1024) fp8_column_sum_kernel(const float* __restrict__ partials, int n, int64_t k,
                                                              float* __restrict__ out) {
  __shared__ float lds[32][33];
  const int x = threadIdx.x & 31, set = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + x;
  float a = 0.0f;
  if (col < k)
    for (int i = set; i < n; i += 32) a += partials[(int64_t)i * k + col];
  lds[set][x] = a;
  __syncthreads();
  if (set == 0 && col < k) {
#pragma unroll
    for (int i = 1; i < 32; ++i) a += lds[i][x];
    out[col] = a;
  }
}

// A weight's tile of 128 x 128 per workgroup: 32 rows at a time, eight lanes to a row, the
// tile's 64 values a lane in registers between its abs-max and its codes.  With codes_t the
// tile goes through LDS into [k][n] order: rows of 33 words, and eight words more every 16 rows,
// so that the eight lanes that gather one output row's 128 bytes (and the eight output rows of a
// wave) lie in different banks.
constexpr int kTileRow = 33;
__device__ __forceinline__ int tile_word(int row) { return row * kTileRow + (row >> 4) * 8; }

template <bool kWF32, bool kTranspose>
__global__ void __launch_bounds__(kThreads) fp8_quantize_weight_kernel(const void* __restrict__ w, int64_t n, int64_t k,
                                                                       uint8_t* __restrict__ codes,
                                                                       float* __restrict__ scales,
                                                                       uint8_t* __restrict__ codes_t,
                                                                       float* __restrict__ scales_t) {
  __shared__ uint32_t wave_max_bits[kThreads / 64];
  __shared__ uint32_t tile[kTranspose ? 128 * kTileRow + 64 : 1];
  const int t = threadIdx.x;
  const int64_t kb = (k + kFp8Block - 1) / kFp8Block, nb = (n + kFp8Block - 1) / kFp8Block;
  const int64_t tk = blockIdx.x % kb, tn = blockIdx.x / kb;
  const int64_t n0 = tn * kFp8Block, k0 = tk * kFp8Block;
  const int rl = t >> 3;
  const int64_t col = k0 + 16 * (t & 7);
  float v[4][16];
  uint32_t m = 0;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int64_t row = n0 + 32 * p + rl;
    if (row < n && col < k) {
      if constexpr (kWF32) load16_f32(static_cast<const float*>(w) + row * k + col, v[p]);
      else load16_bf16(static_cast<const uint16_t*>(w) + row * k + col, v[p]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[p][i] = 0.0f;
    }
    m = max(m, ck_amax_bits(v[p]));
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
  if ((t & 63) == 0) wave_max_bits[t >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) m = max(m, wave_max_bits[i]);
  float factor;
  const float scale = fp8_scale(m, factor);
  if (t == 0) {
    scales[tn * kb + tk] = scale;
    if constexpr (kTranspose) scales_t[tk * nb + tn] = scale;
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int r = 32 * p + rl;
    const uint4 c = fp8_encode16(v[p], factor);
    if (n0 + r < n && col < k) *reinterpret_cast<uint4*>(codes + (n0 + r) * k + col) = c;
    if constexpr (kTranspose) {
      uint32_t* d = tile + tile_word(r) + 4 * (t & 7);
      d[0] = c.x;
      d[1] = c.y;
      d[2] = c.z;
      d[3] = c.w;
    }
  }
  if constexpr (kTranspose) {
    __syncthreads();
    // lane: rows 16 (t % 8) .. + 15 of the tile, word t / 8 (four columns): four rows by four
    // columns of bytes at a time turned over
    const int r0 = 16 * (t & 7), word = t >> 3;
    uint32_t o[4][4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint32_t a[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) a[q] = tile[tile_word(r0 + 4 * g + q) + word];
      const uint32_t lo01 = __builtin_amdgcn_perm(a[1], a[0], 0x05010400), hi01 = __builtin_amdgcn_perm(a[1], a[0], 0x07030602);
      const uint32_t lo23 = __builtin_amdgcn_perm(a[3], a[2], 0x05010400), hi23 = __builtin_amdgcn_perm(a[3], a[2], 0x07030602);
      o[0][g] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100);
      o[1][g] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302);
      o[2][g] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100);
      o[3][g] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t kr = k0 + 4 * word + i;
      if (kr < k && n0 + r0 < n)
        *reinterpret_cast<uint4*>(codes_t + kr * n + n0 + r0) = make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
    }
  }
}

// Codes back to values fp32(code * scale), 16 per thread.  rows_per_scale 1: scales
// [ceil(k / 128)][rows]; 128: [ceil(rows / 128)][ceil(k / 128)].
template <bool kOutBf16>
__global__ void __launch_bounds__(kThreads) fp8_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                  const float* __restrict__ scales, int64_t rows,
                                                                  int64_t k, bool weight, void* __restrict__ out) {
  const int64_t chunks = k / 16, total = rows * chunks;
  const int64_t kb = (k + kFp8Block - 1) / kFp8Block;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < total; u += (int64_t)gridDim.x * kThreads) {
    const int64_t row = u / chunks, c = u - row * chunks, blk = c >> 3;
    const float s = weight ? scales[(row >> 7) * kb + blk] : scales[blk * rows + row];
    const uint4 q = *reinterpret_cast<const uint4*>(codes + u * 16);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    float v[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
      const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
      v[4 * i] = __fmul_rn(lo[0], s);
      v[4 * i + 1] = __fmul_rn(lo[1], s);
      v[4 * i + 2] = __fmul_rn(hi[0], s);
      v[4 * i + 3] = __fmul_rn(hi[1], s);
    }
    if constexpr (kOutBf16) {
      uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + u * 16);
      d[0] = make_uint4(gemm::pack_bf16x2(v[0], v[1]), gemm::pack_bf16x2(v[2], v[3]), gemm::pack_bf16x2(v[4], v[5]),
                        gemm::pack_bf16x2(v[6], v[7]));
      d[1] = make_uint4(gemm::pack_bf16x2(v[8], v[9]), gemm::pack_bf16x2(v[10], v[11]),
                        gemm::pack_bf16x2(v[12], v[13]), gemm::pack_bf16x2(v[14], v[15]));
    } else {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(out) + u * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
  }
}

int64_t column_groups(int64_t k) { return (k + kQBlocks * kFp8Block - 1) / (kQBlocks * kFp8Block); }

// Row walkers of the form with column sums: about eight workgroups a compute unit over all columns.
int64_t sum_walkers(int64_t rows, int64_t k) {
  const int64_t most = std::max<int64_t>(2048 / column_groups(k), 1);
  return std::min<int64_t>((rows + kQRows - 1) / kQRows, most);
}

}  // namespace

size_t fp8_column_sum_floats(int64_t rows, int64_t k) { return (size_t)sum_walkers(rows, k) * (size_t)k; }

hipError_t launch_fp8_quantize(const uint16_t* x, const uint16_t* up, int64_t rows, int64_t k, uint8_t* codes,
                               float* scales, float* column_sum, float* partials, uint8_t* ck_codes, uint8_t* ck_scales,
                               hipStream_t s) {
  const int64_t groups = column_groups(k);
  if (column_sum != nullptr) {
    const int64_t walkers = sum_walkers(rows, k);
    if (walkers > 0)
      hipLaunchKernelGGL((fp8_quantize_kernel<false, true, false>), dim3((uint32_t)groups, (uint32_t)walkers),
                         dim3(kThreads), 0, s, x, up, rows, k, codes, scales, partials, nullptr, nullptr);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    hipLaunchKernelGGL(fp8_column_sum_kernel, dim3((uint32_t)((k + 31) / 32)), dim3(1024), 0, s, partials, (int)walkers, k,
                       column_sum);
    return hipGetLastError();
  }
  const auto fn = up != nullptr ? fp8_quantize_kernel<true, false, false>
                  : ck_codes != nullptr ? fp8_quantize_kernel<false, false, true>
                                        : fp8_quantize_kernel<false, false, false>;
  const dim3 grid((uint32_t)groups, (uint32_t)std::min<int64_t>((rows + kQRows - 1) / kQRows, 65535));
  hipLaunchKernelGGL(fn, grid, dim3(kThreads), 0, s, x, up, rows, k, codes, scales, partials, ck_codes, ck_scales);
  return hipGetLastError();
}

hipError_t launch_fp8_quantize_weight(const void* w, bool w_f32, int64_t n, int64_t k, uint8_t* codes, float* scales,
                                      uint8_t* codes_t, float* scales_t, hipStream_t s) {
  const int64_t tiles = ((n + kFp8Block - 1) / kFp8Block) * ((k + kFp8Block - 1) / kFp8Block);
  using Fn = void (*)(const void*, int64_t, int64_t, uint8_t*, float*, uint8_t*, float*);
  static constexpr Fn f[2][2] = {{fp8_quantize_weight_kernel<false, false>, fp8_quantize_weight_kernel<false, true>},
                                 {fp8_quantize_weight_kernel<true, false>, fp8_quantize_weight_kernel<true, true>}};
  hipLaunchKernelGGL(f[w_f32 ? 1 : 0][codes_t != nullptr ? 1 : 0], dim3((uint32_t)tiles), dim3(kThreads), 0, s, w, n, k,
                     codes, scales, codes_t, scales_t);
  return hipGetLastError();
}

hipError_t launch_fp8_dequantize(const uint8_t* codes, const float* scales, int64_t rows, int64_t k, bool weight,
                                 void* out, bool out_bf16, hipStream_t s) {
  const int64_t chunks = rows * (k / 16);
  const dim3 grid((uint32_t)std::min<int64_t>((chunks + kThreads - 1) / kThreads, 1 << 20));
  if (out_bf16)
    hipLaunchKernelGGL(fp8_dequantize_kernel<true>, grid, dim3(kThreads), 0, s, codes, scales, rows, k, weight, out);
  else
    hipLaunchKernelGGL(fp8_dequantize_kernel<false>, grid, dim3(kThreads), 0, s, codes, scales, rows, k, weight, out);
  return hipGetLastError();
}

}  // namespace nvfp4
