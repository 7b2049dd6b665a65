// RMS norm with the residual's addition, on gfx950: its output as bf16 (with or without an
// 8-bit checkpoint) or as NVFP4 codes and scales for the linear, and its gradient.
//
//   r = x + residual                      (rounded to the stream's type, stored)
//   s = fp32(1 / sqrt(sum(r^2) / K + eps))
//   y = bf16(fp32(fp32(r * s) * w))
//
// The squares of bf16 and fp32 values are exact in fp64, and their sum is off by far less than
// fp32's spacing.  Every output form adds a row in the same order, which row_shape fixes for
// its K, so s has the same bits in all of them and the codes of y are the quantizer's bit for
// bit.  (Another order would give the same s too, but where the value lies within the sum's
// error of a rounding border of fp32.)  The fp64 additions (one per value) stay hidden under
// the HBM traffic that bounds every form.
//
// A lane owns 16 consecutive values (one NVFP4 block, half a checkpoint block).  Rows of
// at most 1024 values take a power-of-two group of lanes inside a wave, several rows per
// workgroup; longer rows (to 16384) take a workgroup of their own with one chunk per lane.
// Either way the row stays in registers between its sum and its output: one read, one write
// (4096 x 5120, bf16 x and fp32 residual to y, r and y's checkpoint: 273 MB in 52 us,
// 5.3 TB/s; a plain copy of that size reaches 5.2).  A dynamic scale needs the abs-max of
// all rows before the first code, so its many-row form reads r again in a second pass
// (4096 x 5120 in bf16: 126 MB in 25 us, then 58 MB in 14.5).  One row is one workgroup
// and one launch (5120 values: 4.2 us, the launch and two dependent memory accesses).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <numeric>

#include "checkpoint_device.h"
#include "nvfp4_device.h"
#include "nvfp4_launch.h"
#include "quantize_device.h"

namespace nvfp4 {
namespace {

constexpr int kGroupThreads = 256;   // workgroup of the several-rows form

// Lanes per row and threads per workgroup for rows of k values.
struct RowShape {
  int lanes, threads;
};
RowShape row_shape(int64_t k) {
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

// kRes: no residual, one in bf16, one in fp32 (the stream's type is the residual's, or
// x's without one).  What becomes of y is a.mode: bf16 with an optional checkpoint,
// codes under a static scale, codes of a single row under its own dynamic scale, or
// (first pass of a dynamic scale over many rows) only s and the abs-max of y.
template <bool kXF32, int kRes, bool kWF32>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormForward a) {
  constexpr bool kSF32 = kRes == 0 ? kXF32 : kRes == 2;
  __shared__ double part[16];
  __shared__ float pmax[16];
  const int t = threadIdx.x;
  const int rows_here = blockDim.x / a.lanes;
  const int sub = rows_here == 1 ? 0 : t / a.lanes;
  const int c = t - sub * a.lanes;
  const int64_t k = a.k;
  const bool in_k = c < k / kBlock;
  Raw16<kWF32> w;
  if (in_k) w.load(a.w, (int64_t)c * kBlock);
  else w.zero();
  const float gsf_static = a.mode == kNormStatic ? *a.gsf : 0.0f;
  if (a.mode == kNormStatic && a.gsf_out != nullptr && blockIdx.x == 0 && t == 0) *a.gsf_out = gsf_static;
  float mx = 0.0f;

  for (int64_t row0 = (int64_t)blockIdx.x * rows_here; row0 < a.rows; row0 += (int64_t)gridDim.x * rows_here) {
    const int64_t row = row0 + sub;
    const bool valid = row < a.rows && in_k;
    const int64_t off = row * k + (int64_t)c * kBlock;
    float v[16];
    if (valid) {
      load_stream16<kXF32>(a.x, off, v);
      if constexpr (kRes != 0) {
        float q[16];
        load_stream16<kRes == 2>(a.residual, off, q);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __fadd_rn(v[i], q[i]);
        if constexpr (!kSF32) round_bf16(v);
        store_stream16<kSF32>(a.r, off, v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    }
    double ss = group_sum(sum_squares(v), a.lanes < 64 ? a.lanes : 64);
    if (a.lanes > 64) {
      if ((t & 63) == 0) part[t >> 6] = ss;
      __syncthreads();
      ss = 0.0;
      for (int i = 0; i < (int)(blockDim.x >> 6); ++i) ss += part[i];
      __syncthreads();
    }
    const float s = row_scale(ss, k, a.eps);
    normalize16<kWF32>(v, s, w);

    if (a.mode == kNormOut) {
      if (valid) store16_bf16(a.y + off, v);
      if (a.codes != nullptr) {
        uint32_t sb;
        const uint4 code = ck_pack16(v, sb);
        if (valid) {
          *reinterpret_cast<uint4*>(a.codes + off) = code;
          if ((c & 1) == 0) a.scales[row * ((k + kCkBlock - 1) / kCkBlock) + (c >> 1)] = (uint8_t)sb;
        }
      }
      continue;
    }
    float gsf = gsf_static;
    if (a.mode != kNormStatic) {
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, fabsf(v[i]));
      if (a.mode == kNormStats) {
        if (c == 0 && row < a.rows) a.rstd[row] = s;
        continue;
      }
      // the one row: its abs-max over the workgroup (rows beyond it are zeros)
      mx = wave_max(mx);
      if ((t & 63) == 0) pmax[t >> 6] = mx;
      __syncthreads();
      for (int i = 0; i < (int)(blockDim.x >> 6); ++i) mx = fmaxf(mx, pmax[i]);
      gsf = global_scale_from_amax(mx);
      if (t == 0 && a.gsf_out != nullptr) *a.gsf_out = gsf;
    }
    // lanes past the row's last 128-wide tile hold no unit of this row
    const int64_t urow = c < (k + kScaleTileK - 1) / kScaleTileK * 8 ? row : a.rows;
    quantize_unit<false>(v, urow, c >> 3, c & 7, a.rows, k, 0, 1.0f, gsf, a.codes, a.scales, nullptr);
  }
  if (a.mode == kNormStats) {
    mx = wave_max(mx);
    if ((t & 63) == 0) pmax[t >> 6] = mx;
    __syncthreads();
    if (t == 0) {
      for (int i = 1; i < (int)(blockDim.x >> 6); ++i) mx = fmaxf(mx, pmax[i]);
      a.partials[blockIdx.x] = mx;
    }
  }
}

// Second pass of a dynamic scale: y again from r and s (r is in the memory-side cache, and
// storing y in the first pass would cost more than forming it twice), then its codes.
// Eight lanes own a 128-wide tile of a row, as in the quantizer's own pass; the grid is a
// whole number of rows wide (quantize_blocks), so a lane keeps its tile of the weight and
// walks down the rows, the next row's load in flight (4096 x 5120: 14.5 us; 1, 2 or 4 tiles
// in flight per lane without the fixed column 15.1-17.7).
constexpr int kQThreads = 256;
template <bool kSF32, bool kWF32>
__global__ void __launch_bounds__(kQThreads) rmsnorm_quantize_kernel(const NormForward a, int n_partials) {
  __shared__ float lds[kQThreads / 64];
  float m = 0.0f;
  for (int i = threadIdx.x; i < n_partials; i += kQThreads) m = fmaxf(m, a.partials[i]);
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQThreads / 64; ++i) m = fmaxf(m, lds[i]);
  const float gsf = global_scale_from_amax(m);
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.gsf_out != nullptr) *a.gsf_out = gsf;

  const int kt_count = (int)((a.k + kScaleTileK - 1) / kScaleTileK);
  const int j = threadIdx.x & 7;
  const uint32_t unit = blockIdx.x * (kQThreads / 8) + (threadIdx.x >> 3);
  const int kt = (int)(unit % (uint32_t)kt_count);
  const int64_t stride = gridDim.x * (kQThreads / 8) / (uint32_t)kt_count;   // rows
  const int64_t first = unit / (uint32_t)kt_count;
  const int blk = kt * 8 + j;
  const bool in_k = blk < a.k / kBlock;
  const void* r = a.r != nullptr ? a.r : a.x;
  Raw16<kWF32> w;
  if (in_k) w.load(a.w, (int64_t)blk * kBlock);
  else w.zero();
  Raw16<kSF32> cur;
  float s = 0.0f;
  auto fetch = [&](int64_t row) {
    if (row < a.rows && in_k) {
      cur.load(r, row * a.k + (int64_t)blk * kBlock);
      s = a.rstd[row];
    } else {
      cur.zero();
      s = 0.0f;
    }
  };
  fetch(first);
  // the wave loops while any of its rows is left: quantize_unit shuffles across its lanes
  for (int64_t row = first; __any(row < a.rows); row += stride) {
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = cur.get(i);
    const float sr = s;
    fetch(row + stride);
    normalize16<kWF32>(y, sr, w);
    quantize_unit<false>(y, row, kt, j, a.rows, a.k, 0, 1.0f, gsf, a.codes, a.scales, nullptr);
  }
}

// Gradient.  With n = r s, g = gy w and d = sum(g r) over the row:
//   grad_r = s g - r (s^3 d / K) + grad_residual,   grad_w = sum over rows of gy n
// (the rounding of y taken as the identity).  s^2 leaves fp32's range from row magnitudes of
// 1e19 up (and d, summed over a row, long before r does) while s^2 d is of the order of s g:
// a lane sums its 16 products in fp32, the row's sum is fp64, and s multiplies its mean twice
// (4096 x 5120 and 16384 x 1040 take the same time as with all of it in fp32; with the
// products in fp64 too, 3 and 5 % more).
//
// Each workgroup walks its rows with its lanes' 16 columns of grad_w in registers and writes
// one partial row of them; rmsnorm_weight_grad_kernel adds the partials in a fixed order.
// The bound of 1024 threads
// also holds every variant to 128 registers, four waves per SIMD, whose loads cover each
// other's: fetching the next row ahead spilled, and cost more than it hid (4096 x 5120, both
// kernels: bf16 stream 39 us ahead, 36 so, of which this one 31.7, 5.3 TB/s; fp32 stream 97
// and 49, 6.0 TB/s).
template <bool kSF32, bool kWF32, bool kRes>
__global__ void __launch_bounds__(1024) rmsnorm_backward_kernel(const NormBackward a) {
  __shared__ double part_ss[2][16], part_d[2][16];
  __shared__ float colsum[kGroupThreads * 16];
  const int t = threadIdx.x;
  const int rows_here = blockDim.x / a.lanes;
  const int sub = rows_here == 1 ? 0 : t / a.lanes;
  const int c = t - sub * a.lanes;
  const int64_t k = a.k;
  const bool in_k = c < k / kBlock;
  Raw16<kWF32> w;
  if (in_k) w.load(a.w, (int64_t)c * kBlock);
  else w.zero();
  float gw[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) gw[i] = 0.0f;

  const int64_t stride = (int64_t)gridDim.x * rows_here;
  const double inv_k = 1.0 / (double)k;
  int parity = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * rows_here; row0 < a.rows; row0 += stride, parity ^= 1) {
    const int64_t row = row0 + sub;
    const int64_t off = row * k + (int64_t)c * kBlock;
    const bool valid = row < a.rows && in_k;
    Raw16<kSF32> rr, gres;
    Raw16<false> gy;
    if (valid) {
      rr.load(a.r, off);
      gy.load(a.gy, off);
      if constexpr (kRes) gres.load(a.grad_residual, off);
    } else {
      rr.zero();
      gy.zero();
      if constexpr (kRes) gres.zero();
    }
    float r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = rr.get(i);
    double ss = sum_squares(r);
    float dl = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) dl = fmaf(gy.get(i) * w.get(i), r[i], dl);
    double d = (double)dl;
    const int lanes = a.lanes < 64 ? a.lanes : 64;
    ss = group_sum(ss, lanes);
    d = group_sum(d, lanes);
    if (a.lanes > 64) {
      // the other parity's slots may still be read by slower waves; these are free
      if ((t & 63) == 0) {
        part_ss[parity][t >> 6] = ss;
        part_d[parity][t >> 6] = d;
      }
      __syncthreads();
      ss = 0.0;
      d = 0.0;
      for (int i = 0; i < (int)(blockDim.x >> 6); ++i) {
        ss += part_ss[parity][i];
        d += part_d[parity][i];
      }
    }
    // 0 for the rows a workgroup has beyond the last: with eps = 0 theirs would be infinite, and
    // their part of grad_w (0 times it) NaN
    const float s = row < a.rows ? row_scale(ss, k, a.eps) : 0.0f;
    const float f = s * (s * (float)(d * inv_k));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float n = r[i] * s, g = gy.get(i);
      gw[i] = fmaf(g, n, gw[i]);
      const float x = fmaf(s, g * w.get(i), -(n * f));
      r[i] = kRes ? x + gres.get(i) : x;
    }
    if (valid) {
      if constexpr (!kSF32) round_bf16(r);
      store_stream16<kSF32>(a.grad_r, off, r);
    }
  }
  if (a.grad_w == nullptr) return;
  if (rows_here == 1) {
    if (in_k) store_stream16<true>(a.partials, (int64_t)blockIdx.x * k + (int64_t)c * kBlock, gw);
    return;
  }
  // the workgroup's rows side by side in LDS, added in row order
#pragma unroll
  for (int i = 0; i < 16; ++i) colsum[t * 16 + i] = gw[i];
  __syncthreads();
  if (sub == 0 && in_k) {
    for (int s = 1; s < rows_here; ++s)
#pragma unroll
      for (int i = 0; i < 16; ++i) gw[i] += colsum[(s * a.lanes + c) * 16 + i];
    store_stream16<true>(a.partials, (int64_t)blockIdx.x * k + (int64_t)c * kBlock, gw);
  }
}

// grad_w[j] = sum of n partial rows: 32 columns per workgroup, 32 interleaved row sets
// added in order.
__global__ void __launch_bounds__(1024) rmsnorm_weight_grad_kernel(const float* __restrict__ partials, int n,
                                                                   int64_t k, float* __restrict__ grad_w) {
  __shared__ float lds[32][33];
  const int x = threadIdx.x & 31, set = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + x;
  float a = 0.0f;
  if (col < k) {
#pragma unroll 8
    for (int i = set; i < n; i += 32) a += partials[(int64_t)i * k + col];
  }
  lds[set][x] = a;
  __syncthreads();
  if (set == 0 && col < k) {
#pragma unroll
    for (int i = 1; i < 32; ++i) a += lds[i][x];
    grad_w[col] = a;
  }
}

using ForwardFn = void (*)(const NormForward);

ForwardFn forward_kernel(const NormForward& a) {
  const int w = a.w_f32 ? 1 : 0;
  if (a.residual == nullptr) {
    static constexpr ForwardFn f[2][2] = {{rmsnorm_kernel<false, 0, false>, rmsnorm_kernel<false, 0, true>},
                                          {rmsnorm_kernel<true, 0, false>, rmsnorm_kernel<true, 0, true>}};
    return f[a.x_f32 ? 1 : 0][w];
  }
  static constexpr ForwardFn f[3][2] = {{rmsnorm_kernel<false, 1, false>, rmsnorm_kernel<false, 1, true>},
                                        {rmsnorm_kernel<false, 2, false>, rmsnorm_kernel<false, 2, true>},
                                        {rmsnorm_kernel<true, 2, false>, rmsnorm_kernel<true, 2, true>}};
  return f[!a.stream_f32 ? 0 : !a.x_f32 ? 1 : 2][w];
}

// Workgroups of the row-walking kernels, whose results are joined afterwards: two for each
// compute unit where they have four waves or more, about ten waves a unit where fewer.
// Gradient, both kernels: 4096 x 5120 (five waves) with 256 / 512 / 768 workgroups 48 / 36 /
// 44 us, 16384 x 1040 (two waves) with 512 / 1024 / 1280 75 / 44 / 41.  Statistics and second
// pass of the dynamic scale: 4096 x 5120 with 256 / 512 / 768 / 1024 48.9 / 39.4 / 39.7 / 41.1,
// 16384 x 5120 201 / 149 / 150 / 165, 16384 x 1040 with 512 / 1280 71 / 45.
int64_t walking_blocks(int64_t rows, const RowShape& s) {
  const int64_t per = s.threads / s.lanes;
  const int64_t most = s.threads >= 256 ? 512 : 2560 * 64 / s.threads;
  static_assert(2560 * 64 / 128 <= kNormPartials, "rows longer than 1024 take two waves at least");
  return std::min<int64_t>((rows + per - 1) / per, most);
}

// Second-pass workgroups: a whole number of rows' tiles (at most 128) between a lane's
// units, so that its tile of the weight stays the same.
int64_t quantize_blocks(int64_t rows, int64_t k) {
  const int64_t kt = (k + kScaleTileK - 1) / kScaleTileK;
  const int64_t want = std::min<int64_t>((rows * kt + kQThreads / 8 - 1) / (kQThreads / 8), 2048);
  const int64_t unit = kt / std::gcd(kt, (int64_t)(kQThreads / 8));
  return std::max<int64_t>(want / unit, 1) * unit;
}

}  // namespace

hipError_t launch_rmsnorm(NormForward a, hipStream_t s) {
  const RowShape shape = row_shape(a.k);
  a.lanes = shape.lanes;
  const int64_t per = shape.threads / shape.lanes;
  int64_t blocks = std::min<int64_t>((a.rows + per - 1) / per, 1 << 20);   // the rest by the row loop
  if (a.mode == kNormDynamic) {
    // one row needs no second pass: its workgroup knows the whole abs-max
    a.mode = a.rows == 1 ? kNormOneRow : kNormStats;
    blocks = walking_blocks(a.rows, shape);
  }
  hipLaunchKernelGGL(forward_kernel(a), dim3((uint32_t)blocks), dim3((uint32_t)shape.threads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.mode != kNormStats) return e;
  using QuantFn = void (*)(const NormForward, int);
  static constexpr QuantFn q[2][2] = {{rmsnorm_quantize_kernel<false, false>, rmsnorm_quantize_kernel<false, true>},
                                      {rmsnorm_quantize_kernel<true, false>, rmsnorm_quantize_kernel<true, true>}};
  const int64_t grid = quantize_blocks(a.rows, a.k);
  const bool sf32 = a.residual != nullptr ? a.stream_f32 : a.x_f32;
  hipLaunchKernelGGL(q[sf32 ? 1 : 0][a.w_f32 ? 1 : 0], dim3((uint32_t)grid), dim3(kQThreads), 0, s, a, (int)blocks);
  return hipGetLastError();
}

size_t rmsnorm_backward_partial_floats(int64_t rows, int64_t k) {
  return (size_t)walking_blocks(rows, row_shape(k)) * (size_t)k;
}

hipError_t launch_rmsnorm_backward(NormBackward a, hipStream_t s) {
  const RowShape shape = row_shape(a.k);
  a.lanes = shape.lanes;
  const int64_t blocks = walking_blocks(a.rows, shape);
  using Fn = void (*)(const NormBackward);
  static constexpr Fn f[2][2][2] = {
      {{rmsnorm_backward_kernel<false, false, false>, rmsnorm_backward_kernel<false, false, true>},
       {rmsnorm_backward_kernel<false, true, false>, rmsnorm_backward_kernel<false, true, true>}},
      {{rmsnorm_backward_kernel<true, false, false>, rmsnorm_backward_kernel<true, false, true>},
       {rmsnorm_backward_kernel<true, true, false>, rmsnorm_backward_kernel<true, true, true>}}};
  if (blocks > 0)
    hipLaunchKernelGGL(f[a.stream_f32 ? 1 : 0][a.w_f32 ? 1 : 0][a.grad_residual != nullptr ? 1 : 0],
                       dim3((uint32_t)blocks), dim3((uint32_t)shape.threads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.grad_w == nullptr) return e;
  hipLaunchKernelGGL(rmsnorm_weight_grad_kernel, dim3((uint32_t)((a.k + 31) / 32)), dim3(1024), 0, s, a.partials,
                     (int)blocks, a.k, a.grad_w);
  return hipGetLastError();
}

}  // namespace nvfp4
