// Layer norm with the residual's addition, on gfx950: its output as bf16 (with or without an
// 8-bit checkpoint), as 8-bit block codes or as NVFP4 codes, and its gradient; and the RMS
// norm's output as 8-bit block codes.
//
//   r = x + residual                      (rounded to the stream's type, stored)
//   mu = mean(r),  s = fp32(1 / sqrt(mean((r - mu)^2) + eps))
//   y = bf16(fp32(fp32(fp32(r - mu) * s) * w) + b)
//
// Mean and variance come from one pass over the row, which stays in registers: with the
// row's first value p as a pivot, S1 = sum(r - p) and S2 = sum((r - p)^2) in fp64 give
// mu = p + S1 / K and the variance S2 / K - (S1 / K)^2.  p is one of the K values, so
// (p - mu)^2 is at most K times the variance: the subtraction costs 14 of fp64's 53 bits at
// most, where sums without a pivot lose as many bits as the mean is larger than the spread.
//
// The layout is the RMS norm's (norm_device.h): a lane owns 16 consecutive values, a row a
// power-of-two group of lanes or a workgroup of its own; one read, one write.
//
// All of it is bound by HBM traffic.  4096 x 5120 with a bf16 residual and fp32 weights, each call
// on other tensors (a 1 GiB copy reaches 5.06 TB/s): bf16 y and r 37.3 us, 4.5 TB/s; 8-bit codes and
// r 40.2 us, 3.7 TB/s (RMS norm 33.1); with the checkpoint 43.9 us, 4.3 TB/s.  One row: 4.3 us,
// a launch and its one read.
// (Neighbouring rows kept on one XCD, so that the block-major scales of 16 rows meet in its L2, give
// 2 % on 4096 x 5120 to 8-bit codes and take 9 % at 16384 x 1024: rows go out in launch order.)
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "checkpoint_device.h"
#include "fp8_device.h"
#include "norm_device.h"
#include "nvfp4_device.h"
#include "nvfp4_launch.h"
#include "quantize_device.h"

namespace nvfp4 {
namespace {

// Value i of a row's stream, rounded as it is stored.
template <bool kXF32, int kRes>
__device__ __forceinline__ float stream_value(const void* x, const void* residual, int64_t i) {
  float v = kXF32 ? static_cast<const float*>(x)[i] : bf16_to_f32(static_cast<const uint16_t*>(x)[i]);
  if constexpr (kRes == 1)
    v = bf16_to_f32(gemm::pack_bf16x2(__fadd_rn(v, bf16_to_f32(static_cast<const uint16_t*>(residual)[i])), 0.0f) & 0xFFFFu);
  if constexpr (kRes == 2) v = __fadd_rn(v, static_cast<const float*>(residual)[i]);
  return v;
}

// Four values at a time: the scheduler would convert all 16 to fp64 at once (32 registers more).
__device__ __forceinline__ void by_four(int i) {
  if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);
}

// Sums of d = v - p and d^2 over a lane's 16 values.
__device__ __forceinline__ void pivot_sums(const float (&v)[16], float p, double& s1, double& s2) {
  double a1 = 0.0, b1 = 0.0, a2 = 0.0, b2 = 0.0;
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const double d = (double)v[i] - (double)p, e = (double)v[i + 1] - (double)p;
    a1 += d;
    b1 += e;
    a2 = fma(d, d, a2);
    b2 = fma(e, e, b2);
    by_four(i + 1);
  }
  s1 = a1 + b1;
  s2 = a2 + b2;
}

// Ends what the compiler knows of v: it would keep its 16 fp64 conversions (32 registers) from the
// sums to the output, which spills; converting again costs less.
__device__ __forceinline__ void forget(float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) asm("" : "+v"(v[i]));
}

template <bool kF32>
__device__ __forceinline__ void forget(Raw16<kF32>& v) {
#pragma unroll
  for (int i = 0; i < (kF32 ? 4 : 2); ++i) asm("" : "+v"(v.raw[i].x), "+v"(v.raw[i].y), "+v"(v.raw[i].z), "+v"(v.raw[i].w));
}

// Sum over the `lanes` lanes of a row (a power of two from 8 to 64), the same bits in each: by the
// vector unit's own lane moves, where shuffles through LDS (two for each fp64 step) cost the
// gradient's four sums more than its memory traffic.
template <int kCtrl>
__device__ __forceinline__ double lane_move(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, kCtrl, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), kCtrl, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <bool k32>
__device__ __forceinline__ double swap_sum(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t l = (uint32_t)u, h = (uint32_t)(u >> 32);
  const auto lo = k32 ? __builtin_amdgcn_permlane32_swap(l, l, false, false) : __builtin_amdgcn_permlane16_swap(l, l, false, false);
  const auto hi = k32 ? __builtin_amdgcn_permlane32_swap(h, h, false, false) : __builtin_amdgcn_permlane16_swap(h, h, false, false);
  return __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]) + __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
}
__device__ __forceinline__ double lanes_sum(double v, int lanes) {
  v += lane_move<0xB1>(v);                     // lane ^ 1
  v += lane_move<0x4E>(v);                     // lane ^ 2
  v += lane_move<0x141>(v);                    // 7 - lane of eight: the other four
  if (lanes >= 16) v += lane_move<0x140>(v);   // 15 - lane of 16: the other eight
  if (lanes >= 32) v = swap_sum<false>(v);
  if (lanes >= 64) v = swap_sum<true>(v);
  return v;
}

// Mean and scale from the row's sums.  The variance's last bits may fall below zero; NaN stays.
__device__ __forceinline__ float row_statistics(double s1, double s2, float p, int64_t k, double eps, double& mu) {
  const double m = s1 / (double)k;
  double var = s2 / (double)k - m * m;
  var = var < 0.0 ? 0.0 : var;
  mu = (double)p + m;
  return (float)(1.0 / sqrt(var + eps));
}

// y = bf16(fp32(fp32(fp32(r - mu) * s) * w) + b), over r.
template <bool kWF32>
__device__ __forceinline__ void layernorm16(float (&v)[16], double mu, float s, const Raw16<kWF32>& w,
                                            const Raw16<kWF32>& b, bool has_bias) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = __fmul_rn(__fmul_rn((float)((double)v[i] - mu), s), w.get(i));
    by_four(i);
  }
  if (has_bias) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __fadd_rn(v[i], b.get(i));
  }
  round_bf16(v);
}

// kRes: no residual, one in bf16, one in fp32 (the stream's type is the residual's, or x's
// without one).  kMean: the layer norm; otherwise the RMS norm, whose row sum is added as in
// norm.hip, so that its y has the same bits.  What becomes of y is kMode: bf16 with an optional
// checkpoint, 8-bit block codes, NVFP4 codes under a static scale, those of a single row under
// its own dynamic scale, or (first pass of a dynamic scale over many rows) only the statistics
// and the abs-max of y.
template <bool kXF32, int kRes, bool kWF32, bool kMean, int kMode>
__global__ void __launch_bounds__(1024) layernorm_kernel(const NormForward a) {
  constexpr bool kSF32 = kRes == 0 ? kXF32 : kRes == 2;
  __shared__ double part[2][16];
  __shared__ float pmax[16];
  const int t = threadIdx.x;
  const int rows_here = blockDim.x / a.lanes;
  const int sub = rows_here == 1 ? 0 : t / a.lanes;
  const int c = t - sub * a.lanes;
  const int64_t k = a.k;
  const bool in_k = c < k / kBlock;
  const bool has_bias = kMean && a.b != nullptr;
  Raw16<kWF32> w, b;
  if (in_k) w.load(a.w, (int64_t)c * kBlock);
  else w.zero();
  if (in_k && has_bias) b.load(a.b, (int64_t)c * kBlock);
  else b.zero();
  const float gsf_static = kMode == kNormStatic ? *a.gsf : 0.0f;
  if (kMode == kNormStatic && a.gsf_out != nullptr && blockIdx.x == 0 && t == 0) *a.gsf_out = gsf_static;
  float mx = 0.0f;

  for (int64_t row0 = (int64_t)blockIdx.x * rows_here; row0 < a.rows; row0 += (int64_t)gridDim.x * rows_here) {
    const int64_t row = row0 + sub;
    const bool valid = row < a.rows && in_k;
    const int64_t off = row * k + (int64_t)c * kBlock;
    float v[16];
    float p = 0.0f;
    if (valid) {
      load_stream16<kXF32>(a.x, off, v);
      if constexpr (kRes != 0) {
        float q[16];
        load_stream16<kRes == 2>(a.residual, off, q);
        // the pivot before r is written: r may be the residual or x
        if constexpr (kMean) p = stream_value<kXF32, kRes>(a.x, a.residual, row * k);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __fadd_rn(v[i], q[i]);
        if constexpr (!kSF32) round_bf16(v);
      } else if constexpr (kMean) {
        p = stream_value<kXF32, kRes>(a.x, nullptr, row * k);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    }
    const int lanes = a.lanes < 64 ? a.lanes : 64;
    double s1 = 0.0, s2;
    if constexpr (kMean) pivot_sums(v, p, s1, s2);   // lanes without values: all zero
    else s2 = sum_squares(v);
    if constexpr (kMean) {
      s1 = lanes_sum(s1, lanes);
      s2 = lanes_sum(s2, lanes);
    } else {
      s2 = group_sum(s2, lanes);
    }
    if (a.lanes > 64) {
      if ((t & 63) == 0) {
        part[0][t >> 6] = s1;
        part[1][t >> 6] = s2;
      }
      __syncthreads();
      s1 = 0.0;
      s2 = 0.0;
      for (int i = 0; i < (int)(blockDim.x >> 6); ++i) {
        if constexpr (kMean) s1 += part[0][i];
        s2 += part[1][i];
      }
      __syncthreads();
    }
    // behind the barrier (or, inside a wave, behind the sums): every lane of the row has its pivot
    if constexpr (kRes != 0)
      if (valid) store_stream16<kSF32>(a.r, off, v);
    float s;
    double mu = 0.0;
    forget(v);
    if constexpr (kMean) {
      s = row_statistics(s1, s2, p, k, a.eps, mu);
      layernorm16<kWF32>(v, mu, s, w, b, has_bias);
      if (!valid) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.0f;
      }
    } else {
      s = row_scale(s2, k, a.eps);
      normalize16<kWF32>(v, s, w);
    }

    if constexpr (kMode == kNormFp8) {
      float scale;
      const uint4 code = fp8_block16(v, scale);
      if (valid) {
        *reinterpret_cast<uint4*>(a.codes + off) = code;
        if ((c & 7) == 0) a.block_scales[(int64_t)(c >> 3) * a.rows + row] = scale;
      }
    } else if constexpr (kMode == kNormOut) {
      if (valid) store16_bf16(a.y + off, v);
      if (a.codes != nullptr) {
        uint32_t sb;
        const uint4 code = ck_pack16(v, sb);
        if (valid) {
          *reinterpret_cast<uint4*>(a.codes + off) = code;
          if ((c & 1) == 0) a.scales[row * ((k + kCkBlock - 1) / kCkBlock) + (c >> 1)] = (uint8_t)sb;
        }
      }
    } else if constexpr (kMode == kNormStats) {
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, fabsf(v[i]));
      if (c == 0 && row < a.rows) {
        a.rstd[row] = s;
        a.mean[row] = mu;
      }
    } else {
      float gsf = gsf_static;
      if constexpr (kMode == kNormOneRow) {
        // the one row: its abs-max over the workgroup (rows beyond it are zeros)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, fabsf(v[i]));
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
  }
  if constexpr (kMode == kNormStats) {
    mx = wave_max(mx);
    if ((t & 63) == 0) pmax[t >> 6] = mx;
    __syncthreads();
    if (t == 0) {
      for (int i = 1; i < (int)(blockDim.x >> 6); ++i) mx = fmaxf(mx, pmax[i]);
      a.partials[blockIdx.x] = mx;
    }
  }
}

// Second pass of a dynamic scale: y again from r and the row's statistics, then its codes, as
// the RMS norm's second pass does (norm.hip).  4096 x 5120: 16.9 us (3.2 TB/s), after 31.4 us of the
// pass that writes r and the statistics (4.0 TB/s).
template <bool kSF32, bool kWF32>
__global__ void __launch_bounds__(kNormQThreads) layernorm_quantize_kernel(const NormForward a, int n_partials) {
  __shared__ float lds[kNormQThreads / 64];
  float m = 0.0f;
  for (int i = threadIdx.x; i < n_partials; i += kNormQThreads) m = fmaxf(m, a.partials[i]);
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kNormQThreads / 64; ++i) m = fmaxf(m, lds[i]);
  const float gsf = global_scale_from_amax(m);
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.gsf_out != nullptr) *a.gsf_out = gsf;

  const int kt_count = (int)((a.k + kScaleTileK - 1) / kScaleTileK);
  const int j = threadIdx.x & 7;
  const uint32_t unit = blockIdx.x * (kNormQThreads / 8) + (threadIdx.x >> 3);
  const int kt = (int)(unit % (uint32_t)kt_count);
  const int64_t stride = gridDim.x * (kNormQThreads / 8) / (uint32_t)kt_count;   // rows
  const int64_t first = unit / (uint32_t)kt_count;
  const int blk = kt * 8 + j;
  const bool in_k = blk < a.k / kBlock;
  const bool has_bias = a.b != nullptr;
  const void* r = a.r != nullptr ? a.r : a.x;
  Raw16<kWF32> w, b;
  if (in_k) w.load(a.w, (int64_t)blk * kBlock);
  else w.zero();
  if (in_k && has_bias) b.load(a.b, (int64_t)blk * kBlock);
  else b.zero();
  Raw16<kSF32> cur;
  float s = 0.0f;
  double mu = 0.0;
  auto fetch = [&](int64_t row) {
    if (row < a.rows && in_k) {
      cur.load(r, row * a.k + (int64_t)blk * kBlock);
      s = a.rstd[row];
      mu = a.mean[row];
    } else {
      cur.zero();
      s = 0.0f;
      mu = 0.0;
    }
  };
  fetch(first);
  // the wave loops while any of its rows is left: quantize_unit shuffles across its lanes
  for (int64_t row = first; __any(row < a.rows); row += stride) {
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = cur.get(i);
    const float sr = s;
    const double mr = mu;
    fetch(row + stride);
    layernorm16<kWF32>(y, mr, sr, w, b, has_bias);
    quantize_unit<false>(y, row, kt, j, a.rows, a.k, 0, 1.0f, gsf, a.codes, a.scales, nullptr);
  }
}

// Gradient.  With n = (r - mu) s and g = gy w:
//   grad_r = s (g - mean(g) - n mean(g n)) + grad_residual,
//   grad_w = sum over rows of gy n,   grad_b = sum over rows of gy
// (the rounding of y taken as the identity).  One reduction gives all four row sums, in fp64: those
// of the pivot's distances d = r - p and of d^2, and sum(g), sum(g d) of the products g rounded to
// fp32: mean(g n) = s (sum(g d) - (mu - p) sum(g)) / K.  g d leaves fp32's range long before the
// gradient does: |d| may be twice the largest |r|, and meets the gradients beside small r too.
//
// Each workgroup walks its rows with its lanes' 16 columns of grad_w and grad_b in registers and
// writes one partial row of both; layernorm_weight_grad_kernel adds the partials in a fixed order.
//
// 16384 x 1024 in bf16 28.2 us (4.8 TB/s), 4091 x 5120 with an fp32 stream 64.8 us (4.5 TB/s), and
// 4.0 and 5.5 us for the partials' sums.  Shuffles through LDS in place of lane moves: 61 and 142 us.
// (Eight values a lane, in half the registers, take twice the waves per row and as many sums for
// half the work: with shuffles still, 16384 x 1024 61 us against 45, 4091 x 5120 in fp32 93 against 75.)
template <bool kSF32, bool kWF32, bool kRes>
__global__ void __launch_bounds__(1024) layernorm_backward_kernel(const NormBackward a) {
  __shared__ double part[2][4][16];
  __shared__ float colsum[kGroupThreads * 16];
  const int t = threadIdx.x;
  const int rows_here = blockDim.x / a.lanes;
  const int sub = rows_here == 1 ? 0 : t / a.lanes;
  const int c = t - sub * a.lanes;
  const int64_t k = a.k;
  const bool in_k = c < k / kBlock;
  Raw16<kWF32> w;
  w.zero();
  if (in_k) w.load(a.w, (int64_t)c * kBlock);
  float gw[16], gb[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) gw[i] = gb[i] = 0.0f;

  const int64_t stride = (int64_t)gridDim.x * rows_here;
  const double inv_k = 1.0 / (double)k;
  int parity = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * rows_here; row0 < a.rows; row0 += stride, parity ^= 1) {
    const int64_t row = row0 + sub;
    const int64_t off = row * k + (int64_t)c * kBlock;
    const bool valid = row < a.rows && in_k;
    Raw16<kSF32> rr, gres;
    Raw16<false> gy;
    float p = 0.0f;
    double sum[4] = {0.0, 0.0, 0.0, 0.0};
    if (valid) {
      rr.load(a.r, off);
      p = stream_value<kSF32, 0>(a.r, nullptr, row * k);
      gy.load(a.gy, off);
      if constexpr (kRes) gres.load(a.grad_residual, off);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const double d = (double)rr.get(i) - (double)p, g = (double)(gy.get(i) * w.get(i));
        sum[0] += d;
        sum[1] = fma(d, d, sum[1]);
        sum[2] += g;
        sum[3] = fma(g, d, sum[3]);
        by_four(i);
      }
    }
    const int lanes = a.lanes < 64 ? a.lanes : 64;
#pragma unroll
    for (int q = 0; q < 4; ++q) sum[q] = lanes_sum(sum[q], lanes);
    if (a.lanes > 64) {
      // the other parity's slots may still be read by slower waves; these are free
      if ((t & 63) == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) part[parity][q][t >> 6] = sum[q];
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < 4; ++q) sum[q] = 0.0;
      for (int i = 0; i < (int)(blockDim.x >> 6); ++i) {
#pragma unroll
        for (int q = 0; q < 4; ++q) sum[q] += part[parity][q][i];
      }
    }
    // lanes without values add nothing: with eps = 0 the scale of a row beyond the last would be
    // infinite, and its part of grad_w (0 times it) NaN
    if (!valid) continue;
    double mu;
    const float s = row_statistics(sum[0], sum[1], p, k, a.eps, mu);
    const float f1 = (float)(sum[2] * inv_k);
    const float f2 = (float)((double)s * ((sum[3] - (mu - (double)p) * sum[2]) * inv_k));
    forget(rr);
#pragma unroll
    for (int h = 0; h < 16; h += 8) {
      float x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int i = h + q;
        const float n = (float)((double)rr.get(i) - mu) * s, g = gy.get(i);
        gw[i] = fmaf(g, n, gw[i]);
        gb[i] += g;
        x[q] = s * (fmaf(g, w.get(i), -f1) - n * f2);
        if constexpr (kRes) x[q] += gres.get(i);
      }
      if constexpr (kSF32) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(a.grad_r) + off + h);
        d[0] = make_float4(x[0], x[1], x[2], x[3]);
        d[1] = make_float4(x[4], x[5], x[6], x[7]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.grad_r) + off + h) =
            make_uint4(gemm::pack_bf16x2(x[0], x[1]), gemm::pack_bf16x2(x[2], x[3]), gemm::pack_bf16x2(x[4], x[5]),
                       gemm::pack_bf16x2(x[6], x[7]));
      }
    }
  }
  if (a.partials == nullptr) return;
  float* const row_out = a.partials + (int64_t)blockIdx.x * 2 * k + (int64_t)c * kBlock;
  auto store = [&](const float (&g)[16], int64_t at) {
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<float4*>(row_out + at + i) = make_float4(g[i], g[i + 1], g[i + 2], g[i + 3]);
  };
  if (rows_here == 1) {
    if (in_k) {
      store(gw, 0);
      store(gb, k);
    }
    return;
  }
  // the workgroup's rows side by side in LDS, added in row order
  auto join = [&](float (&g)[16], int64_t at) {
#pragma unroll
    for (int i = 0; i < 16; ++i) colsum[t * 16 + i] = g[i];
    __syncthreads();
    if (sub == 0 && in_k) {
      for (int s = 1; s < rows_here; ++s)
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] += colsum[(s * a.lanes + c) * 16 + i];
      store(g, at);
    }
  };
  join(gw, 0);
  __syncthreads();
  join(gb, k);
}

// grad_w[j], then grad_b[j - k], = sum of n partial rows of 2 k: 32 columns per workgroup, 32
// interleaved row sets added in order.
__global__ void __launch_bounds__(1024) layernorm_weight_grad_kernel(const float* __restrict__ partials, int n,
                                                                     int64_t k, float* __restrict__ grad_w,
                                                                     float* __restrict__ grad_b) {
  __shared__ float lds[32][33];
  const int x = threadIdx.x & 31, set = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + x;
  float a = 0.0f;
  if (col < 2 * k) {
#pragma unroll 8
    for (int i = set; i < n; i += 32) a += partials[(int64_t)i * 2 * k + col];
  }
  lds[set][x] = a;
  __syncthreads();
  if (set == 0 && col < 2 * k) {
#pragma unroll
    for (int i = 1; i < 32; ++i) a += lds[i][x];
    if (col < k) grad_w[col] = a;
    else grad_b[col - k] = a;
  }
}

using ForwardFn = void (*)(const NormForward);

template <bool kMean, int kMode>
ForwardFn forward_of(const NormForward& a) {
  const int w = a.w_f32 ? 1 : 0;
  if (a.residual == nullptr) {
    static constexpr ForwardFn f[2][2] = {
        {layernorm_kernel<false, 0, false, kMean, kMode>, layernorm_kernel<false, 0, true, kMean, kMode>},
        {layernorm_kernel<true, 0, false, kMean, kMode>, layernorm_kernel<true, 0, true, kMean, kMode>}};
    return f[a.x_f32 ? 1 : 0][w];
  }
  static constexpr ForwardFn f[3][2] = {
      {layernorm_kernel<false, 1, false, kMean, kMode>, layernorm_kernel<false, 1, true, kMean, kMode>},
      {layernorm_kernel<false, 2, false, kMean, kMode>, layernorm_kernel<false, 2, true, kMean, kMode>},
      {layernorm_kernel<true, 2, false, kMean, kMode>, layernorm_kernel<true, 2, true, kMean, kMode>}};
  return f[!a.stream_f32 ? 0 : !a.x_f32 ? 1 : 2][w];
}

ForwardFn forward_kernel(const NormForward& a, bool mean) {
  if (!mean) return forward_of<false, kNormFp8>(a);
  switch (a.mode) {
    case kNormFp8: return forward_of<true, kNormFp8>(a);
    case kNormOut: return forward_of<true, kNormOut>(a);
    case kNormStatic: return forward_of<true, kNormStatic>(a);
    case kNormOneRow: return forward_of<true, kNormOneRow>(a);
    default: return forward_of<true, kNormStats>(a);
  }
}

}  // namespace

hipError_t launch_layernorm(NormForward a, bool mean, hipStream_t s) {
  const RowShape shape = row_shape(a.k);
  a.lanes = shape.lanes;
  const int64_t per = shape.threads / shape.lanes;
  // Workgroups of more than four waves walk down the rows with the weight and bias in registers; others
  // take their rows at once, the rest by the row loop.  Two walkers for each compute unit, which has room
  // for 16 waves of the layer norm's; four of the RMS norm's, which has for 28, with up to eight waves and
  // nothing in fp32 to read (above, or with it, traffic is the bound either way).  Layer norm, bf16 stream
  // with a residual, to bf16, with 512 / 768 / 1024 workgroups and one for every row: 600 x 5120 10.3 / - / - /
  // 11.1 us, 768 11.4 / - / - / 12.3, 1000 13.6 / 15.5 / - / 17.5, 2048 21.9 / 23.6 / 27.0 / 27.1, 4096 37.3 / 43.3 /
  // 46.0 / 47.1; to 8-bit codes 600 10.2 and 10.7, 1000 14.9 and 18.0, 4096 40.2 / 46.8 / 49.8 / 47.9; 1000 x 16384
  // 35.1 and 40.4; 4096 x 4096 (four waves) 33.8 and, one for every row, 31.8.  RMS norm to 8-bit codes, 512 /
  // 768 / 1024 / all: 1000 x 5120 13.3 / 12.4 / - / 12.4, 4096 35.6 / 33.0 / 33.1 / 34.3, 4096 x 8192 50.7 / 50.2 / 50.7 /
  // 50.2, x 16384 96.5 / 97.7 / 99.2 / 108.6; with an fp32 residual 4096 x 5120 51.5 / 52.0 / 52.4 / 53.6.
  const bool f32 = a.x_f32 || (a.residual != nullptr && a.stream_f32);
  const int64_t walkers = !mean && !f32 && shape.lanes <= 512 ? 1024 : 512;
  int64_t blocks = std::min<int64_t>((a.rows + per - 1) / per, shape.lanes > 256 ? walkers : 1 << 20);
  if (a.mode == kNormDynamic) {
    // one row needs no second pass: its workgroup knows the whole abs-max
    a.mode = a.rows == 1 ? kNormOneRow : kNormStats;
    blocks = walking_blocks(a.rows, shape);
  }
  hipLaunchKernelGGL(forward_kernel(a, mean), dim3((uint32_t)blocks), dim3((uint32_t)shape.threads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.mode != kNormStats) return e;
  using QuantFn = void (*)(const NormForward, int);
  static constexpr QuantFn q[2][2] = {{layernorm_quantize_kernel<false, false>, layernorm_quantize_kernel<false, true>},
                                      {layernorm_quantize_kernel<true, false>, layernorm_quantize_kernel<true, true>}};
  const int64_t grid = quantize_blocks(a.rows, a.k);
  const bool sf32 = a.residual != nullptr ? a.stream_f32 : a.x_f32;
  hipLaunchKernelGGL(q[sf32 ? 1 : 0][a.w_f32 ? 1 : 0], dim3((uint32_t)grid), dim3(kNormQThreads), 0, s, a, (int)blocks);
  return hipGetLastError();
}

size_t layernorm_backward_partial_floats(int64_t rows, int64_t k) {
  return (size_t)walking_blocks(rows, row_shape(k)) * 2 * (size_t)k;
}

hipError_t launch_layernorm_backward(NormBackward a, hipStream_t s) {
  const RowShape shape = row_shape(a.k);
  a.lanes = shape.lanes;
  const int64_t blocks = walking_blocks(a.rows, shape);
  if (a.grad_w == nullptr) a.partials = nullptr;
  using Fn = void (*)(const NormBackward);
  static constexpr Fn f[2][2][2] = {
      {{layernorm_backward_kernel<false, false, false>, layernorm_backward_kernel<false, false, true>},
       {layernorm_backward_kernel<false, true, false>, layernorm_backward_kernel<false, true, true>}},
      {{layernorm_backward_kernel<true, false, false>, layernorm_backward_kernel<true, false, true>},
       {layernorm_backward_kernel<true, true, false>, layernorm_backward_kernel<true, true, true>}}};
  if (blocks > 0)
    hipLaunchKernelGGL(f[a.stream_f32 ? 1 : 0][a.w_f32 ? 1 : 0][a.grad_residual != nullptr ? 1 : 0],
                       dim3((uint32_t)blocks), dim3((uint32_t)shape.threads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.grad_w == nullptr) return e;
  hipLaunchKernelGGL(layernorm_weight_grad_kernel, dim3((uint32_t)((2 * a.k + 31) / 32)), dim3(1024), 0, s, a.partials,
                     (int)blocks, a.k, a.grad_w, a.grad_b);
  return hipGetLastError();
}

}  // namespace nvfp4
