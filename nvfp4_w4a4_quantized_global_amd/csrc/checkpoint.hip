// 8-bit activation checkpoints on gfx950: packing (with the block rotation) and unpacking,
// SwiGLU with its operands kept in 8 bits, and the gradients of SwiGLU and of the linear's
// activations read from checkpoints or from bf16.
//
// All of it is HBM-bound streaming over [rows][k] arrays: a lane owns 16 consecutive
// values (32 bytes of bf16, 16 code bytes), eight lanes a 128-wide tile of a row, lane
// pairs a 32-value checkpoint block.  The format is in checkpoint_device.h.
//
// Measured at 4096 x 25600: SwiGLU with both checkpoints 846 MB in 172 us (4.9 TB/s; the
// product's exact exp and divide are the rest), its gradient from them 847 MB in 162 us
// (5.2 TB/s).  Packing 777 x 5120 values with a rotation takes 6.9 us, most of it the launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "activation_device.h"
#include "checkpoint_device.h"
#include "nvfp4_device.h"
#include "nvfp4_launch.h"
#include "quantize_device.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 8192;

// Where a lane's 16 values are: tiles of 128 values, counted row by row.
struct Place {
  int64_t row, chunk;   // chunk: 16-value chunk of the row
  bool valid;
};
__device__ __forceinline__ Place place_of(int64_t unit, int64_t rows, int64_t k) {
  const int64_t kt = (k + kScaleTileK - 1) / kScaleTileK;
  Place p;
  // 64-bit division only where 32 bits do not hold the count
  if (rows * kt <= 0x7FFFFFFF - kMaxBlocks * 32) p.row = (uint32_t)unit / (uint32_t)kt;
  else p.row = unit / kt;
  p.chunk = (unit - p.row * kt) * 8 + (threadIdx.x & 7);
  p.valid = p.row < rows && p.chunk < k / kBlock;
  return p;
}
__device__ __forceinline__ int64_t scale_at(const Place& p, int64_t k) {
  return p.row * ((k + kCkBlock - 1) / kCkBlock) + (p.chunk >> 1);
}

__device__ __forceinline__ void zero16(float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
}

// fp32 values to bf16 bits, 16 of them.
__device__ __forceinline__ void store16_rounded(uint16_t* p, const float (&v)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = gemm::pack_bf16x2(v[2 * i], v[2 * i + 1]);
  uint4* d = reinterpret_cast<uint4*>(p);
  d[0] = make_uint4(w[0], w[1], w[2], w[3]);
  d[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

__device__ __forceinline__ void store_checkpoint(const float (&v)[16], const Place& p, int64_t k, uint8_t* codes,
                                                 uint8_t* scales) {
  uint32_t sb;
  const uint4 c = ck_pack16(v, sb);
  if (!p.valid) return;
  *reinterpret_cast<uint4*>(codes + p.row * k + p.chunk * kBlock) = c;
  if ((p.chunk & 1) == 0) scales[scale_at(p, k)] = (uint8_t)sb;
}

// 16 saved values: bf16 (scales NULL) or checkpoint codes.
template <bool kPacked>
__device__ __forceinline__ void load_saved16(const void* saved, const uint8_t* scales, const Place& p, int64_t k,
                                             float (&v)[16]) {
  const int64_t off = p.row * k + p.chunk * kBlock;
  if constexpr (kPacked) {
    const uint4 c = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(saved) + off);
    ck_decode16(c, scales[scale_at(p, k)], v);
  } else {
    load16_bf16(static_cast<const uint16_t*>(saved) + off, v);
  }
}

template <bool kRotate>
__global__ void __launch_bounds__(kThreads) checkpoint_pack_kernel(const uint16_t* __restrict__ x, int64_t rows,
                                                                    int64_t k, int group, float inv_sqrt_g,
                                                                    uint8_t* __restrict__ codes,
                                                                    uint8_t* __restrict__ scales, int64_t units) {
  for (int64_t u = (int64_t)blockIdx.x * 32; u < units; u += (int64_t)gridDim.x * 32) {
    const Place p = place_of(u + (threadIdx.x >> 3), rows, k);
    float v[16];
    if (p.valid) load16_bf16(x + p.row * k + p.chunk * kBlock, v);
    else zero16(v);
    if (kRotate) rotate16_bf16(v, group, inv_sqrt_g);
    store_checkpoint(v, p, k, codes, scales);
  }
}

template <bool kOutBf16>
__global__ void __launch_bounds__(kThreads) checkpoint_unpack_kernel(const uint8_t* __restrict__ codes,
                                                                      const uint8_t* __restrict__ scales, int64_t rows,
                                                                      int64_t k, void* __restrict__ out,
                                                                      int64_t units) {
  for (int64_t u = (int64_t)blockIdx.x * 32; u < units; u += (int64_t)gridDim.x * 32) {
    const Place p = place_of(u + (threadIdx.x >> 3), rows, k);
    if (!p.valid) continue;
    float v[16];
    load_saved16<true>(codes, scales, p, k, v);
    const int64_t off = p.row * k + p.chunk * kBlock;
    if (kOutBf16) {
      store16_bf16(static_cast<uint16_t*>(out) + off, v);
    } else {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(out) + off);
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
  }
}

// The SwiGLU product (the bits of nvfp4_swiglu) and both operands' checkpoints in one pass.
__global__ void __launch_bounds__(kThreads) swiglu_checkpoint_kernel(
    const uint16_t* __restrict__ gate, const uint16_t* __restrict__ up, int64_t rows, int64_t k,
    uint16_t* __restrict__ x, uint8_t* __restrict__ gate_codes, uint8_t* __restrict__ gate_scales,
    uint8_t* __restrict__ up_codes, uint8_t* __restrict__ up_scales, int64_t units) {
  for (int64_t u = (int64_t)blockIdx.x * 32; u < units; u += (int64_t)gridDim.x * 32) {
    const Place p = place_of(u + (threadIdx.x >> 3), rows, k);
    const int64_t off = p.row * k + p.chunk * kBlock;
    float g[16], h[16];
    if (p.valid) {
      load16_bf16(gate + off, g);
      load16_bf16(up + off, h);
    } else {
      zero16(g);
      zero16(h);
    }
    store_checkpoint(g, p, k, gate_codes, gate_scales);
    store_checkpoint(h, p, k, up_codes, up_scales);
    if (p.valid) {
#pragma unroll
      for (int i = 0; i < 16; ++i) g[i] = swiglu_bf16(g[i], h[i]);
      store16_bf16(x + off, g);
    }
  }
}

// x = g sigma(g) u:  grad_g = gy u sigma (1 + g (1 - sigma)),  grad_u = gy g sigma.
template <bool kPacked>
__global__ void __launch_bounds__(kThreads) swiglu_backward_kernel(
    const uint16_t* __restrict__ gy, const void* __restrict__ gate, const uint8_t* __restrict__ gate_scales,
    const void* __restrict__ up, const uint8_t* __restrict__ up_scales, int64_t rows, int64_t k,
    uint16_t* __restrict__ grad_gate, uint16_t* __restrict__ grad_up, int64_t units) {
  for (int64_t u = (int64_t)blockIdx.x * 32; u < units; u += (int64_t)gridDim.x * 32) {
    const Place p = place_of(u + (threadIdx.x >> 3), rows, k);
    if (!p.valid) continue;
    const int64_t off = p.row * k + p.chunk * kBlock;
    float y[16], g[16], h[16];
    load16_bf16(gy + off, y);
    load_saved16<kPacked>(gate, gate_scales, p, k, g);
    load_saved16<kPacked>(up, up_scales, p, k, h);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      h[i] = y[i] * h[i] * activate_grad(g[i], NVFP4_ACT_SILU);
      g[i] = y[i] * activate(g[i], NVFP4_ACT_SILU);
    }
    store16_rounded(grad_gate + off, h);
    store16_rounded(grad_up + off, g);
  }
}

// grad_z = gy act'(z) from a checkpoint of z.
__global__ void __launch_bounds__(kThreads) activation_backward_packed_kernel(
    const uint16_t* __restrict__ gy, const uint8_t* __restrict__ z, const uint8_t* __restrict__ z_scales, int64_t rows,
    int64_t k, int act, uint16_t* __restrict__ grad_z, int64_t units) {
  for (int64_t u = (int64_t)blockIdx.x * 32; u < units; u += (int64_t)gridDim.x * 32) {
    const Place p = place_of(u + (threadIdx.x >> 3), rows, k);
    if (!p.valid) continue;
    const int64_t off = p.row * k + p.chunk * kBlock;
    float y[16], v[16];
    load16_bf16(gy + off, y);
    load_saved16<true>(z, z_scales, p, k, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = y[i] * activate_grad(v[i], act);
    store16_rounded(grad_z + off, v);
  }
}

// The same from bf16 z, over any count of elements (rows of any length).
__global__ void __launch_bounds__(kThreads) activation_backward_kernel(const uint16_t* __restrict__ gy,
                                                                        const uint16_t* __restrict__ z, int64_t count,
                                                                        int act, uint16_t* __restrict__ grad_z) {
  const int64_t stride = (int64_t)gridDim.x * kThreads * 16;
  for (int64_t off = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 16; off < count; off += stride) {
    if (off + 16 <= count) {
      float y[16], v[16];
      load16_bf16(gy + off, y);
      load16_bf16(z + off, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = y[i] * activate_grad(v[i], act);
      store16_rounded(grad_z + off, v);
    } else {
      for (int64_t i = off; i < count; ++i) {
        const float d = bf16_to_f32(gy[i]) * activate_grad(bf16_to_f32(z[i]), act);
        grad_z[i] = (uint16_t)gemm::pack_bf16x2(d, 0.0f);
      }
    }
  }
}

int64_t units_of(int64_t rows, int64_t k) { return rows * ((k + kScaleTileK - 1) / kScaleTileK); }
dim3 grid_of(int64_t units) { return dim3((uint32_t)std::min<int64_t>((units + 31) / 32, kMaxBlocks)); }

}  // namespace

hipError_t launch_checkpoint_pack(const uint16_t* x, int64_t rows, int64_t k, int group, float inv_sqrt_g,
                                  uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int64_t units = units_of(rows, k);
  if (group > 1)
    hipLaunchKernelGGL(checkpoint_pack_kernel<true>, grid_of(units), dim3(kThreads), 0, s, x, rows, k, group,
                       inv_sqrt_g, codes, scales, units);
  else
    hipLaunchKernelGGL(checkpoint_pack_kernel<false>, grid_of(units), dim3(kThreads), 0, s, x, rows, k, group,
                       inv_sqrt_g, codes, scales, units);
  return hipGetLastError();
}

hipError_t launch_checkpoint_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t k, void* out,
                                    bool out_bf16, hipStream_t s) {
  const int64_t units = units_of(rows, k);
  if (out_bf16)
    hipLaunchKernelGGL(checkpoint_unpack_kernel<true>, grid_of(units), dim3(kThreads), 0, s, codes, scales, rows, k,
                       out, units);
  else
    hipLaunchKernelGGL(checkpoint_unpack_kernel<false>, grid_of(units), dim3(kThreads), 0, s, codes, scales, rows, k,
                       out, units);
  return hipGetLastError();
}

hipError_t launch_swiglu_checkpoint(const uint16_t* gate, const uint16_t* up, int64_t rows, int64_t k, uint16_t* x,
                                    uint8_t* gate_codes, uint8_t* gate_scales, uint8_t* up_codes, uint8_t* up_scales,
                                    hipStream_t s) {
  const int64_t units = units_of(rows, k);
  hipLaunchKernelGGL(swiglu_checkpoint_kernel, grid_of(units), dim3(kThreads), 0, s, gate, up, rows, k, x, gate_codes,
                     gate_scales, up_codes, up_scales, units);
  return hipGetLastError();
}

hipError_t launch_swiglu_backward(const uint16_t* gy, const void* gate, const uint8_t* gate_scales, const void* up,
                                  const uint8_t* up_scales, int64_t rows, int64_t k, uint16_t* grad_gate,
                                  uint16_t* grad_up, hipStream_t s) {
  const int64_t units = units_of(rows, k);
  if (gate_scales != nullptr)
    hipLaunchKernelGGL(swiglu_backward_kernel<true>, grid_of(units), dim3(kThreads), 0, s, gy, gate, gate_scales, up,
                       up_scales, rows, k, grad_gate, grad_up, units);
  else
    hipLaunchKernelGGL(swiglu_backward_kernel<false>, grid_of(units), dim3(kThreads), 0, s, gy, gate, gate_scales, up,
                       up_scales, rows, k, grad_gate, grad_up, units);
  return hipGetLastError();
}

hipError_t launch_activation_backward(const uint16_t* gy, const void* z, const uint8_t* z_scales, int64_t rows,
                                      int64_t k, int act, uint16_t* grad_z, hipStream_t s) {
  if (z_scales != nullptr) {
    const int64_t units = units_of(rows, k);
    hipLaunchKernelGGL(activation_backward_packed_kernel, grid_of(units), dim3(kThreads), 0, s, gy,
                       static_cast<const uint8_t*>(z), z_scales, rows, k, act, grad_z, units);
  } else {
    const int64_t count = rows * k;
    const int64_t blocks = std::min<int64_t>((count + 16 * kThreads - 1) / (16 * kThreads), kMaxBlocks);
    hipLaunchKernelGGL(activation_backward_kernel, dim3((uint32_t)blocks), dim3(kThreads), 0, s, gy,
                       static_cast<const uint16_t*>(z), count, act, grad_z);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
