// The activations of the linear's epilogue and their derivatives, in fp32:
//   silu       z sigma(z)
//   gelu       z Phi(z) = z erfc(-z / sqrt(2)) / 2
//   gelu_tanh  z (1 + tanh(p(z))) / 2 = z sigma(2 p(z)),  p(z) = sqrt(2/pi) (z + 0.044715 z^3)
// sigma(t) = 1 / (1 + 2^(-t log2 e)) on the hardware's exp2 and reciprocal (each within
// one fp32 ulp): the results are rounded to bf16, 2^16 times coarser, and the IEEE divide
// and a software exp would double an epilogue's vector work.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/nvfp4.h"

namespace nvfp4 {

constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kGeluP1 = 0.7978845608028654f;                 // sqrt(2 / pi)
constexpr float kGeluP3 = 0.7978845608028654f * 0.044715f;
constexpr float kInvSqrt2 = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

__device__ __forceinline__ float sigmoid_fast(float t) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-t * kLog2e));
}

__device__ __forceinline__ float activate(float z, int act) {
  if (act == NVFP4_ACT_SILU) return z * sigmoid_fast(z);
  if (act == NVFP4_ACT_GELU_TANH) return z * sigmoid_fast(2.0f * z * fmaf(kGeluP3, z * z, kGeluP1));
  if (act == NVFP4_ACT_GELU) return 0.5f * z * erfcf(-z * kInvSqrt2);
  return z;
}

// The derivative.  Past |z| = 90 each is 0 or 1 to the last bit, so z is held there: the
// products of a vanishing and an infinite factor do not arise.  NaN stays NaN.
__device__ __forceinline__ float activate_grad(float z, int act) {
  if (z != z) return z;
  z = fminf(fmaxf(z, -90.0f), 90.0f);
  if (act == NVFP4_ACT_SILU) {
    const float s = sigmoid_fast(z);
    return s * fmaf(z, 1.0f - s, 1.0f);
  }
  if (act == NVFP4_ACT_GELU_TANH) {
    const float z2 = z * z;
    const float s = sigmoid_fast(2.0f * z * fmaf(kGeluP3, z2, kGeluP1));
    return s * fmaf(z * (1.0f - s), 2.0f * fmaf(3.0f * kGeluP3, z2, kGeluP1), 1.0f);
  }
  if (act == NVFP4_ACT_GELU)
    return fmaf(z * kInvSqrt2Pi, __builtin_amdgcn_exp2f(-0.5f * kLog2e * z * z), 0.5f * erfcf(-z * kInvSqrt2));
  return 1.0f;
}

}  // namespace nvfp4
