// The activations of the linear's epilogue and their derivatives, in fp32:
//   silu       z sigma(z)
//   gelu       z Phi(z), Phi the normal distribution function
//   gelu_tanh  z (1 + tanh(p(z))) / 2 = z sigma(2 p(z)),  p(z) = sqrt(2/pi) (z + 0.044715 z^3)
// sigma(t) = 1 / (1 + 2^(-t log2 e)) on the hardware's exp2 and reciprocal (each within
// one fp32 ulp): the results are rounded to bf16, 2^16 times coarser, and the IEEE divide
// and a software exp would double an epilogue's vector work.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/nvfp4.h"

namespace nvfp4 {

constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kGeluP1 = 0.7978845608028654f;                 // sqrt(2 / pi)
constexpr float kGeluP3 = 0.7978845608028654f * 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

__device__ __forceinline__ float sigmoid_fast(float t) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-t * kLog2e));
}

// Phi(-|z|) = exp(-z^2 / 2) q(t) / 2 with q(t) = erfc(x) exp(x^2), x = |z| / sqrt(2),
// t = 1 / (1 + 0.42 x).  q is a degree-8 polynomial fitted here by reweighted least
// squares on the nodes of t over x in [0, 10]: within 4.2e-8 of q relatively, 4e-7 in fp32
// arithmetic, in the tail too (erfc - 1 would lose it).  e receives exp(-z^2 / 2).
__device__ __forceinline__ float normal_tail(float z, float& e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.42f * 0.7071067811865476f, fabsf(z), 1.0f));
  float q = 0x1.411560p-4f;
  q = fmaf(q, t, -0x1.6d84acp-2f);
  q = fmaf(q, t, 0x1.0549ecp-1f);
  q = fmaf(q, t, -0x1.a02ab2p-3f);
  q = fmaf(q, t, 0x1.41c022p-2f);
  q = fmaf(q, t, 0x1.6b1ecap-3f);
  q = fmaf(q, t, 0x1.f2d5bep-3f);
  q = fmaf(q, t, 0x1.e3ff48p-3f);
  q = fmaf(q, t, 0x1.b332f2p-16f);
  e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * z * z);
  return 0.5f * e * q;
}

template <int kAct>
__device__ __forceinline__ float activate_t(float z) {
  if constexpr (kAct == NVFP4_ACT_SILU) return z * sigmoid_fast(z);
  if constexpr (kAct == NVFP4_ACT_GELU_TANH) return z * sigmoid_fast(2.0f * z * fmaf(kGeluP3, z * z, kGeluP1));
  if constexpr (kAct == NVFP4_ACT_GELU) {
    float e;
    const float tail = normal_tail(z, e);
    return z * (z < 0.0f ? tail : 1.0f - tail);
  }
  return z;
}

__device__ __forceinline__ float activate(float z, int act) {
  if (act == NVFP4_ACT_SILU) return activate_t<NVFP4_ACT_SILU>(z);
  if (act == NVFP4_ACT_GELU_TANH) return activate_t<NVFP4_ACT_GELU_TANH>(z);
  if (act == NVFP4_ACT_GELU) return activate_t<NVFP4_ACT_GELU>(z);
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
  if (act == NVFP4_ACT_GELU) {
    float e;
    const float tail = normal_tail(z, e);
    return fmaf(z * kInvSqrt2Pi, e, z < 0.0f ? tail : 1.0f - tail);
  }
  return 1.0f;
}

}  // namespace nvfp4
