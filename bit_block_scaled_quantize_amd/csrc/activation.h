// The element functions around a linear layer's GEMM, in FP32: act(z), and act'(z) for the
// backward pass. Kinds as nvfp4_act in include/nvfp4.h.
//   relu2  max(z, 0)^2                 2 max(z, 0)
//   gelu   z s(2u), u = sqrt(2/pi) (z + 0.044715 z^3), s(t) = 1 / (1 + exp(-t)): the tanh form,
//          since (1 + tanh u) / 2 = s(2u)
//          s + z s (1 - s) 2u'
//   silu   z s(z)                      s + z s (1 - s)
// exp(-t) overflows to infinity for t below about -88, where s is 0 as it should be; z s is then
// -0 and not the true value, which is smaller than 2^-120. For z = -inf, z s would be NaN; it is 0.
// The reciprocal is the hardware's (1 ulp): two roundings more than a division's one, three
// orders below the BF16 rounding of what is stored.
#pragma once

#include "device_common.h"

namespace nvfp4 {

enum ActKind : int { kActNone = 0, kActRelu2 = 1, kActGelu = 2, kActSilu = 3 };

// sigmoid(t) of the argument u = -t log2(e); the gelu's u is one polynomial in z with the base
// change in its coefficients (two fused steps: four roundings on t in all).
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kGelu1 = 1.59576912160573f, kGelu3 = 0.0713548162726002f;   // 2 sqrt(2/pi) (1, 0.044715)
constexpr float kGelu1L = 2.302208198144325f, kGelu3L = 0.102943239580023f;    // the same times log2(e)

__device__ __forceinline__ float sigmoid_exp2(float u) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u));
}

template <int ACT>
__device__ __forceinline__ float sigmoid_of(float z) {
  if constexpr (ACT == kActSilu) return sigmoid_exp2(z * -kLog2e);
  else return sigmoid_exp2(-z * __builtin_fmaf(kGelu3L, z * z, kGelu1L));
}

template <int ACT>
__device__ __forceinline__ float act(float z) {
  if constexpr (ACT == kActRelu2) {
    return z <= 0.0f ? 0.0f : z * z;                          // NaN stays NaN
  } else if constexpr (ACT == kActGelu || ACT == kActSilu) {
    const float y = z * sigmoid_of<ACT>(z);
    return z == -INFINITY ? 0.0f : y;
  } else {
    return z;
  }
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == kActRelu2) {
    return z <= 0.0f ? 0.0f : 2.0f * z;
  } else if constexpr (ACT == kActGelu || ACT == kActSilu) {
    constexpr bool gelu = ACT == kActGelu;
    const float dt = gelu ? __builtin_fmaf(3.0f * kGelu3, z * z, kGelu1) : 1.0f;
    const float s = sigmoid_of<ACT>(z);
    const float c = z * (1.0f - s) * dt;                      // grows while s vanishes, and the other way
    const float y = __builtin_fmaf(s, c, s);
    // past this s is exactly 0 or 1 in FP32, and a factor that overflows would make 0 * inf of it
    return fabsf(z) > (gelu ? 30.0f : 200.0f) ? (z > 0.0f ? 1.0f : 0.0f) : y;
  } else {
    return 1.0f;
  }
}

// act with a kind known at run time (uniform), for epilogues of few elements.
__device__ __forceinline__ float act_of(int kind, float z) {
  return kind == kActRelu2 ? act<kActRelu2>(z) : kind == kActGelu ? act<kActGelu>(z)
       : kind == kActSilu ? act<kActSilu>(z) : z;
}

}  // namespace nvfp4
