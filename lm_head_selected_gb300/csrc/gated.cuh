// Activations of the gated linear layer and their derivatives, in fp32.
#pragma once

#include <cuda_runtime.h>

#include "sm103_ptx.cuh"

namespace llp {

enum GatedAct { kActSilu = 0, kActGelu = 1, kActGeluTanh = 2, kNumActs = 3 };

// 1 / (1 + 2^t), t the exponent times -log2(e): 0 where 2^t is infinite.
__device__ __forceinline__ float logistic2(float t) { return __fdividef(1.f, 1.f + ex2_approx(t)); }

constexpr float kLog2eG = 1.4426950408889634f;
constexpr float kTanhK = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kTanhC = 0.044715f;
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// silu z s(z); gelu z Phi(z), Phi by erfc, which keeps its digits for negative z; the tanh form of
// gelu as z s(k (z + c z^3)), s the logistic function: (1 + tanh t) / 2 = s(2 t).
template <int ACT>
__device__ __forceinline__ float gated_act(float z) {
  if (ACT == kActGelu) return 0.5f * z * erfcf(-kSqrtHalf * z);
  const float t = ACT == kActSilu ? z : kTanhK * fmaf(kTanhC * z * z, z, z);
  return z * logistic2(-kLog2eG * t);
}

// The activation and its derivative.
template <int ACT>
__device__ __forceinline__ void gated_act_slope(float z, float& a, float& slope) {
  if (ACT == kActGelu) {
    const float phi = 0.5f * erfcf(-kSqrtHalf * z);
    a = z * phi;
    slope = fmaf(z, kInvSqrt2Pi * ex2_approx(-0.5f * kLog2eG * z * z), phi);
  } else if (ACT == kActSilu) {
    const float s = logistic2(-kLog2eG * z);
    a = z * s;
    slope = fmaf(a, 1.f - s, s);
  } else {
    const float s = logistic2(-kLog2eG * kTanhK * fmaf(kTanhC * z * z, z, z));
    a = z * s;
    // 1 - s is 0 in fp32 long before the polynomial's slope could make that 0 * infinity
    const float d = fabsf(z) > 16.f ? 0.f : kTanhK * fmaf(3.f * kTanhC * z, z, 1.f);
    slope = fmaf(a * (1.f - s), d, s);
  }
}

}  // namespace llp
