// Activations of the gated linear layer and their derivatives, in fp32.
#pragma once

#include "elem.cuh"
#include "sm103_ptx.cuh"

namespace llp {

enum GatedAct { kActSilu = 0, kActGelu = 1, kActGeluTanh = 2, kNumActs = 3 };

constexpr float kLog2eG = 1.4426950408889634f;
constexpr float kTanhK = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kTanhC = 0.044715f;
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

__device__ __forceinline__ F2 ex2_pair(F2 a) { return f2(ex2_approx(a.x), ex2_approx(a.y)); }
__device__ __forceinline__ F2 inverse_pair(F2 a) { return f2(inverse_ftz(a.x), inverse_ftz(a.y)); }

// 1 / (1 + 2^t), t the exponent times -log2(e): 0 where 2^t is infinite.
__device__ __forceinline__ F2 logistic2(F2 t) { return inverse_pair(add2(ex2_pair(t), f2(1.f))); }

// 1 - Phi(|z|) = exp(-z^2 / 2) P(t) / 2 with t = 1 / (1 + 0.425 |z| / sqrt 2): P, without a constant term, is
// the least-maximum fit of erfcx(x) = exp(x^2) erfc(x) over 0 <= x <= 12 (Lawson's reweighted least squares
// in 64 bits), 2.5e-7 of its value away at most: the fit alone.  The exponential adds its rounded argument's
// error, at most 1.5 z^2 2^-24 (7e-6 at |z| = 12).  It keeps its digits far into the tail, as 1 + erf does
// not, and takes a third of erfcf's time.  `bell`: exp(-z^2 / 2).
__device__ __forceinline__ F2 normal_tail(F2 z, F2& bell) {
  const float c[8] = {2.397032969e-01f, 2.414485773e-01f, 2.032271325e-01f,
                      2.465589095e-01f, -8.680285066e-02f, 3.894496163e-01f,
                      -3.024697204e-01f, 6.888479261e-02f};
  bell = ex2_pair(mul2(mul2(z, z), f2(-0.5f * kLog2eG)));
  const F2 t = inverse_pair(fma2(f2(fabsf(z.x), fabsf(z.y)), f2(0.425f * kSqrtHalf), f2(1.f)));
  F2 p = f2(c[7]);
#pragma unroll
  for (int i = 6; i >= 0; --i) p = fma2(p, t, f2(c[i]));
  return mul2(mul2(p, t), mul2(bell, f2(0.5f)));
}
__device__ __forceinline__ F2 normal_cdf(F2 z, F2& bell) {
  const F2 q = normal_tail(z, bell);
  return f2(z.x < 0.f ? q.x : 1.f - q.x, z.y < 0.f ? q.y : 1.f - q.y);
}

// silu z s(z); gelu z Phi(z); the tanh form of gelu as z s(k (z + c z^3)), s the logistic function:
// (1 + tanh t) / 2 = s(2 t).  Two at a time.  Towards -infinity the relative error grows with the
// exponential's argument t, which is rounded to fp32: beside 2^-19, silu's by 2 |z| 2^-24 and the tanh form's by
// 5 |t| 2^-24 (1.4e-5 at z = -10), far below one rounding to 16 bits; a factor below 2^-126 counts as 0.
template <int ACT>
__device__ __forceinline__ F2 gated_act(F2 z) {
  if (ACT == kActGelu) {
    F2 bell;
    return mul2(z, normal_cdf(z, bell));
  }
  const F2 t = ACT == kActSilu ? mul2(z, f2(-kLog2eG))
                               : mul2(mul2(z, f2(-kLog2eG * kTanhK)), fma2(mul2(z, f2(kTanhC)), z, f2(1.f)));
  return mul2(z, logistic2(t));
}

// The activation and its derivative.
template <int ACT>
__device__ __forceinline__ void gated_act_slope(F2 z, F2& a, F2& slope) {
  if (ACT == kActGelu) {
    F2 bell;
    const F2 phi = normal_cdf(z, bell);
    a = mul2(z, phi);
    slope = fma2(mul2(z, f2(kInvSqrt2Pi)), bell, phi);
  } else if (ACT == kActSilu) {
    const F2 s = logistic2(mul2(z, f2(-kLog2eG)));
    a = mul2(z, s);
    slope = fma2(a, fma2(s, f2(-1.f), f2(1.f)), s);
  } else {
    const F2 s = logistic2(mul2(mul2(z, f2(-kLog2eG * kTanhK)), fma2(mul2(z, f2(kTanhC)), z, f2(1.f))));
    a = mul2(z, s);
    // s (1 - s) is 0 in fp32 long before the polynomial's slope could make that 0 * infinity
    const F2 d = mul2(fma2(mul2(z, f2(3.f * kTanhC)), z, f2(1.f)), f2(kTanhK));
    const F2 e = f2(fabsf(z.x) > 16.f ? 0.f : d.x, fabsf(z.y) > 16.f ? 0.f : d.y);
    slope = fma2(mul2(a, fma2(s, f2(-1.f), f2(1.f))), e, s);
  }
}

}  // namespace llp
