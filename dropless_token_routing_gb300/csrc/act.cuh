// The activations of the linear layer and their derivatives, in fp32.
#pragma once

#include "common.cuh"

namespace moe {

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kGeluC = 0.79788456080286536f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// The fp32 forms keep their relative accuracy where the result is small (z well below 0): the normal
// distribution's cumulative is erfc, the tanh form z times the logistic of 2 u. Written as 1 + erf and
// 1 + tanh they cancel there (4 % off at z = -5, everything at -6).
__device__ __forceinline__ float gelu_u(float z) { return kGeluC * (z + kGeluA * z * z * z); }
// The tanh form's slope is 0 or 1 to the last bit past 12; its polynomial would overflow further out.
__device__ __forceinline__ float gelu_clamp(float z) { return z > 12.f ? 12.f : z < -12.f ? -12.f : z; }   // keeps NaN

template <int ACT> __device__ __forceinline__ float act_f(float z) {
  if constexpr (ACT == MOE_ACT_RELU) return z < 0.f ? 0.f : z;   // keeps NaN
  if constexpr (ACT == MOE_ACT_SILU) return silu_f(z);
  if constexpr (ACT == MOE_ACT_GELU) return 0.5f * z * erfcf(-z * kSqrtHalf);
  if constexpr (ACT == MOE_ACT_GELU_TANH) return z / (1.f + expf(-2.f * gelu_u(z)));
  return z;
}

template <int ACT> __device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == MOE_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if constexpr (ACT == MOE_ACT_SILU) {
    const float sg = 1.f / (1.f + expf(-z));
    return sg * (1.f + z * (1.f - sg));
  }
  if constexpr (ACT == MOE_ACT_GELU)
    return 0.5f * erfcf(-z * kSqrtHalf) + z * kInvSqrt2Pi * expf(-0.5f * z * z);
  if constexpr (ACT == MOE_ACT_GELU_TANH) {
    // act = z s(2u), s' = s(2u) s(-2u); of these the one below 1/2 is e / (1 + e), the other 1 / (1 + e)
    const float v = gelu_clamp(z), u = 2.f * gelu_u(v), e = expf(-fabsf(u)), big = 1.f / (1.f + e), small = e * big;
    return (u > 0.f ? big : small) + v * big * small * 2.f * kGeluC * (1.f + 3.f * kGeluA * v * v);
  }
  return 1.f;
}

// The forms for results that are rounded to bf16 (2^-9): the hardware's exponential and reciprocal,
// a few 2^-22 off, take a third of the instructions; in the product kernels' epilogues the exact
// forms cost a 4096 x 2816 x 2048 product 15 of 55 us. The normal distribution's cumulative is erfc's
// five-term approximation 7.1.26 of Abramowitz and Stegun, "Handbook of Mathematical Functions", on
// the side where it is small. Its bound is absolute, 1.5e-7 (7.5e-8 of the cumulative); relative to a
// cumulative that is small itself it is 1.6e-3 off at z = -5, 3.6e-3 at -6 and 2e-2 at -10, where a
// bf16 result's own rounding is 2e-3 (the values are below 2e-6 there).
__device__ __forceinline__ float logistic_fast(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }
// exp(-z^2 / 2) goes to `e`
__device__ __forceinline__ float normal_cdf_fast(float z, float& e) {
  const float x = fabsf(z) * kSqrtHalf;
  const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
  e = __expf(-x * x);
  const float p = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f), 0.254829592f);
  const float tail = 0.5f * p * e;
  return z < 0.f ? tail : 1.f - tail;
}

template <int ACT> __device__ __forceinline__ float act_fast(float z) {
  if constexpr (ACT == MOE_ACT_SILU) return z * logistic_fast(z);
  if constexpr (ACT == MOE_ACT_GELU) {
    float e;
    return z * normal_cdf_fast(z, e);
  }
  if constexpr (ACT == MOE_ACT_GELU_TANH) return z * logistic_fast(2.f * gelu_u(z));
  return act_f<ACT>(z);
}

template <int ACT> __device__ __forceinline__ float act_slope_fast(float z) {
  if constexpr (ACT == MOE_ACT_SILU) {
    const float s = logistic_fast(z);
    return s * (1.f + z * (1.f - s));
  }
  if constexpr (ACT == MOE_ACT_GELU) {
    float e;
    const float c = normal_cdf_fast(z, e);
    return fmaf(z * kInvSqrt2Pi, e, c);
  }
  if constexpr (ACT == MOE_ACT_GELU_TANH) {
    // act = z s(2u), s' = s (1 - s)
    const float v = gelu_clamp(z), s = logistic_fast(2.f * gelu_u(v));
    return s + v * s * (1.f - s) * 2.f * kGeluC * (1.f + 3.f * kGeluA * v * v);
  }
  return act_slope<ACT>(z);
}

// The activations by a value that is the same in the whole launch.
__device__ __forceinline__ float act_any(int act, float z) {
  switch (act) {
    case MOE_ACT_RELU: return act_f<MOE_ACT_RELU>(z);
    case MOE_ACT_SILU: return act_f<MOE_ACT_SILU>(z);
    case MOE_ACT_GELU: return act_f<MOE_ACT_GELU>(z);
    case MOE_ACT_GELU_TANH: return act_f<MOE_ACT_GELU_TANH>(z);
    default: return z;
  }
}
__device__ __forceinline__ float act_any_fast(int act, float z) {
  switch (act) {
    case MOE_ACT_RELU: return act_fast<MOE_ACT_RELU>(z);
    case MOE_ACT_SILU: return act_fast<MOE_ACT_SILU>(z);
    case MOE_ACT_GELU: return act_fast<MOE_ACT_GELU>(z);
    case MOE_ACT_GELU_TANH: return act_fast<MOE_ACT_GELU_TANH>(z);
    default: return z;
  }
}

// CALL(ACT) with the activation `act` (validated by the caller) as a constant.
#define MOE_ACT_SWITCH(act, CALL)                                    \
  switch (act) {                                                     \
    case MOE_ACT_RELU: CALL(MOE_ACT_RELU); break;                    \
    case MOE_ACT_SILU: CALL(MOE_ACT_SILU); break;                    \
    case MOE_ACT_GELU: CALL(MOE_ACT_GELU); break;                    \
    case MOE_ACT_GELU_TANH: CALL(MOE_ACT_GELU_TANH); break;          \
    default: CALL(MOE_ACT_NONE); break;                              \
  }

}  // namespace moe
