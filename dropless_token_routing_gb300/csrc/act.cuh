// The activations of the linear layer and their derivatives, in fp32.
#pragma once

#include "common.cuh"

namespace moe {

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kGeluC = 0.79788456080286536f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

template <int ACT> __device__ __forceinline__ float act_f(float z) {
  if constexpr (ACT == MOE_ACT_RELU) return z < 0.f ? 0.f : z;   // keeps NaN
  if constexpr (ACT == MOE_ACT_SILU) return silu_f(z);
  if constexpr (ACT == MOE_ACT_GELU) return 0.5f * z * (1.f + erff(z * kSqrtHalf));
  if constexpr (ACT == MOE_ACT_GELU_TANH) return 0.5f * z * (1.f + tanhf(kGeluC * (z + kGeluA * z * z * z)));
  return z;
}

template <int ACT> __device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == MOE_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if constexpr (ACT == MOE_ACT_SILU) {
    const float sg = 1.f / (1.f + expf(-z));
    return sg * (1.f + z * (1.f - sg));
  }
  if constexpr (ACT == MOE_ACT_GELU)
    return 0.5f * (1.f + erff(z * kSqrtHalf)) + z * kInvSqrt2Pi * expf(-0.5f * z * z);
  if constexpr (ACT == MOE_ACT_GELU_TANH) {
    const float th = tanhf(kGeluC * (z + kGeluA * z * z * z));
    return 0.5f * (1.f + th) + 0.5f * z * (1.f - th * th) * kGeluC * (1.f + 3.f * kGeluA * z * z);
  }
  return 1.f;
}

// The activation by a value that is the same in the whole launch.
__device__ __forceinline__ float act_any(int act, float z) {
  switch (act) {
    case MOE_ACT_RELU: return act_f<MOE_ACT_RELU>(z);
    case MOE_ACT_SILU: return act_f<MOE_ACT_SILU>(z);
    case MOE_ACT_GELU: return act_f<MOE_ACT_GELU>(z);
    case MOE_ACT_GELU_TANH: return act_f<MOE_ACT_GELU_TANH>(z);
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
