// Activations of the dense product and their derivatives, in FP32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "nvfp4moe.h"

namespace nvfp4moe {

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f;

// 1 / (1 + exp(-z)); exp(-z) = inf gives 0.
__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

// NaN stays NaN in every activation.  The activation is a template argument, chosen once per tile or
// launch: chosen per value it became an indirect jump per value (8192 x 8192, K = 64, ReLU: 239 us
// against 72 without an activation).
template <int kAct>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (kAct == NVFP4MOE_ACT_RELU) return z < 0.0f ? 0.0f : z;
  else if constexpr (kAct == NVFP4MOE_ACT_SILU) return z * sigmoid_f(z);
  else if constexpr (kAct == NVFP4MOE_ACT_GELU) return 0.5f * z * (1.0f + erff(z * kSqrtHalf));
  // 0.5 (1 + tanh(u)) = 1 / (1 + exp(-2u))
  else if constexpr (kAct == NVFP4MOE_ACT_GELU_TANH)
    return z * sigmoid_f(2.0f * kSqrt2OverPi * (z + 0.044715f * z * z * z));
  else return z;
}

// `limit` where the formula is 0 times inf, and at a NaN, where it is NaN itself.
__device__ __forceinline__ float or_limit(float v, float limit) { return v == v ? v : limit; }

// d act / dz; its limits 0 and 1 at infinite z (a saved sum beyond its 16-bit type) and where z's square is beyond FP32.
template <int kAct>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (kAct == NVFP4MOE_ACT_RELU) {
    return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
  } else if constexpr (kAct == NVFP4MOE_ACT_SILU) {
    const float p = sigmoid_f(z);
    return or_limit(p * (1.0f + z * (1.0f - p)), p);
  } else if constexpr (kAct == NVFP4MOE_ACT_GELU) {
    const float phi = 0.5f * (1.0f + erff(z * kSqrtHalf)), e = __expf(-0.5f * z * z);
    return or_limit(phi + z * e * kInvSqrt2Pi, phi);
  } else if constexpr (kAct == NVFP4MOE_ACT_GELU_TANH) {
    const float z2 = z * z;
    const float p = sigmoid_f(2.0f * kSqrt2OverPi * (z + 0.044715f * z * z2));
    // p + z p (1 - p) d(2u)/dz
    return or_limit(p + z * p * (1.0f - p) * (2.0f * kSqrt2OverPi) * (1.0f + 3.0f * 0.044715f * z2), p);
  } else {
    return 1.0f;
  }
}

// Calls f with the activation as an integral constant.
template <int kAct>
struct ActConst {
  static constexpr int value = kAct;
};
template <typename F>
__host__ __device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case NVFP4MOE_ACT_RELU: f(ActConst<NVFP4MOE_ACT_RELU>{}); break;
    case NVFP4MOE_ACT_SILU: f(ActConst<NVFP4MOE_ACT_SILU>{}); break;
    case NVFP4MOE_ACT_GELU: f(ActConst<NVFP4MOE_ACT_GELU>{}); break;
    case NVFP4MOE_ACT_GELU_TANH: f(ActConst<NVFP4MOE_ACT_GELU_TANH>{}); break;
    default: f(ActConst<NVFP4MOE_ACT_NONE>{});
  }
}

// The same with the operands' type: f(ActConst<...>{}, BoolConst<fp16>{}).  Tested per value, the type costs a
// branch per conversion.
template <bool kValue>
struct BoolConst {
  static constexpr bool value = kValue;
};
template <typename F>
__host__ __device__ __forceinline__ void with_act(int act, bool fp16, F&& f) {
  if (fp16) with_act(act, [&](auto a) { f(a, BoolConst<true>{}); });
  else with_act(act, [&](auto a) { f(a, BoolConst<false>{}); });
}

// Two FP32 -> two 16-bit values in one word (lo in the low half), round to nearest even.
__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool fp16) {
  if (fp16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ float2 unpack16(uint32_t w, bool fp16) {
  if (fp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

}  // namespace nvfp4moe
