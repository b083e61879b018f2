// The nonlinearities of taco_linear.h on the device, and their slopes, in fp32.
//
// Each keeps a NaN and takes its limits at the infinities: the factor that
// meets a vanishing one is held at a magnitude from which on that is 0.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "taco_linear.h"

namespace {

// 2^x and 1 / x are the hardware's, to one unit in the last place.  Where x
// comes from a product its rounding grows with it: a relative error of at most
// (|x| + 4) 2^-24 in all.
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float over_one(float x) { return __builtin_amdgcn_rcpf(x); }

constexpr float kLog2E = 1.44269504f;

// 1 / (1 + 2^-x); 2^-x may be infinite.
__device__ __forceinline__ float sigmoid2(float x) { return over_one(1.0f + exp2_of(-x)); }

// The normal distribution function at -a, 0 <= a <= 40, and its density: a
// polynomial in s = 1 / (1 + 0.31 a) times exp(-a^2 / 2), fitted so that the
// largest relative error over a <= 14 is least: 1.6e-7, and under 6e-7 as it is
// evaluated here, besides the exponential's.  Beyond 14 it is under 2^-146.
__device__ __forceinline__ void normal_tail(float a, float& tail, float& density) {
  const float s = over_one(fmaf(0.31f, a, 1.0f)), e = exp2_of(a * a * (-0.5f * kLog2E));
  float p = fmaf(0.035841189f, s, -0.14160217f);
  p = fmaf(p, s, 0.15506335f);
  p = fmaf(p, s, -0.014898892f);
  p = fmaf(p, s, 0.11010755f);
  p = fmaf(p, s, 0.10777194f);
  p = fmaf(p, s, 0.12406019f);
  p = fmaf(p, s, 0.12365692f);
  tail = p * s * e;
  density = 0.39894228f * e;
}

// 2 sqrt(2 / pi) (t + 0.044715 t^3) log2(e), so that (1 + tanh(..)) / 2 is its sigmoid2.
__device__ __forceinline__ float tanh_argument(float t) { return t * fmaf(t * t, 0.10294324f, 2.3022082f); }

template <int ACT>
__device__ __forceinline__ float activate(float t) {
  if constexpr (ACT == TACO_ACT_RELU) return __builtin_elementwise_maximum(t, 0.0f);      // of a NaN: NaN
  if constexpr (ACT == TACO_ACT_GELU) {            // t P(t) = max(t, 0) - |t| P(-|t|)
    float tail, density;
    const float a = fminf(fabsf(t), 40.0f);
    normal_tail(a, tail, density);
    return fmaf(-a, tail, __builtin_elementwise_maximum(t, 0.0f));
  }
  if constexpr (ACT == TACO_ACT_GELU_TANH) return fmaxf(t, -40.0f) * sigmoid2(tanh_argument(t));
  if constexpr (ACT == TACO_ACT_SILU) return fmaxf(t, -128.0f) * sigmoid2(kLog2E * t);
  return t;
}

template <int ACT>
__device__ __forceinline__ float slope(float t) {
  if constexpr (ACT == TACO_ACT_NONE) return 1.0f;
  float v = t > 0.0f ? 1.0f : 0.0f;
  if constexpr (ACT == TACO_ACT_GELU) {            // P(t) + t p(t)
    float tail, density;
    const float a = fminf(fabsf(t), 40.0f);
    normal_tail(a, tail, density);
    const float up = fmaf(a, density, -tail);      // P(a) + a p(a) - 1
    v = t < 0.0f ? -up : 1.0f + up;
  } else if constexpr (ACT == TACO_ACT_GELU_TANH) {
    const float x = fminf(fmaxf(t, -40.0f), 40.0f), s = sigmoid2(tanh_argument(x));
    v = s * fmaf(x * (1.0f - s), fmaf(x * x, 0.21406446f, 1.5957691f), 1.0f);
  } else if constexpr (ACT == TACO_ACT_SILU) {
    const float x = fminf(fmaxf(t, -128.0f), 128.0f), s = sigmoid2(kLog2E * x);
    v = s * fmaf(x, 1.0f - s, 1.0f);
  }
  return t != t ? t : v;
}

// f(integral_constant) of the activation that a call names; uniform over the launch.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F f) {
  if (act == TACO_ACT_NONE) f(std::integral_constant<int, TACO_ACT_NONE>{});
  else if (act == TACO_ACT_RELU) f(std::integral_constant<int, TACO_ACT_RELU>{});
  else if (act == TACO_ACT_GELU) f(std::integral_constant<int, TACO_ACT_GELU>{});
  else if (act == TACO_ACT_GELU_TANH) f(std::integral_constant<int, TACO_ACT_GELU_TANH>{});
  else f(std::integral_constant<int, TACO_ACT_SILU>{});
}

inline bool activation_ok(int32_t act) { return act >= TACO_ACT_NONE && act <= TACO_ACT_SILU; }

}  // namespace
