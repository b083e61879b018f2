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

// Values are taken some at a time, and each step of a formula for all of them
// before the next: the steps of one value wait for each other, the hardware's
// exponential and reciprocal longest, and the compiler left to itself puts one
// value's behind another's (the scheduling barriers hold it off that).
__device__ __forceinline__ void next_step() { __builtin_amdgcn_sched_barrier(0); }

// P(-a), the normal distribution function, 0 <= a <= 20: its binary logarithm as
// a polynomial of a, no reciprocal and one exponential; 2/3 of the instructions of
// the form below, and the epilogue of a large product is bound by them.  Fitted
// so that the result's relative error over (4 w + 24) 2^-24 2^max(0, a - 1), w = a^2
// / 2, is least, which lets it grow where a P(-a) vanishes: 1.52, and 1.65 as it
// is evaluated here.  Beyond 14 it is under 2^-147.
template <int N>
__device__ __forceinline__ void normal_tail(const float (&a)[N], float (&tail)[N]) {
  constexpr float kPoly[] = {3.1970519e-08f, -2.3084929e-06f, 6.2982836e-05f, -9.2093681e-04f, 8.4395139e-03f,
                             -5.3809188e-02f, -4.5859540e-01f, -1.1512135e+00f, -9.9999689e-01f};
#pragma unroll
  for (int j = 0; j < N; ++j) tail[j] = kPoly[0];
#pragma unroll
  for (int i = 1; i < 9; ++i) {
#pragma unroll
    for (int j = 0; j < N; ++j) tail[j] = fmaf(tail[j], a[j], kPoly[i]);
    next_step();
  }
#pragma unroll
  for (int j = 0; j < N; ++j) tail[j] = exp2_of(tail[j]);
}

// P(-a) and exp(-a^2 / 2), 0 <= a <= 40: a
// polynomial in s = 1 / (1 + 0.31 a) times the latter, fitted so that the largest
// relative error over a <= 14 is least: 1.6e-7, and under 6e-7 as it is
// evaluated here, besides the exponential's.  Beyond 14 it is under 2^-146.
template <int N>
__device__ __forceinline__ void normal_tail(const float (&a)[N], float (&tail)[N], float (&e)[N]) {
  constexpr float kPoly[] = {0.035841189f, -0.14160217f, 0.15506335f, -0.014898892f,
                             0.11010755f,  0.10777194f,  0.12406019f, 0.12365692f};
  float s[N];
#pragma unroll
  for (int j = 0; j < N; ++j) s[j] = fmaf(0.31f, a[j], 1.0f);
#pragma unroll
  for (int j = 0; j < N; ++j) e[j] = a[j] * a[j];
  next_step();
#pragma unroll
  for (int j = 0; j < N; ++j) s[j] = over_one(s[j]);
#pragma unroll
  for (int j = 0; j < N; ++j) e[j] *= -0.5f * kLog2E;
  next_step();
#pragma unroll
  for (int j = 0; j < N; ++j) e[j] = exp2_of(e[j]);
#pragma unroll
  for (int j = 0; j < N; ++j) tail[j] = kPoly[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    next_step();
#pragma unroll
    for (int j = 0; j < N; ++j) tail[j] = fmaf(tail[j], s[j], kPoly[i]);
  }
  next_step();
#pragma unroll
  for (int j = 0; j < N; ++j) s[j] *= e[j];
#pragma unroll
  for (int j = 0; j < N; ++j) tail[j] *= s[j];
}

// 2 sqrt(2 / pi) (t + 0.044715 t^3) log2(e), so that (1 + tanh(..)) / 2 is its sigmoid2.
__device__ __forceinline__ float tanh_argument(float t) { return t * fmaf(t * t, 0.10294324f, 2.3022082f); }

// 1 / (1 + 2^-x); 2^-x may be infinite.
template <int N>
__device__ __forceinline__ void sigmoid2(const float (&x)[N], float (&s)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) s[j] = exp2_of(-x[j]);
  next_step();
#pragma unroll
  for (int j = 0; j < N; ++j) s[j] += 1.0f;
  next_step();
#pragma unroll
  for (int j = 0; j < N; ++j) s[j] = over_one(s[j]);
  next_step();
}

// (`minimum` and `maximum` of a NaN are NaN, unlike fminf and fmaxf.)
template <int ACT, int N>
__device__ __forceinline__ void activate(float (&t)[N]) {
  if constexpr (ACT == TACO_ACT_RELU) {
#pragma unroll
    for (int j = 0; j < N; ++j) t[j] = __builtin_elementwise_maximum(t[j], 0.0f);
  } else if constexpr (ACT == TACO_ACT_GELU) {     // t P(t) = max(t, 0) - |t| P(-|t|)
    float a[N], tail[N];
#pragma unroll
    for (int j = 0; j < N; ++j) a[j] = __builtin_elementwise_minimum(__builtin_fabsf(t[j]), 20.0f);
    normal_tail(a, tail);
#pragma unroll
    for (int j = 0; j < N; ++j) t[j] = fmaf(-a[j], tail[j], __builtin_elementwise_maximum(t[j], 0.0f));
  } else if constexpr (ACT == TACO_ACT_GELU_TANH || ACT == TACO_ACT_SILU) {
    constexpr float kLeast = ACT == TACO_ACT_SILU ? -128.0f : -40.0f;
    float x[N], s[N];
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = ACT == TACO_ACT_SILU ? kLog2E * t[j] : tanh_argument(t[j]);
    sigmoid2(x, s);
#pragma unroll
    for (int j = 0; j < N; ++j) t[j] = __builtin_elementwise_maximum(t[j], kLeast) * s[j];
  }
}

// t becomes the slope there.
template <int ACT, int N>
__device__ __forceinline__ void slope(float (&t)[N]) {
  float v[N];
  if constexpr (ACT == TACO_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < N; ++j) t[j] = 1.0f;
  } else if constexpr (ACT == TACO_ACT_RELU) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = t[j] > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == TACO_ACT_GELU) {     // P(t) + t p(t)
    float a[N], tail[N], e[N];
#pragma unroll
    for (int j = 0; j < N; ++j) a[j] = __builtin_elementwise_minimum(__builtin_fabsf(t[j]), 40.0f);
    normal_tail(a, tail, e);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float up = fmaf(a[j] * 0.39894228f, e[j], -tail[j]);      // P(a) + a p(a) - 1
      v[j] = t[j] < 0.0f ? -up : 1.0f + up;
    }
  } else {
    constexpr float kMost = ACT == TACO_ACT_SILU ? 128.0f : 40.0f;
    float x[N], z[N], s[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      x[j] = fminf(fmaxf(t[j], -kMost), kMost);
      z[j] = ACT == TACO_ACT_SILU ? kLog2E * x[j] : tanh_argument(x[j]);
    }
    sigmoid2(z, s);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float steep = ACT == TACO_ACT_SILU ? 1.0f : fmaf(x[j] * x[j], 0.21406446f, 1.5957691f);
      v[j] = s[j] * fmaf(x[j] * (1.0f - s[j]), steep, 1.0f);
    }
  }
  if constexpr (ACT != TACO_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < N; ++j) t[j] = t[j] != t[j] ? t[j] : v[j];
  }
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
