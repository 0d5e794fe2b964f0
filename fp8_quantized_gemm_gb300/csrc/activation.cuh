// Activations of the linear layer's epilogue and their derivatives, in fp32
// from the formulas, on the hardware base-2 exponential and reciprocal (each
// within about 2^-22 of the exact value; the results are rounded to 8
// significant bits or fewer, or feed fp32 sums at that accuracy).
//
//   relu  max(z, 0)       relu2  max(z, 0)^2       silu  z s(z)
//   gelu  z Phi(z)        gelu, tanh form  z s(2 sqrt(2/pi) (z + 0.044715 z^3))
//
// with s(z) = 1 / (1 + e^-z); the tanh form uses (1 + tanh u) / 2 = s(2u), so
// that its left tail keeps its relative accuracy.  A NaN stays a NaN.
#pragma once

#include "common.cuh"
#include "elementwise.cuh"

namespace fp8k {

enum Act : int { kActNone = 0, kActRelu = 1, kActRelu2 = 2, kActSilu = 3, kActGeluTanh = 4, kActGelu = 5 };

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 2 sqrt(2/pi) and its product with 0.044715
constexpr float kGeluC1 = 1.5957691216057308f, kGeluC3 = 0.07135481627159726f;

// Phi(z), the normal distribution function, and E = e^(-z^2/2): with
// x = |z| / sqrt 2 the tail is Phi(-|z|) = E erfcx(x) / 2, and erfcx(x) / 2
// is t times a degree-8 polynomial in t = 1 / (1 + 0.4 x) (least squares on
// Chebyshev nodes with the weights driven to equal relative error: 1.3e-7
// over t in (0, 1], that is for every z).
__device__ __forceinline__ float normal_cdf(float z, float &E) {
  E = ex2_approx_ftz(__fmul_rn(__fmul_rn(z, z), -0.72134752044448170f));
  const float t = rcp_approx(__fmaf_rn(fabsf(z), 0.28284271247461901f, 1.0f));
  float p = 0.025127250701189041f;
  p = __fmaf_rn(p, t, -0.091437287628650665f);
  p = __fmaf_rn(p, t, 0.084523670375347137f);
  p = __fmaf_rn(p, t, -0.0027899211272597313f);
  p = __fmaf_rn(p, t, 0.070710234344005585f);
  p = __fmaf_rn(p, t, 0.084272146224975586f);
  p = __fmaf_rn(p, t, 0.10392123460769653f);
  p = __fmaf_rn(p, t, 0.11283480376005173f);
  p = __fmaf_rn(p, t, 0.11283793300390244f);
  const float tail = __fmul_rn(E, __fmul_rn(p, t));
  return z < 0.0f ? tail : 1.0f - tail;
}

template <int A>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (A == kActRelu) return max_nan(z, 0.0f);
  if constexpr (A == kActRelu2) {
    const float p = max_nan(z, 0.0f);
    return __fmul_rn(p, p);
  }
  if constexpr (A == kActSilu) return __fmul_rn(z, sigmoidf_(z));
  if constexpr (A == kActGeluTanh)
    return __fmul_rn(z, sigmoidf_(__fmul_rn(z, __fmaf_rn(kGeluC3, __fmul_rn(z, z), kGeluC1))));
  if constexpr (A == kActGelu) {
    float E;
    return __fmul_rn(z, normal_cdf(z, E));
  }
  return z;
}

// The derivative.  Beyond |z| = 100 every one of the smooth activations has
// slope 0 or 1 in fp32: z is clamped there, so that no product of a vanished
// factor and an overflowed one is formed.
template <int A>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (A == kActRelu) return z > 0.0f ? 1.0f : (z == z ? 0.0f : z);
  if constexpr (A == kActRelu2) return 2.0f * max_nan(z, 0.0f);
  if constexpr (A == kActNone) return 1.0f;
  const float c = max_nan(min_nan(z, 100.0f), -100.0f);
  if constexpr (A == kActSilu) {
    const float s = sigmoidf_(c);
    return __fmul_rn(s, __fmaf_rn(c, 1.0f - s, 1.0f));
  }
  if constexpr (A == kActGeluTanh) {
    const float zz = __fmul_rn(c, c);
    const float s = sigmoidf_(__fmul_rn(c, __fmaf_rn(kGeluC3, zz, kGeluC1)));
    const float du = __fmaf_rn(3.0f * kGeluC3, zz, kGeluC1);
    return __fmaf_rn(__fmul_rn(c, s), __fmul_rn(1.0f - s, du), s);
  }
  float E;
  const float cdf = normal_cdf(c, E);
  return __fmaf_rn(__fmul_rn(c, E), 0.39894228040143268f, cdf);
}

// Calls f with the activation as a compile-time constant (one uniform branch
// per call, outside the loop over values).
template <typename Fn>
__device__ __forceinline__ void with_act(int act, Fn &&f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActRelu2: f(std::integral_constant<int, kActRelu2>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    default: break;
  }
}

}  // namespace fp8k
