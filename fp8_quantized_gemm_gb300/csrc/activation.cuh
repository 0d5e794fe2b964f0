// Activations of the linear layer's epilogue and their derivatives, in fp32
// from the formulas, on the hardware base-2 exponential and reciprocal (each
// within about 2^-22 of the exact value; the results are rounded to 8
// significant bits or fewer, or feed fp32 sums at that accuracy).
//
//   relu  max(z, 0)       relu2  max(z, 0)^2       silu  z s(z)
//   gelu  z Phi(z)        gelu, tanh form  z s(2 sqrt(2/pi) (z + 0.044715 z^3))
//
// with s(z) = 1 / (1 + e^-z); the tanh form uses (1 + tanh u) / 2 = s(2u), so
// that its left tail keeps its relative accuracy.  A NaN stays a NaN; at an
// infinite z (finite values near the top of fp32 are infinite in a bf16
// pre-activation) every function and slope takes its limit: a factor that has
// vanished there never meets an infinite one.
//
// Two values at a time: the products and sums are packed f32x2 instructions
// (each half rounded as the scalar instruction), which halves what the
// epilogue issues.  These GEMMs run at the board's power limit, where every
// instruction per output element costs clock: the GELU product of 16384 x
// 14336 x 4096 took 757 us with scalar arithmetic and IEEE quotients.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "elementwise.cuh"
#include "pairs.cuh"

namespace fp8k {

enum Act : int { kActNone = 0, kActRelu = 1, kActRelu2 = 2, kActSilu = 3, kActGeluTanh = 4, kActGelu = 5 };

// 1 / x; a subnormal result becomes zero (x > 2^126: a vanished logistic value)
__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ F2 exp2_2(F2 a) { return each(a, [](float x) { return ex2_approx_ftz(x); }); }
__device__ __forceinline__ F2 rcp_2(F2 a) { return each(a, [](float x) { return rcp_ftz(x); }); }
__device__ __forceinline__ F2 relu_2(F2 a) { return each(a, [](float x) { return max_nan(x, 0.0f); }); }

// Bounds beyond which the logistic function and the normal tail are 0 or 1 in
// fp32 (from |z| = 150 on) while z and z^3 are far from overflow.
constexpr float kFar = 1e4f, kFarCubed = 1e3f;
// z within [-b, b], one instruction: min(|z|, b) with the sign of z (b > 0)
__device__ __forceinline__ F2 within_2(F2 a, float b) {
  return each(a, [b](float x) {
    float r;
    asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(b));
    return r;
  });
}
// z where its logistic factor is not zero yet
__device__ __forceinline__ F2 left_capped(F2 a) {
  return each(a, [](float x) { return max_nan(x, -kFar); });
}

// s(-t / log2 e) = 1 / (1 + 2^t)
__device__ __forceinline__ F2 logistic2(F2 t) { return rcp_2(exp2_2(t) + F2(1.0f)); }

// -2 sqrt(2/pi) log2 e and its product with 0.044715: the exponent of the
// tanh form's logistic function is t = z (kT1 + kT3 z^2)
constexpr float kT1 = -2.3022081985175f, kT3 = -0.10294323959671f;
// 2 sqrt(2/pi) and 3 x 0.044715 of it: d/dz of its argument
constexpr float kD1 = 1.5957691216057308f, kD3 = 0.21406444881478f;

// E = e^(-z^2/2), a = |z| (at most kFar, where E is 0) and
// Phi(-a) / E = erfcx(a / sqrt 2) / 2, which is t times a degree-8 polynomial
// in t = 1 / (1 + 0.4 a / sqrt 2) (least squares on Chebyshev nodes with the
// weights driven to equal relative error: 1.6e-7 with the coefficients as
// rounded here, over t in (0, 1], that is for every z).
__device__ __forceinline__ F2 normal_tail(F2 z, F2 &a, F2 &E) {
  a = each(z, [](float x) { return fminf(fabsf(x), kFar); });  // (E keeps a NaN)
  E = exp2_2(z * z * F2(-0.72134752044448170f));
  const F2 t = rcp_2(fma2(a, F2(0.28284271247461901f), F2(1.0f)));
  F2 p(0.025127250701189041f);
  p = fma2(p, t, F2(-0.091437287628650665f));
  p = fma2(p, t, F2(0.084523670375347137f));
  p = fma2(p, t, F2(-0.0027899211272597313f));
  p = fma2(p, t, F2(0.070710234344005585f));
  p = fma2(p, t, F2(0.084272146224975586f));
  p = fma2(p, t, F2(0.10392123460769653f));
  p = fma2(p, t, F2(0.11283480376005173f));
  p = fma2(p, t, F2(0.11283793300390244f));
  return p * t;
}

template <int A>
__device__ __forceinline__ F2 act_value2(F2 z) {
  if constexpr (A == kActRelu) return relu_2(z);
  if constexpr (A == kActRelu2) {
    const F2 p = relu_2(z);
    return p * p;
  }
  if constexpr (A == kActSilu) return left_capped(z) * logistic2(z * F2(kNegLog2e));
  if constexpr (A == kActGeluTanh)
    return left_capped(z) * logistic2(z * fma2(z * z, F2(kT3), F2(kT1)));
  if constexpr (A == kActGelu) {
    // z Phi(z) = max(z, 0) - |z| Phi(-|z|)
    F2 a(0.0f), E(0.0f);
    const F2 q = normal_tail(z, a, E);
    return fma2(a * F2(-1.0f), E * q, relu_2(z));
  }
  return z;
}

// The derivative (z bounded where the slope is 0 or 1: see above).
template <int A>
__device__ __forceinline__ F2 act_slope2(F2 z) {
  if constexpr (A == kActRelu)
    return each(z, [](float x) { return x > 0.0f ? 1.0f : (x == x ? 0.0f : x); });
  if constexpr (A == kActRelu2) {
    const F2 p = relu_2(z);
    return p + p;
  }
  if constexpr (A == kActSilu) {
    const F2 b = within_2(z, kFar), s = logistic2(b * F2(kNegLog2e));
    return s * fma2(b, fma2(s, F2(-1.0f), F2(1.0f)), F2(1.0f));
  }
  if constexpr (A == kActGeluTanh) {
    const F2 b = within_2(z, kFarCubed), bb = b * b;
    const F2 s = logistic2(b * fma2(bb, F2(kT3), F2(kT1)));
    return fma2(b * s, fma2(s, F2(-1.0f), F2(1.0f)) * fma2(bb, F2(kD3), F2(kD1)), s);
  }
  if constexpr (A == kActGelu) {
    // Phi(z) + z phi(z) = u for z < 0 and 1 - u otherwise, with
    // u = Phi(-|z|) - |z| phi(z) = E (q - |z| / sqrt(2 pi))
    F2 a(0.0f), E(0.0f);
    const F2 q = normal_tail(z, a, E);
    const F2 u = E * fma2(a, F2(-0.39894228040143268f), q);
    float u0, u1, z0, z1;
    u.get(u0, u1);
    z.get(z0, z1);
    return F2(z0 < 0.0f ? u0 : 1.0f - u0, z1 < 0.0f ? u1 : 1.0f - u1);
  }
  return F2(1.0f);
}

// Calls f with the activation as a compile-time constant (one uniform branch
// per call, outside the loop over values); for kActNone only with NONE.
template <bool NONE = false, typename Fn>
__device__ __forceinline__ void with_act(int act, Fn &&f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActRelu2: f(std::integral_constant<int, kActRelu2>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    default:
      if constexpr (NONE) f(std::integral_constant<int, kActNone>{});
      break;
  }
}

}  // namespace fp8k
