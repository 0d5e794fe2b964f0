// Pairs of fp32 values: products, sums and fmas as packed f32x2 instructions
// (each half rounded as the scalar instruction), and what the norms and the
// linear epilogue do with them on the way to FP8 codes.
#pragma once

#include "common.cuh"

namespace fp8k {

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// A packed pair of fp32 values.
struct F2 {
  uint64_t v;
  __device__ __forceinline__ F2() : v(0) {}
  __device__ __forceinline__ F2(uint64_t x) : v(x) {}
  __device__ __forceinline__ F2(float a, float b) : v(f32x2_pack(a, b)) {}
  __device__ __forceinline__ explicit F2(float a) : v(f32x2_pack(a, a)) {}
  __device__ __forceinline__ void get(float &a, float &b) const { f32x2_unpack(v, a, b); }
};
__device__ __forceinline__ F2 operator*(F2 a, F2 b) { return f32x2_mul(a.v, b.v); }
__device__ __forceinline__ F2 operator+(F2 a, F2 b) { return f32x2_add(a.v, b.v); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) { return f32x2_fma(a.v, b.v, c.v); }
template <typename Fn>
__device__ __forceinline__ F2 each(F2 a, Fn &&f) {
  float x, y;
  a.get(x, y);
  return F2(f(x), f(y));
}

__device__ __forceinline__ F2 bf16_pair(uint32_t w) {
  return F2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t to_bf16_pair(F2 v) {
  float a, b;
  v.get(a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Running max |x| (a NaN stays one, above every number as an integer).
__device__ __forceinline__ float max_abs2(float m, F2 v) {
  float a, b;
  v.get(a, b);
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return m;
}

// The codes' scale.  The quotient y / s is formed as y times the correctly
// rounded reciprocal of s where that is a normal number, and by division
// elsewhere: y is an fp32 result with a rounding of its own, which the exact
// quotient's last bit does not sharpen, and the exact quotient of the
// standalone quantizers costs six more instructions per element (57 of 757 us
// on the 16384 x 14336 x 4096 product with codes; it bound the 16384 x 4096
// norm at 68 us of arithmetic).
struct CodeScale {
  float s, inv;
  bool fast;
  __device__ __forceinline__ explicit CodeScale(float scale) {
    s = scale;
    inv = __frcp_rn(s);
    fast = s >= 0x1p-120f && s <= 0x1p120f;
  }
  __device__ __forceinline__ F2 quotient(F2 y) const {
    if (fast) return y * F2(inv);
    return each(y, [this](float x) { return __fdiv_rn(x, s); });
  }
};

}  // namespace fp8k
