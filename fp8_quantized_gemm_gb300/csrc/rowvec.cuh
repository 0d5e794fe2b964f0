// Runs of 16 consecutive elements of a row per lane, eight lanes to a 1x128
// group: what the expert-row and checkpoint kernels load, quantize and store.
#pragma once

#include "common.cuh"
#include "pairs.cuh"
#include "quant_common.cuh"

namespace fp8k {

// The i-th pair of a raw vector of eight.
template <typename T>
__device__ __forceinline__ F2 raw_pair(const Raw8<T> &r, int i) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
    return bf16_pair(w[i]);
  } else {
    const uint4 &u = r.w[i >> 1];
    return i & 1 ? F2(__uint_as_float(u.z), __uint_as_float(u.w))
                 : F2(__uint_as_float(u.x), __uint_as_float(u.y));
  }
}

// Four pairs rounded to T.
template <typename T>
__device__ __forceinline__ Raw8<T> round8(const F2 *v) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 2) {
    r.w[0] = make_uint4(to_bf16_pair(v[0]), to_bf16_pair(v[1]), to_bf16_pair(v[2]), to_bf16_pair(v[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float a, b, c, d;
      v[2 * i].get(a, b);
      v[2 * i + 1].get(c, d);
      r.w[i] = make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
    }
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const Raw8<T> &r) {
#pragma unroll
  for (int i = 0; i < Raw8<T>::kWords; ++i) reinterpret_cast<uint4 *>(p)[i] = r.w[i];
}
template <typename T>
__device__ __forceinline__ void store16(T *p, const F2 (&y)[8]) {
  store8(p, round8<T>(y));
  store8(p + 8, round8<T>(y + 4));
}

// Four values -> four codes, packed (the second conversion lands in the upper
// half of the word).
template <int F>
__device__ __forceinline__ uint32_t pack4(F2 lo, F2 hi) {
  float a, b, c, d;
  lo.get(a, b);
  hi.get(c, d);
  uint32_t r;
  if constexpr (F == 0)
    asm("{ .reg .b16 l, h; cvt.rn.satfinite.e4m3x2.f32 l, %2, %1; "
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3; mov.b32 %0, {l, h}; }"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
  else
    asm("{ .reg .b16 l, h; cvt.rn.satfinite.e5m2x2.f32 l, %2, %1; "
        "cvt.rn.satfinite.e5m2x2.f32 h, %4, %3; mov.b32 %0, {l, h}; }"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
template <int F>
__device__ __forceinline__ uint4 pack16(const F2 (&y)[8]) {
  return make_uint4(pack4<F>(y[0], y[1]), pack4<F>(y[2], y[3]), pack4<F>(y[4], y[5]),
                    pack4<F>(y[6], y[7]));
}

// Asynchronous 16-byte copies to shared memory.
// (bytes 16, or 0: sixteen zero bytes, nothing is read)
__device__ __forceinline__ void copy16_async(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// max of a key over the eight lanes of a group
__device__ __forceinline__ uint32_t group8_max(uint32_t key) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
  return key;
}

// Exponent of the smallest power of two not below amax / MAX, clamped to a
// UE8M0 byte's range (0 for an all-zero or NaN amax: scale 1).
__device__ __forceinline__ int ue8m0_exponent(float amax, float mx) {
  return amax > 0.0f ? min(max(ceil_log2_pos(__fdiv_rn(amax, mx)), -127), 127) : 0;
}

// The scale of a group by its amax, and what its values are multiplied by.  In
// the common range (`fast`: amax zero, or far from the ends of fp32) the scale is
// the correctly rounded amax / MAX by one corrected product (the quotient by a
// constant: q + (amax - MAX q) / MAX with the exact remainder), and the factor
// its reciprocal within an ulp: three instructions and one, where the general
// division and reciprocal take twenty.  Elsewhere (infinities and NaN too) the
// general forms and IEEE quotients, out of line.
struct GroupScale {
  float s, inv;
  uint32_t stored;  // fp32 bits, or the UE8M0 byte
  bool fast;
};
template <int F>
__device__ __forceinline__ GroupScale group_scale(float amax, int sfmt) {
  constexpr float mx = F == 0 ? kE4M3Max : kE5M2Max, r = 1.0f / mx;
  GroupScale g;
  g.fast = amax == 0.0f || (amax >= 0x1p-80f && amax <= 0x1p80f);
  const float q = __fmul_rn(amax, r);
  g.s = amax == 0.0f ? 1.0f : __fmaf_rn(__fmaf_rn(-mx, q, amax), r, q);
  if (sfmt == 0) {
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(g.inv) : "f"(g.s));
    g.stored = __float_as_uint(g.s);
  } else {  // up to a power of two: its byte, and the reciprocal's
    const uint32_t b = __float_as_uint(g.s), e = (b >> 23) + ((b & 0x7FFFFFu) != 0u ? 1u : 0u);
    g.stored = e;
    g.inv = __uint_as_float((254u - e) << 23);
  }
  return g;
}
template <int F>
__device__ __noinline__ GroupScale group_scale_any(float amax, int sfmt) {
  constexpr float mx = F == 0 ? kE4M3Max : kE5M2Max;
  GroupScale g;
  g.fast = false;
  g.inv = 0.0f;
  if (sfmt == 0) {
    g.s = scale_from_amax(amax, mx);
    g.stored = __float_as_uint(g.s);
  } else {
    const int e = ue8m0_exponent(amax, mx);
    g.s = exp2_int(e);
    g.stored = (uint32_t)(e + 127);
  }
  return g;
}
// IEEE quotients' codes of four and of 16 values (operands in registers: an
// array would live in local memory).
template <int F>
__device__ __noinline__ uint32_t codes4_ieee(uint64_t lo, uint64_t hi, float s) {
  auto q = [s](float x) { return __fdiv_rn(x, s); };
  return pack4<F>(each(F2(lo), q), each(F2(hi), q));
}
template <int F>
__device__ __forceinline__ uint4 codes16_any(const F2 (&y)[8], float s) {
  return make_uint4(codes4_ieee<F>(y[0].v, y[1].v, s), codes4_ieee<F>(y[2].v, y[3].v, s),
                    codes4_ieee<F>(y[4].v, y[5].v, s), codes4_ieee<F>(y[6].v, y[7].v, s));
}
// Codes of 16 values times a factor.
template <int F>
__device__ __forceinline__ uint4 codes16_times(const F2 (&y)[8], float factor) {
  const F2 f(factor);
  F2 z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = y[i] * f;
  return pack16<F>(z);
}
__device__ __forceinline__ void store_scale(void *scales, int64_t at, uint32_t stored, int sfmt) {
  if (sfmt == 0)
    static_cast<uint32_t *>(scales)[at] = stored;
  else
    static_cast<uint8_t *>(scales)[at] = (uint8_t)stored;
}

// 16 elements as loaded.
template <typename T>
struct Vec16 {
  Raw8<T> r[2];
  __device__ __forceinline__ void load(const T *p) {
    r[0].load_stream(p);
    r[1].load_stream(p + 8);
  }
  __device__ __forceinline__ void zero() {
    r[0].zero();
    r[1].zero();
  }
  __device__ __forceinline__ void store(T *p) const {
    store8(p, r[0]);
    store8(p + 8, r[1]);
  }
  __device__ __forceinline__ F2 pair(int i) const { return raw_pair(r[i >> 2], i & 3); }
  // max |x| as an fp32 bit pattern
  __device__ __forceinline__ uint32_t max_key() const {
    uint32_t a = 0, b = 0;
    r[0].max_abs(a, b);
    r[1].max_abs(a, b);
    return Raw8<T>::merge_keys(a, b);
  }
  // the exact quotients' codes under a scale of the common range formed from an
  // amax that covers them
  template <int F>
  __device__ __forceinline__ uint4 codes_own(const ScaleDiv &d) const {
    const uint2 lo = quant8_own_scale<F>(r[0], d), hi = quant8_own_scale<F>(r[1], d);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
  // under the power of two 1 / inv
  template <int F>
  __device__ __forceinline__ uint4 codes_pow2(float inv) const {
    const uint64_t inv2 = f32x2_pack(inv, inv);
    const uint2 lo = quant8_pow2<F>(r[0], inv2), hi = quant8_pow2<F>(r[1], inv2);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
};

// 16 codes
template <>
struct Vec16<uint8_t> {
  uint4 w[1];
  __device__ __forceinline__ void load(const uint8_t *p) {
    w[0] = __ldcs(reinterpret_cast<const uint4 *>(p));
  }
  __device__ __forceinline__ void zero() { w[0] = make_uint4(0u, 0u, 0u, 0u); }
};

}  // namespace fp8k
