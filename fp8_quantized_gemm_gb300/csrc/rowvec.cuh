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

// 16 values -> 16 codes.
template <int F>
__device__ __forceinline__ uint4 pack16(const F2 (&y)[8]) {
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i].get(a[2 * i], a[2 * i + 1]);
    y[i + 4].get(b[2 * i], b[2 * i + 1]);
  }
  const uint2 lo = pack8<F>(a), hi = pack8<F>(b);
  return make_uint4(lo.x, lo.y, hi.x, hi.y);
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
  // the exact quotients' codes under a scale formed from an amax that covers them
  template <int F>
  __device__ __forceinline__ uint4 codes(const ScaleDiv &d) const {
    uint2 lo, hi;
    if (d.fast) {
      lo = quant8_own_scale<F>(r[0], d);
      hi = quant8_own_scale<F>(r[1], d);
    } else {
      lo = quant8_ieee<F>(r[0], d);
      hi = quant8_ieee<F>(r[1], d);
    }
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
