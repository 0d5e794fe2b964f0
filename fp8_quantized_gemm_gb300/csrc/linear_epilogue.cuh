// The linear layer's epilogue, applied to a GEMM's scaled fp32 results before
// they leave the chip:
//
//   forward   z = result + bias;  pre <- bf16(z);  y = act(z) + residual;
//             c <- y in its type, q <- FP8 codes of y / q_scale, amax <- max |y|
//   gradient  y = result * act'(pre);  c, q, amax as above;
//             bias gradient: column sums of y over 32-row pieces
//
// Everything is formed in fp32 and rounded once per stored copy.  A thread
// holds 32 neighbouring columns of one row (the TMEM lane layout), so its
// operands are whole 32-byte sectors of that row; they are fetched a chunk
// ahead as raw words (RowIn) while the accumulator is still being waited for.
#pragma once

#include <type_traits>

#include "activation.cuh"
#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"
#include "quant_common.cuh"

namespace fp8k {

// Kernel parameter of the variants with (true) and without (false) the
// epilogue.
template <bool EPI>
struct EpParam {};
template <>
struct EpParam<true> {
  LinearEp e;
};

// 32 operand values of one row, undecoded: 16 words of bf16 pairs or 32 of fp32.
struct RowIn {
  uint32_t w[32];
};

// The row operand of the epilogue: pre (gradient) or residual (forward).
template <bool GRAD>
__device__ __forceinline__ void fetch_row32(const GemmArgs &a, const LinearEp &e, int64_t row,
                                            int64_t col0, RowIn &in) {
  const bool f32 = !GRAD && e.res_dt == 0;
  const void *src = GRAD ? static_cast<const void *>(e.pre) : e.res;
  if (src == nullptr || row >= a.M || col0 >= a.N) return;
  const int64_t off = row * (GRAD ? e.ld_pre : e.ld_res) + col0;
  const bool full = col0 + 32 <= a.N && (GRAD ? e.pre_vec : e.res_vec);
  if (!f32) {
    const uint16_t *p = static_cast<const uint16_t *>(src) + off;
    if (full) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
        in.w[4 * i] = u.x; in.w[4 * i + 1] = u.y; in.w[4 * i + 2] = u.z; in.w[4 * i + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t lo = col0 + 2 * i < a.N ? p[2 * i] : 0u;
        const uint32_t hi = col0 + 2 * i + 1 < a.N ? p[2 * i + 1] : 0u;
        in.w[i] = lo | hi << 16;
      }
    }
  } else {
    const uint32_t *p = static_cast<const uint32_t *>(src) + off;
    if (full) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
        in.w[4 * i] = u.x; in.w[4 * i + 1] = u.y; in.w[4 * i + 2] = u.z; in.w[4 * i + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) in.w[i] = col0 + i < a.N ? p[i] : 0u;
    }
  }
}

__device__ __forceinline__ float bf16_of(const RowIn &in, int i) {
  return __uint_as_float(i & 1 ? in.w[i >> 1] & 0xFFFF0000u : in.w[i >> 1] << 16);
}

// 32 bf16 values of one row
__device__ __forceinline__ void put_bf16x32(__nv_bfloat16 *dst, bool full, int64_t n,
                                            const float (&v)[32]) {
  if (full) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<uint4 *>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < n) dst[i] = __float2bfloat16_rn(v[i]);
  }
}

// c, codes and running max |y| of 32 finished values of one row
__device__ __forceinline__ void put_row32(const GemmArgs &a, const LinearEp &e, int64_t row,
                                          int64_t col0, const float (&v)[32], const ScaleDiv &d,
                                          uint32_t &key) {
  const bool whole = col0 + 32 <= a.N;
  if (a.c != nullptr) {
    if (a.out_dt == 1) {
      put_bf16x32(static_cast<__nv_bfloat16 *>(a.c) + row * a.ldc + col0, whole && a.vec_store,
                  a.N - col0, v);
    } else {
      float *dst = static_cast<float *>(a.c) + row * a.ldc + col0;
      if (whole && a.vec_store) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          reinterpret_cast<float4 *>(dst)[i] =
              make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (col0 + i < a.N) dst[i] = v[i];
      }
    }
  }
  if (e.q == nullptr) return;
  if (e.q_amax != nullptr) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (whole || col0 + i < a.N) key = max(key, abs_key(v[i]));
  }
  uint8_t *q = e.q + row * a.N + col0;
  uint2 c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float y[8];
    div8(d, v + 8 * j, y);
    c[j] = pack8(e.q_fmt, y);
  }
  if (whole && e.q_vec) {
    reinterpret_cast<uint4 *>(q)[0] = make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
    reinterpret_cast<uint4 *>(q)[1] = make_uint4(c[2].x, c[2].y, c[3].x, c[3].y);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t w = (i & 4) ? c[i >> 3].y : c[i >> 3].x;
      if (col0 + i < a.N) q[i] = (uint8_t)(w >> (8 * (i & 3)));
    }
  }
}

// Forward epilogue of 32 columns of one row (v: the scaled results; in: the
// residual of fetch_row32).
__device__ __forceinline__ void linear_row32(const GemmArgs &a, const LinearEp &e, int64_t row,
                                             int64_t col0, float (&v)[32], const RowIn &in,
                                             const ScaleDiv &d, uint32_t &key) {
  if (row >= a.M || col0 >= a.N) return;
  if (a.bias != nullptr) {
    if (col0 + 32 <= a.N && (reinterpret_cast<uintptr_t>(a.bias + col0) & 15u) == 0) {
      const float4 *b4 = reinterpret_cast<const float4 *>(a.bias + col0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 b = __ldg(b4 + i);
        v[4 * i] += b.x; v[4 * i + 1] += b.y; v[4 * i + 2] += b.z; v[4 * i + 3] += b.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (col0 + i < a.N) v[i] += __ldg(a.bias + col0 + i);
    }
  }
  if (e.pre != nullptr)
    put_bf16x32(static_cast<__nv_bfloat16 *>(e.pre) + row * e.ld_pre + col0,
                col0 + 32 <= a.N && e.pre_vec, a.N - col0, v);
  with_act(e.act, [&](auto act) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = act_value<decltype(act)::value>(v[i]);
  });
  if (e.res != nullptr) {
    if (e.res_dt == 0) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += __uint_as_float(in.w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += bf16_of(in, i);
    }
  }
  put_row32(a, e, row, col0, v, d, key);
}

// Gradient epilogue.  Every lane of the warp calls it (rows row0 + lane); the
// sums of the warp's 32 rows go to part[row0 / 32][col0 + lane] by a
// transposing reduction: at each of five steps a lane passes on the half of
// its columns that it does not keep.
__device__ __forceinline__ void grad_row32(const GemmArgs &a, const LinearEp &e, int64_t row0,
                                           int64_t col0, float (&v)[32], const RowIn &in,
                                           const ScaleDiv &d, uint32_t &key) {
  const uint32_t lane = lane_id();
  const int64_t row = row0 + lane;
  if (row0 >= a.M || col0 >= a.N) return;  // the same for the whole warp
  if (row < a.M) {
    with_act(e.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= act_slope<decltype(act)::value>(bf16_of(in, i));
    });
    put_row32(a, e, row, col0, v, d, key);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0.0f;
  }
  if (e.part == nullptr) return;
  __syncwarp();
#pragma unroll
  for (int h = 16; h > 0; h >>= 1) {
    const bool upper = (lane & h) != 0;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float give = upper ? v[i] : v[i + h];
      const float keep = upper ? v[i + h] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, h);
    }
  }
  if (col0 + lane < a.N) e.part[(row0 >> 5) * a.N + col0 + lane] = v[0];
}

// pre, activation and residual of one value z = result + bias: returns y.
__device__ __forceinline__ float linear_value(const LinearEp &e, int64_t row, int64_t col, float z) {
  if (e.pre != nullptr)
    static_cast<__nv_bfloat16 *>(e.pre)[row * e.ld_pre + col] = __float2bfloat16_rn(z);
  with_act(e.act, [&](auto act) { z = act_value<decltype(act)::value>(z); });
  if (e.res != nullptr) {
    const int64_t at = row * e.ld_res + col;
    z += e.res_dt == 0 ? static_cast<const float *>(e.res)[at]
                       : __bfloat162float(static_cast<const __nv_bfloat16 *>(e.res)[at]);
  }
  return z;
}

// Forward epilogue of up to four columns of one row (the split-K reductions).
__device__ __forceinline__ void linear4(const GemmArgs &a, const LinearEp &e, int64_t row,
                                        int64_t col, int n, float (&v)[4], const ScaleDiv &d,
                                        uint32_t &key) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= n) continue;
    float z = v[i];
    if (a.bias != nullptr) z += __ldg(a.bias + col + i);
    z = linear_value(e, row, col + i, z);
    if (a.c != nullptr) {
      if (a.out_dt == 1)
        static_cast<__nv_bfloat16 *>(a.c)[row * a.ldc + col + i] = __float2bfloat16_rn(z);
      else
        static_cast<float *>(a.c)[row * a.ldc + col + i] = z;
    }
    if (e.q != nullptr) {
      key = max(key, abs_key(z));
      const float y = d.fast ? d.div<true>(z) : d.div<false>(z);
      e.q[row * a.N + col + i] = (uint8_t)cvt_fp8x2(e.q_fmt, y, 0.0f);
    }
  }
}

// The CTA's running max |y| (any warp; every lane calls).
__device__ __forceinline__ void flush_amax(const LinearEp &e, uint32_t key) {
  if (e.q == nullptr || e.q_amax == nullptr) return;
  key = warp_max_u32(key);
  if (lane_id() == 0 && key != 0u) atomicMax(e.q_amax, key);
}

__device__ __forceinline__ ScaleDiv epilogue_scale(const LinearEp &e) {
  return ScaleDiv(e.q != nullptr ? *e.q_scale : 1.0f);
}

}  // namespace fp8k
