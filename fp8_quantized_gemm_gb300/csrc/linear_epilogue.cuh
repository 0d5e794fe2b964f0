// The linear layer's epilogue, applied to a GEMM's fp32 accumulators before
// they leave the chip:
//
//   forward   z = alpha acc + bias;  pre <- bf16(z);  y = act(z) + residual;
//             c <- y in its type, q <- FP8 codes of y / q_scale, amax <- max |y|
//   gradient  y = alpha acc act'(pre);  c, q, amax as above;
//             bias gradient: column sums of y over 32-row pieces
//
// Everything is formed in fp32 and rounded once per stored copy.  A warp
// takes a chunk of 32 rows x 32 columns, a lane one row of it (the TMEM lane
// layout).  Where bases and pitches are multiples of 32 bytes a lane reads and
// writes its own row, a whole sector per access; the operands of the next chunk
// are fetched as raw words (RowIn) while this one is worked on.  Any other
// shape passes through 4 KB of the warp's shared memory (its stage), so that
// the warp touches one row's 32 neighbouring elements at a time: with a lane
// per row, each scalar access would touch 32 rows (1000 x 2053 x 2064 with an
// fp32 residual: 42.5 us that way).
#pragma once

#include "activation.cuh"
#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"
#include "pairs.cuh"
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

__device__ __forceinline__ CodeScale code_scale(const LinearEp &e) {
  return CodeScale(e.q != nullptr ? *e.q_scale : 1.0f);
}

constexpr uint32_t kEpStageBytes = 32 * 128;  // per epilogue warp, 16-byte aligned

// 32 bf16 operand values of one row, as pairs.
struct RowIn {
  uint32_t w[16];
};

// Element (r, c) of a 32 x 32 fp32 stage: rows of 128 bytes whose 16-byte
// units are permuted by the row, so that lanes reading or writing their own
// rows in 16-byte units and lanes walking along one row both spread over the
// banks.
__device__ __forceinline__ uint32_t stage_at(int r, int c) {
  return (uint32_t)(r * 128 + (((c >> 2) ^ (r & 7)) << 4) + (c & 3) * 4);
}
__device__ __forceinline__ void stage_put(uint8_t *stage, const float (&v)[32]) {
  const int lane = (int)lane_id();
  __syncwarp();  // earlier readers are done
#pragma unroll
  for (int u = 0; u < 8; ++u)
    *reinterpret_cast<float4 *>(stage + stage_at(lane, 4 * u)) =
        make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
  __syncwarp();
}

// 32 bytes, one sector, per lane (32-byte aligned).  Operands are read once
// and kept out of L1, what there is of it beside the stages: the bias, which
// every row reads, then stays there.
__device__ __forceinline__ void ld_sector(const void *p, uint32_t *w) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                 "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st_sector(void *p, const uint32_t *w) {
  asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
               : "memory");
}

// Whether lanes access their own rows of a chunk a sector at a time.
__device__ __forceinline__ bool direct(const GemmArgs &a, int64_t col0, int vec) {
  return vec && col0 + 32 <= a.N;
}

// The paths of unaligned or ragged chunks.  They are unrolled no further than
// their latency needs: fully unrolled, their registers spilled the aligned
// path's and cost 2% of the 16384 x 14336 x 4096 products.  rows, cols: the
// chunk's valid part.

// A 32 x 32 chunk of bf16 values into the stage, as fp32, row by row along the
// lanes.
__device__ __forceinline__ void gather_stage(const __nv_bfloat16 *src, int64_t ld, int rows,
                                             int cols, uint8_t *stage) {
  const int lane = (int)lane_id();
  __syncwarp();
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += 8) {
    // (the loads of a batch before its stores: the compiler cannot know that
    // the stage is not the source, and ran them one by one, 319 us against 147
    // at 13019 x 2273 x 256)
    __nv_bfloat16 t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      t[i] = lane < cols && r0 + i < rows ? src[(r0 + i) * ld + lane] : __nv_bfloat16(0.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<float *>(stage + stage_at(r0 + i, lane)) = __bfloat162float(t[i]);
  }
  __syncwarp();
}
// The same of fp32 values: asynchronous copies, all 32 rows in flight (a
// missing element is filled with zero).
__device__ __forceinline__ void gather_stage(const float *src, int64_t ld, int rows, int cols,
                                             uint8_t *stage) {
  const int lane = (int)lane_id();
  __syncwarp();
  for (int r = 0; r < 32; ++r) {
    const bool in = lane < cols && r < rows;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                     smem_u32(stage + stage_at(r, lane))),
                 "l"(in ? src + r * ld + lane : src), "r"(in ? 4 : 0)
                 : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
}

// The staged fp32 chunk to bf16 or fp32 rows.
__device__ __forceinline__ void scatter_stage(void *dst, int64_t ld, int size, int rows,
                                                  int cols, const uint8_t *stage) {
  const int lane = (int)lane_id();
  if (lane >= cols) return;
#pragma unroll 4
  for (int r = 0; r < 32; ++r) {
    if (r >= rows) break;
    const float x = *reinterpret_cast<const float *>(stage + stage_at(r, lane));
    if (size == 2)
      static_cast<__nv_bfloat16 *>(dst)[r * ld + lane] = __float2bfloat16_rn(x);
    else
      static_cast<float *>(dst)[r * ld + lane] = x;
  }
}

// Staged codes, 32 bytes per row.
__device__ __forceinline__ void scatter_codes(uint8_t *q, int64_t ld, int rows, int cols,
                                                  const uint8_t *stage) {
  const int lane = (int)lane_id();
  if (lane >= cols) return;
#pragma unroll 4
  for (int r = 0; r < 32; ++r)
    if (r < rows) q[r * ld + lane] = stage[32 * r + lane];
}

__device__ __forceinline__ int left32(int64_t n) { return n < 32 ? (int)n : 32; }

// Four values of this lane's staged row.
__device__ __forceinline__ float4 stage_row4(const uint8_t *stage, int u) {
  return *reinterpret_cast<const float4 *>(stage + stage_at((int)lane_id(), 4 * u));
}

// The bf16 row operand of the chunk at (row0, col0): pre (gradient) or the
// residual (forward).  Every lane of the warp calls it, a chunk ahead.
template <bool GRAD>
__device__ __forceinline__ void fetch_chunk(const GemmArgs &a, const LinearEp &e, int64_t row0,
                                            int64_t col0, uint8_t *stage, RowIn &in) {
  const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(GRAD ? e.pre : e.res);
  if (src == nullptr || row0 >= a.M || col0 >= a.N || (!GRAD && e.res_dt == 0)) return;
  const int64_t ld = GRAD ? e.ld_pre : e.ld_res, row = row0 + lane_id();
  if (direct(a, col0, GRAD ? e.pre_vec : e.res_vec)) {
    if (row >= a.M) return;
    ld_sector(src + row * ld + col0, in.w);
    ld_sector(src + row * ld + col0 + 16, in.w + 8);
    return;
  }
  gather_stage(src + row0 * ld + col0, ld, left32(a.M - row0), left32(a.N - col0), stage);
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const float4 f = stage_row4(stage, u);
    in.w[2 * u] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
    in.w[2 * u + 1] = __byte_perm(__float_as_uint(f.z), __float_as_uint(f.w), 0x7632);
  }
}

// One 32 x 32 chunk to a row-major matrix of T.
template <typename T>
__device__ __forceinline__ void put_chunk(const GemmArgs &a, T *dst, int64_t ld, int vec,
                                          int64_t row0, int64_t col0, const float (&v)[32],
                                          uint8_t *stage) {
  const int lane = (int)lane_id();
  if (direct(a, col0, vec)) {
    if (row0 + lane >= a.M) return;
    T *p = dst + (row0 + lane) * ld + col0;
    if constexpr (sizeof(T) == 2) {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
      st_sector(p, w);
      st_sector(p + 16, w + 8);
    } else {
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) st_sector(p + 8 * i, w + 8 * i);
    }
    return;
  }
  stage_put(stage, v);
  scatter_stage(dst + row0 * ld + col0, ld, (int)sizeof(T), left32(a.M - row0), left32(a.N - col0),
                stage);
}

// c, codes and the running max |y| (a NaN stays one) of a finished chunk.
__device__ __forceinline__ void put_result(const GemmArgs &a, const LinearEp &e, int64_t row0,
                                           int64_t col0, const float (&v)[32], const CodeScale &d,
                                           uint8_t *stage, float &amax) {
  if (a.c != nullptr) {
    if (a.out_dt == 1)
      put_chunk(a, static_cast<__nv_bfloat16 *>(a.c), a.ldc, e.c_vec, row0, col0, v, stage);
    else
      put_chunk(a, static_cast<float *>(a.c), a.ldc, e.c_vec, row0, col0, v, stage);
  }
  if (e.q == nullptr) return;
  const int lane = (int)lane_id();
  const bool row_in = row0 + lane < a.M;
  if (e.q_amax != nullptr && row_in) {
    if (col0 + 32 <= a.N) {
#pragma unroll
      for (int i = 0; i < 32; i += 2) amax = max_abs2(amax, F2(v[i], v[i + 1]));
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (col0 + i < a.N) amax = max_nan(amax, fabsf(v[i]));
    }
  }
  uint2 c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) d.quotient(F2(v[8 * j + i], v[8 * j + i + 1])).get(y[i], y[i + 1]);
    c[j] = pack8(e.q_fmt, y);
  }
  const uint4 lo = make_uint4(c[0].x, c[0].y, c[1].x, c[1].y), hi = make_uint4(c[2].x, c[2].y, c[3].x, c[3].y);
  if (direct(a, col0, e.q_vec)) {
    if (!row_in) return;
    uint8_t *q = e.q + (row0 + lane) * a.N + col0;
    if (e.q_vec == 2) {
      const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      st_sector(q, w);
    } else {  // N a multiple of 16 (as a GEMM operand's pitch is), not of 32
      reinterpret_cast<uint4 *>(q)[0] = lo;
      reinterpret_cast<uint4 *>(q)[1] = hi;
    }
    return;
  }
  __syncwarp();
  reinterpret_cast<uint4 *>(stage)[2 * lane] = lo;
  reinterpret_cast<uint4 *>(stage)[2 * lane + 1] = hi;
  __syncwarp();
  scatter_codes(e.q + row0 * a.N + col0, a.N, left32(a.M - row0), left32(a.N - col0), stage);
}

// z = alpha acc + bias
__device__ __forceinline__ void scale_bias(const GemmArgs &a, int64_t col0, const uint32_t (&r)[32],
                                           float alpha, float (&v)[32]) {
  const F2 al(alpha);
  auto acc = [&](int i) { return F2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])); };
  if (a.bias == nullptr || col0 >= a.N) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) (acc(i) * al).get(v[i], v[i + 1]);
  } else if (col0 + 32 <= a.N && (reinterpret_cast<uintptr_t>(a.bias + col0) & 15u) == 0) {
    const float4 *b4 = reinterpret_cast<const float4 *>(a.bias + col0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 b = b4[i];
      fma2(acc(4 * i), al, F2(b.x, b.y)).get(v[4 * i], v[4 * i + 1]);
      fma2(acc(4 * i + 2), al, F2(b.z, b.w)).get(v[4 * i + 2], v[4 * i + 3]);
    }
  } else {
    // one value per lane, handed around
    const int64_t n = col0 + lane_id();
    const float b = n < a.N ? a.bias[n] : 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      v[i] = fmaf(__uint_as_float(r[i]), alpha, __shfl_sync(0xffffffffu, b, i));
  }
}

// The residual added to a chunk as it is loaded, 16 columns of registers at a
// time (or through the stage).
template <typename T>
__device__ __forceinline__ void add_rows(const GemmArgs &a, const T *src, int64_t ld, int vec,
                                         int64_t row0, int64_t col0, float (&v)[32],
                                         uint8_t *stage) {
  if (direct(a, col0, vec)) {
    const int64_t row = row0 + lane_id();
    if (row >= a.M) return;
    constexpr int kPer = 32 / sizeof(T);  // values of a sector
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
      uint32_t w[16 * sizeof(T) / 4];
      const T *p = src + row * ld + col0 + h;
#pragma unroll
      for (int i = 0; i < 16 / kPer; ++i) ld_sector(p + i * kPer, w + 8 * i);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        F2 x;
        if constexpr (sizeof(T) == 2)
          x = bf16_pair(w[i / 2]);
        else
          x = F2(__uint_as_float(w[i]), __uint_as_float(w[i + 1]));
        (F2(v[h + i], v[h + i + 1]) + x).get(v[h + i], v[h + i + 1]);
      }
    }
  } else {
    gather_stage(src + row0 * ld + col0, ld, left32(a.M - row0), left32(a.N - col0), stage);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float4 f = stage_row4(stage, u);
      v[4 * u] += f.x; v[4 * u + 1] += f.y; v[4 * u + 2] += f.z; v[4 * u + 3] += f.w;
    }
  }
}

// Forward epilogue of one chunk (v: z of this lane's row).  AHEAD: `in` holds a
// bf16 residual of fetch_chunk; an fp32 one has too many registers for that,
// and so has any in the kernels that keep a tile's accumulators in registers
// (FP32 group scales: 4096 x 7168 x 2048 with bias and silu 92 us on operands
// that L2 still holds, 97-100 on others; a pass of its own per 16 columns took
// 110; the same product without an epilogue takes 76).  Every lane of the warp calls it.
template <bool AHEAD>
__device__ __forceinline__ void linear_chunk(const GemmArgs &a, const LinearEp &e, int64_t row0,
                                             int64_t col0, float (&v)[32], const RowIn &in,
                                             const CodeScale &d, uint8_t *stage, float &amax) {
  if (row0 >= a.M || col0 >= a.N) return;
  if (e.pre != nullptr)
    put_chunk(a, static_cast<__nv_bfloat16 *>(e.pre), e.ld_pre, e.pre_vec, row0, col0, v, stage);
  with_act(e.act, [&](auto act) {
#pragma unroll
    for (int i = 0; i < 32; i += 2)
      act_value2<decltype(act)::value>(F2(v[i], v[i + 1])).get(v[i], v[i + 1]);
  });
  if (e.res != nullptr) {
    if (e.res_dt == 0) {
      add_rows(a, static_cast<const float *>(e.res), e.ld_res, e.res_vec, row0, col0, v, stage);
    } else if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < 32; i += 2)
        (F2(v[i], v[i + 1]) + bf16_pair(in.w[i / 2])).get(v[i], v[i + 1]);
    } else {
      add_rows(a, static_cast<const __nv_bfloat16 *>(e.res), e.ld_res, e.res_vec, row0, col0, v,
               stage);
    }
  }
  put_result(a, e, row0, col0, v, d, stage, amax);
}

// The bias added to a chunk in place.
__device__ __forceinline__ void add_bias(const GemmArgs &a, int64_t col0, float (&v)[32]) {
  if (a.bias == nullptr || col0 >= a.N) return;
  if (col0 + 32 <= a.N && (reinterpret_cast<uintptr_t>(a.bias + col0) & 15u) == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 b = reinterpret_cast<const float4 *>(a.bias + col0)[i];
      v[4 * i] += b.x; v[4 * i + 1] += b.y; v[4 * i + 2] += b.z; v[4 * i + 3] += b.w;
    }
  } else {
    // one value per lane, handed around
    const int64_t n = col0 + lane_id();
    const float b = n < a.N ? a.bias[n] : 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xffffffffu, b, i);
  }
}

// Gradient epilogue of one chunk (r: the accumulators of this lane's row; in:
// pre); its 32 rows' column sums go to
// part[row0 / 32][col0 ...], through the stage: lane l adds 16 rows of the
// columns 2 (l % 16) and the next, then the two halves of the warp add up.
// next(): the accumulators have been used (the whole warp calls it).
template <typename Next>
__device__ __forceinline__ void grad_chunk(const GemmArgs &a, const LinearEp &e, int64_t row0,
                                           int64_t col0, const uint32_t (&r)[32], float alpha,
                                           const RowIn &in, const CodeScale &d, uint8_t *stage,
                                           float &amax, Next &&next) {
  if (row0 >= a.M || col0 >= a.N) {
    next();
    return;
  }
  const int lane = (int)lane_id();
  const F2 al(alpha);
  float v[32];
  if (row0 + lane < a.M) {
    auto scaled = [&](int i) { return F2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])) * al; };
    // (alpha applied here, pair by pair: as a pass of its own it cost 8 us of
    // 41 at 2048 x 5120 x 1024, the registers of a second set of values)
    with_act<true>(e.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < 32; i += 2)
        (scaled(i) * act_slope2<decltype(act)::value>(bf16_pair(in.w[i / 2]))).get(v[i], v[i + 1]);
    });
  } else {  // a row past M adds nothing to the sums
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0.0f;
  }
  __syncwarp();
  next();
  put_result(a, e, row0, col0, v, d, stage, amax);
  if (e.part == nullptr) return;
  stage_put(stage, v);
  F2 sum(0.0f);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 p = *reinterpret_cast<const float2 *>(
        stage + stage_at(16 * (lane >> 4) + i, 2 * (lane & 15)));
    sum = sum + F2(p.x, p.y);
  }
  float s0, s1;
  sum.get(s0, s1);
  s0 += __shfl_xor_sync(0xffffffffu, s0, 16);
  s1 += __shfl_xor_sync(0xffffffffu, s1, 16);
  const int64_t col = col0 + 2 * (lane & 15) + (lane >> 4);  // each half writes one of the pair
  if (col < a.N) e.part[(row0 >> 5) * a.N + col] = lane < 16 ? s0 : s1;
}

// pre, activation and residual of one value z = result + bias: returns y.
__device__ __forceinline__ float linear_value(const LinearEp &e, int64_t row, int64_t col, float z) {
  if (e.pre != nullptr)
    static_cast<__nv_bfloat16 *>(e.pre)[row * e.ld_pre + col] = __float2bfloat16_rn(z);
  with_act(e.act, [&](auto act) {
    float unused;
    act_value2<decltype(act)::value>(F2(z)).get(z, unused);
  });
  if (e.res != nullptr) {
    const int64_t at = row * e.ld_res + col;
    z += e.res_dt == 0 ? static_cast<const float *>(e.res)[at]
                       : __bfloat162float(static_cast<const __nv_bfloat16 *>(e.res)[at]);
  }
  return z;
}

// Forward epilogue of up to four columns of one row, the last step of
// cluster_reduce; the residual is loaded with the partial sums.
struct LinearPut {
  const GemmArgs &a;
  const LinearEp &e;
  const CodeScale d;
  float &amax;
  struct In {
    float r[4];
  };
  // address of four elements that may be accessed as one vector
  static __device__ __forceinline__ bool whole(const void *p, int n, uintptr_t bytes) {
    return n == 4 && (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
  }
  __device__ __forceinline__ In load(int64_t row, int64_t col, int n) const {
    In in = {{0.0f, 0.0f, 0.0f, 0.0f}};
    if (e.res == nullptr) return in;
    const int64_t at = row * e.ld_res + col;
    if (e.res_dt == 0) {
      const float *p = static_cast<const float *>(e.res) + at;
      if (whole(p, n, 16)) {
        const float4 u = *reinterpret_cast<const float4 *>(p);
        in.r[0] = u.x; in.r[1] = u.y; in.r[2] = u.z; in.r[3] = u.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < n) in.r[i] = p[i];
      }
    } else {
      const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(e.res) + at;
      if (whole(p, n, 8)) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        bf16_pair(u.x).get(in.r[0], in.r[1]);
        bf16_pair(u.y).get(in.r[2], in.r[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < n) in.r[i] = __bfloat162float(p[i]);
      }
    }
    return in;
  }
  static __device__ __forceinline__ void put_bf16(__nv_bfloat16 *p, int n, const float (&v)[4]) {
    if (whole(p, n, 8)) {
      *reinterpret_cast<uint2 *>(p) = f32x4_to_bf16(make_float4(v[0], v[1], v[2], v[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) p[i] = __float2bfloat16_rn(v[i]);
    }
  }
  __device__ __forceinline__ void operator()(int64_t row, int64_t col, int n, float (&v)[4],
                                             const In &in) const {
    if (a.bias != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) v[i] += a.bias[col + i];
    }
    if (e.pre != nullptr)
      put_bf16(static_cast<__nv_bfloat16 *>(e.pre) + row * e.ld_pre + col, n, v);
    with_act(e.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < 4; i += 2)
        act_value2<decltype(act)::value>(F2(v[i], v[i + 1])).get(v[i], v[i + 1]);
    });
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += in.r[i];
    if (a.c != nullptr) {
      if (a.out_dt == 1) {
        put_bf16(static_cast<__nv_bfloat16 *>(a.c) + row * a.ldc + col, n, v);
      } else {
        float *p = static_cast<float *>(a.c) + row * a.ldc + col;
        if (whole(p, n, 16)) {
          *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = v[i];
        }
      }
    }
    if (e.q == nullptr) return;
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) amax = max_nan(amax, fabsf(v[i]));
#pragma unroll
    for (int i = 0; i < 4; i += 2) d.quotient(F2(v[i], v[i + 1])).get(y[i], y[i + 1]);
    const uint32_t lo = cvt_fp8x2(e.q_fmt, y[0], y[1]), hi = cvt_fp8x2(e.q_fmt, y[2], y[3]);
    const uint32_t c = __byte_perm(lo, hi, 0x5410);
    uint8_t *q = e.q + row * a.N + col;
    if (whole(q, n, 4)) {
      *reinterpret_cast<uint32_t *>(q) = c;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) q[i] = (uint8_t)(c >> (8 * i));
    }
  }
};

// The warp's running max |y| into the call's, or into its slot where the
// column sums' kernel finishes it (every lane calls; slot: the warp's index
// in the grid).
__device__ __forceinline__ void flush_amax(const LinearEp &e, float amax, int64_t slot) {
  if (e.q == nullptr || e.q_amax == nullptr) return;
  const uint32_t key = warp_max_u32(__float_as_uint(amax));
  if (lane_id() != 0) return;
  if (e.tops != nullptr)
    e.tops[slot] = __uint_as_float(key);
  else if (key != 0u)
    atomicMax(e.q_amax, key);
}

}  // namespace fp8k
