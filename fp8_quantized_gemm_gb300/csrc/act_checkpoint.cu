// An activation between two FP8 products whose arguments are kept for the
// backward pass in 8 bits.
//
// Forward: a = act(h) u (u absent: act(h)) as codes, and the checkpoints: h and
// u as E4M3 codes with a scale per 1x128 group.  Backward, on the values h and u
// that the checkpoints stand for:
//   dh = da u act'(h),   du = da act(h)
// as codes.  Group scales are formed from the group's own fp32 values, per-tensor
// scales are fixed before the call.  (The bf16 h and u of a forward pass are 4
// bytes an element until the backward pass has read them; these are 2.06.)
//
// Every byte is touched once: forward 4 in, 1 + 2.06 out an element, backward
// 2 + 2.06 in, 2 out.  A CTA takes tiles of 32 rows by 128 columns, a row's
// group on eight lanes of 16 elements each (32-byte accesses, and the scales of
// a tile are 32 neighbours of the group-major layout); tiles go by column first.
#include "act_checkpoint.h"
#include "activation.cuh"
#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "pairs.cuh"
#include "quant_common.cuh"
#include "rowvec.cuh"

namespace fp8k {

// act(z) and act'(z) from one exponential (the forms and limits of
// act_value2 / act_slope2).
template <int A>
__device__ __forceinline__ void act_both2(F2 z, F2 &value, F2 &slope) {
  if constexpr (A == kActSilu) {
    const F2 b = within_2(z, kFar), s = logistic2(b * F2(kNegLog2e));
    value = left_capped(z) * s;
    slope = s * fma2(b, fma2(s, F2(-1.0f), F2(1.0f)), F2(1.0f));
  } else if constexpr (A == kActGeluTanh) {
    const F2 b = within_2(z, kFarCubed), bb = b * b;
    const F2 s = logistic2(b * fma2(bb, F2(kT3), F2(kT1)));
    value = left_capped(z) * s;
    slope = fma2(b * s, fma2(s, F2(-1.0f), F2(1.0f)) * fma2(bb, F2(kD3), F2(kD1)), s);
  } else {  // (the normal tail of gelu is common to both: the compiler keeps one)
    value = act_value2<A>(z);
    slope = act_slope2<A>(z);
  }
}

// Codes of 16 fp32 results.  Per tensor: under d, the maximum into `top`; per
// group: under a scale of their own, stored by the group's first lane.
template <int F>
__device__ __forceinline__ uint4 code16(F2 (&y)[8], const CodeScale &d, float &top) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top = max_abs2(top, y[i]);
    y[i] = d.quotient(y[i]);
  }
  return pack16<F>(y);
}
template <int F>
__device__ __forceinline__ uint4 code16_group(F2 (&y)[8], int sfmt, void *scales, int64_t at,
                                              bool owner) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_abs2(m, y[i]);
  const float amax = __uint_as_float(group8_max(__float_as_uint(m)));
  if (sfmt == 0) {
    const float s = scale_from_amax(amax, fmt_max(F));
    if (owner) static_cast<float *>(scales)[at] = s;
    const CodeScale d(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = d.quotient(y[i]);
  } else {
    const int e = ue8m0_exponent(amax, fmt_max(F));
    if (owner) static_cast<uint8_t *>(scales)[at] = (uint8_t)(e + 127);
    const F2 inv(exp2_int(-e));
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = y[i] * inv;
  }
  return pack16<F>(y);
}

// The checkpoint of 16 bf16 values.
__device__ __forceinline__ void keep16(const Vec16<__nv_bfloat16> &v, uint8_t *q, void *scales,
                                       int64_t at, int sfmt, bool in, bool owner) {
  const float amax = __uint_as_float(group8_max(v.max_key()));
  uint4 c;
  if (sfmt == 0) {
    const float s = scale_from_amax(amax, kE4M3Max);
    if (owner) static_cast<float *>(scales)[at] = s;
    c = v.codes<0>(ScaleDiv(s));
  } else {
    const int e = ue8m0_exponent(amax, kE4M3Max);
    if (owner) static_cast<uint8_t *>(scales)[at] = (uint8_t)(e + 127);
    c = v.codes_pow2<0>(exp2_int(-e));
  }
  if (in) *reinterpret_cast<uint4 *>(q) = c;
}

// Two E4M3 codes -> two fp32 values (exact: through half precision, which
// holds every E4M3 value).
__device__ __forceinline__ F2 e4m3_pair(uint32_t two) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)two));
  float lo, hi;
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b; }"
      : "=f"(lo), "=f"(hi)
      : "r"(h2));
  return F2(lo, hi);
}
__device__ __forceinline__ float kept_scale(const void *scales, int64_t at, int sfmt) {
  return sfmt == 0 ? static_cast<const float *>(scales)[at]
                   : exp2_int((int)static_cast<const uint8_t *>(scales)[at] - 127);
}
// the i-th pair of 16 codes under their scale
__device__ __forceinline__ F2 kept_pair(const uint4 &c, int i, F2 s) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  return e4m3_pair(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu) * s;
}

// Rows that are dealt with.
__device__ __forceinline__ int64_t live_rows(const int32_t *valid, int64_t M) {
  return valid == nullptr ? M : max((int64_t)0, min((int64_t)*valid, M));
}

// This thread's place in a tile.
struct TilePlace {
  int64_t row, col, g;
  bool in;     // its elements lie inside the matrix
  bool owner;  // it stores its group's scale
};
__device__ __forceinline__ TilePlace tile_place(int64_t tile, int64_t groups, bool narrow,
                                                int64_t rows, int64_t N) {
  TilePlace p;
  int64_t rt;
  split_task(tile, groups, narrow, rt, p.g);
  p.row = rt * 32 + (threadIdx.x >> 3);
  p.col = p.g * 128 + (threadIdx.x & 7u) * 16;
  p.in = p.row < rows && p.col < N;
  p.owner = p.row < rows && (threadIdx.x & 7u) == 0u;
  return p;
}

template <int A, bool GATE, int F>
__global__ void __launch_bounds__(256) act_checkpoint_kernel(const ActArgs a) {
  launch_dependents();
  grid_dependency_wait();
  const __nv_bfloat16 *h = static_cast<const __nv_bfloat16 *>(a.h);
  const __nv_bfloat16 *u = static_cast<const __nv_bfloat16 *>(a.u);
  const int64_t rows = live_rows(a.valid, a.M);
  const int64_t groups = (a.N + 127) / 128, tiles = (rows + 31) / 32 * groups;
  const bool narrow = tiles + gridDim.x <= (int64_t)0xFFFFFFFFu;
  const CodeScale d(a.scale != nullptr ? *a.scale : 1.0f);
  float top = 0.0f;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const TilePlace p = tile_place(tile, groups, narrow, rows, a.N);
    Vec16<__nv_bfloat16> hv, uv;
    hv.zero();
    uv.zero();
    if (p.in) {
      hv.load(h + p.row * a.ldh + p.col);
      if (GATE) uv.load(u + p.row * a.ldu + p.col);
    }
    const int64_t at = p.g * a.M + p.row, flat = p.row * a.N + p.col;
    if (a.hq != nullptr) keep16(hv, a.hq + flat, a.hs, at, a.keep_sfmt, p.in, p.owner);
    if (GATE && a.uq != nullptr) keep16(uv, a.uq + flat, a.us, at, a.keep_sfmt, p.in, p.owner);
    F2 y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = act_value2<A>(hv.pair(i));
      if (GATE) y[i] = y[i] * uv.pair(i);
    }
    if (a.out != nullptr && p.in)
      store16(static_cast<__nv_bfloat16 *>(a.out) + p.row * a.ld_out + p.col, y);
    const uint4 c = a.scale != nullptr
                        ? code16<F>(y, d, top)
                        : code16_group<F>(y, a.sfmt, a.scales, at, p.owner);
    if (p.in) *reinterpret_cast<uint4 *>(a.q + flat) = c;
  }
  if (a.amax != nullptr) block_max_to(__float_as_uint(top), a.amax);
}

template <int A, bool GATE, int F>
__global__ void __launch_bounds__(256) act_checkpoint_grad_kernel(const ActGradArgs a) {
  launch_dependents();
  grid_dependency_wait();
  const __nv_bfloat16 *da = static_cast<const __nv_bfloat16 *>(a.da);
  const int64_t rows = live_rows(a.valid, a.M);
  const int64_t groups = (a.N + 127) / 128, tiles = (rows + 31) / 32 * groups;
  const bool narrow = tiles + gridDim.x <= (int64_t)0xFFFFFFFFu;
  const bool tensor = a.tensor != 0;
  const CodeScale dh(a.scale_h != nullptr ? *a.scale_h : 1.0f);
  const CodeScale du(a.scale_u != nullptr ? *a.scale_u : 1.0f);
  float top_h = 0.0f, top_u = 0.0f;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const TilePlace p = tile_place(tile, groups, narrow, rows, a.N);
    const int64_t at = p.g * a.M + p.row, flat = p.row * a.N + p.col;
    Vec16<__nv_bfloat16> v;
    Vec16<uint8_t> hc, uc;
    v.zero();
    hc.zero();
    uc.zero();
    F2 hs(0.0f), us(0.0f);
    if (p.in) {
      v.load(da + p.row * a.ld_da + p.col);
      hc.load(a.hq + flat);
      hs = F2(kept_scale(a.hs, at, a.keep_sfmt));
      if (GATE) {
        uc.load(a.uq + flat);
        us = F2(kept_scale(a.us, at, a.keep_sfmt));
      }
    }
    F2 yh[8], yu[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      F2 value, slope;
      const F2 g = v.pair(i);
      act_both2<A>(kept_pair(hc.w[0], i, hs), value, slope);
      if (GATE) {
        yh[i] = g * kept_pair(uc.w[0], i, us) * slope;
        yu[i] = g * value;
      } else {
        yh[i] = g * slope;
      }
    }
    const int64_t qat = p.row * a.ld_q + p.col, dat = p.row * a.ld_d + p.col;
    if (a.dh != nullptr && p.in) store16(static_cast<__nv_bfloat16 *>(a.dh) + dat, yh);
    if (GATE && a.du != nullptr && p.in) store16(static_cast<__nv_bfloat16 *>(a.du) + dat, yu);
    if (a.qh != nullptr) {
      const uint4 c = tensor ? code16<F>(yh, dh, top_h)
                             : code16_group<F>(yh, a.sfmt, a.sh, at, p.owner);
      if (p.in) *reinterpret_cast<uint4 *>(a.qh + qat) = c;
    }
    if (GATE && a.qu != nullptr) {
      const uint4 c = tensor ? code16<F>(yu, du, top_u)
                             : code16_group<F>(yu, a.sfmt, a.su, at, p.owner);
      if (p.in) *reinterpret_cast<uint4 *>(a.qu + qat) = c;
    }
  }
  if (a.amax_h != nullptr) block_max_to(__float_as_uint(top_h), a.amax_h);
  if (GATE && a.amax_u != nullptr) {
    __syncthreads();  // block_max_to's shared scratch is used again
    block_max_to(__float_as_uint(top_u), a.amax_u);
  }
}

// The maxima's words (nullable) ahead of the kernel that raises them, in the
// programmatic launch chain.
__global__ void clear_maxima_kernel(uint32_t *p, uint32_t *q) {
  launch_dependents();
  grid_dependency_wait();
  if (threadIdx.x == 0 && p != nullptr) *p = 0u;
  if (threadIdx.x == 0 && q != nullptr) *q = 0u;
}
static cudaError_t clear_maxima(uint32_t *p, uint32_t *q, cudaStream_t st) {
  if (p == nullptr && q == nullptr) return cudaSuccess;
  return launch_serial(clear_maxima_kernel, 1, 32, st, p, q);
}

static int64_t tile_blocks(int64_t M, int64_t N, int sms) {
  const int64_t tiles = (M + 31) / 32 * ((N + 127) / 128), most = (int64_t)sms * 8;
  return tiles < most ? tiles : most;
}

// Calls f with gate and format as compile-time constants.
template <typename Fn>
static void with_gate(bool gate, int fmt, Fn &&f) {
  using std::integral_constant;
  if (gate) {
    if (fmt == 0) f(integral_constant<bool, true>{}, integral_constant<int, 0>{});
    else f(integral_constant<bool, true>{}, integral_constant<int, 1>{});
  } else {
    if (fmt == 0) f(integral_constant<bool, false>{}, integral_constant<int, 0>{});
    else f(integral_constant<bool, false>{}, integral_constant<int, 1>{});
  }
}

// Calls f with the activation as a compile-time constant, on the host.
template <typename Fn>
static void each_act(int act, Fn &&f) {
  using std::integral_constant;
  switch (act) {
    case kActRelu: f(integral_constant<int, kActRelu>{}); break;
    case kActRelu2: f(integral_constant<int, kActRelu2>{}); break;
    case kActSilu: f(integral_constant<int, kActSilu>{}); break;
    case kActGeluTanh: f(integral_constant<int, kActGeluTanh>{}); break;
    case kActGelu: f(integral_constant<int, kActGelu>{}); break;
    default: f(integral_constant<int, kActNone>{}); break;
  }
}

cudaError_t launch_act_checkpoint(const ActArgs &a, int sms, cudaStream_t st) {
  cudaError_t e = clear_maxima(a.amax, nullptr, st);
  if (e != cudaSuccess || a.M == 0) return e;
  const int64_t blocks = tile_blocks(a.M, a.N, sms);
  each_act(a.act, [&](auto act) {
    with_gate(a.u != nullptr, a.fmt, [&](auto gate, auto fmt) {
      e = launch_serial(act_checkpoint_kernel<act.value, gate.value, fmt.value>, blocks, 256, st, a);
    });
  });
  return e;
}

cudaError_t launch_act_checkpoint_grad(const ActGradArgs &a, int sms, cudaStream_t st) {
  cudaError_t e = clear_maxima(a.amax_h, a.amax_u, st);
  if (e != cudaSuccess || a.M == 0) return e;
  const int64_t blocks = tile_blocks(a.M, a.N, sms);
  each_act(a.act, [&](auto act) {
    with_gate(a.uq != nullptr, a.fmt, [&](auto gate, auto fmt) {
      e = launch_serial(act_checkpoint_grad_kernel<act.value, gate.value, fmt.value>, blocks, 256,
                        st, a);
    });
  });
  return e;
}

}  // namespace fp8k
