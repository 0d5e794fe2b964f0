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
// 16384 x 14336 gated: forward 260 us (94% of the copy rate), backward 231 (92%).
// Gelu is bound by its instructions (without a gate 207 and 208 us, where silu
// takes 158 and 149).
#include "act_checkpoint.h"
#include "activation.cuh"
#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "pairs.cuh"
#include "quant_common.cuh"
#include "rowvec.cuh"

namespace fp8k {

// act(z) and act'(z) from one exponential, the forms of act_value2 /
// act_slope2 without their bounds: |z| is at most 2^49 here.
template <int A>
__device__ __forceinline__ void act_both2(F2 z, F2 &value, F2 &slope) {
  if constexpr (A == kActSilu) {
    const F2 s = logistic2(z * F2(kNegLog2e));
    value = z * s;
    slope = fma2(value, fma2(s, F2(-1.0f), F2(1.0f)), s);
  } else if constexpr (A == kActGeluTanh) {
    const F2 zz = z * z, s = logistic2(z * fma2(zz, F2(kT3), F2(kT1)));
    value = z * s;
    slope = fma2(value, fma2(s, F2(-1.0f), F2(1.0f)) * fma2(zz, F2(kD3), F2(kD1)), s);
  } else {  // (the normal tail of gelu is common to both: the compiler keeps one)
    value = act_value2<A>(z);
    slope = act_slope2<A>(z);
  }
}
// Eight pairs of the activation's values from raw bf16 arguments.  silu and the
// tanh form need their argument bounded on the left (-inf times a factor that has
// vanished): two at a time on the bf16 pair.
template <int A>
__device__ __forceinline__ F2 act_of_word(uint32_t w) {
  if constexpr (A == kActSilu || A == kActGeluTanh) {
    uint32_t c;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(w), "r"(0xC61CC61Cu));  // -9984
    const F2 z = bf16_pair(c);
    if constexpr (A == kActSilu) return z * logistic2(z * F2(kNegLog2e));
    return z * logistic2(z * fma2(z * z, F2(kT3), F2(kT1)));
  } else {
    return act_value2<A>(bf16_pair(w));
  }
}

// 16 bf16 values as two vectors of eight
struct Words16 {
  uint4 a, b;
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    return w[i];
  }
  __device__ __forceinline__ F2 pair(int i) const { return bf16_pair(word(i)); }
  // max |x| (one instruction a pair; the sign that it leaves is dropped)
  __device__ __forceinline__ float max_abs() const {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(word(i)));
    m &= 0x7FFF7FFFu;
    return __uint_as_float(max(m << 16, m & 0xFFFF0000u));
  }
};

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
// A checkpoint's scale as loaded (KEPT 0: fp32 bits, 1: the UE8M0 byte; nothing is
// done with it before the tile that it was loaded ahead for), and its value.
template <int KEPT>
__device__ __forceinline__ uint32_t kept_bits(const void *scales, int64_t at) {
  if constexpr (KEPT == 0) return static_cast<const uint32_t *>(scales)[at];
  return static_cast<const uint8_t *>(scales)[at];
}
template <int KEPT>
__device__ __forceinline__ float kept_scale(uint32_t bits) {
  if constexpr (KEPT == 0) return __uint_as_float(bits);
  return __uint_as_float(max(bits << 23, 0x00400000u));  // 2^(e - 127)
}
// the i-th pair of 16 codes under their scale
__device__ __forceinline__ F2 kept_pair(const uint4 &c, int i, F2 s) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  return e4m3_pair(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu) * s;
}

// Rows that are dealt with.
__device__ __forceinline__ uint32_t live_rows(const int32_t *valid, int64_t M) {
  return valid == nullptr ? (uint32_t)M : (uint32_t)max((int64_t)0, min((int64_t)*valid, M));
}

// A CTA's walk over the tiles blockIdx.x, blockIdx.x + gridDim.x, ... of 32 rows
// by 128 columns, column first; this thread's row and first column.  (Rows,
// columns and pitches are below 2^31: one wide multiplication an address.)
struct TileWalk {
  int64_t left;  // tiles from here to the end, this one included
  uint32_t row, g, groups, step_rows, step_g;
  __device__ __forceinline__ TileWalk(uint32_t rows, uint32_t N) {
    groups = (N + 127) / 128;
    const uint32_t rt = blockIdx.x / groups;
    left = (int64_t)((rows + 31) / 32) * groups - blockIdx.x;
    g = blockIdx.x - rt * groups;
    row = rt * 32 + (threadIdx.x >> 3);
    step_rows = gridDim.x / groups * 32;
    step_g = gridDim.x % groups;
  }
  __device__ __forceinline__ void next() {
    left -= gridDim.x;
    row += step_rows;
    g += step_g;
    if (g >= groups) {
      g -= groups;
      row += 32;
    }
  }
  // how many tiles of the walk are ahead of this one (few enough for 32 bits)
  __device__ __forceinline__ uint32_t step(uint32_t rows) const {
    return (uint32_t)((int64_t)((rows + 31) / 32) * groups - blockIdx.x - left) / gridDim.x;
  }
  __device__ __forceinline__ uint32_t col() const { return g * 128 + (threadIdx.x & 7u) * 16; }
  __device__ __forceinline__ int64_t at(int64_t pitch) const {
    return (int64_t)((uint64_t)row * (uint32_t)pitch + col());
  }
  __device__ __forceinline__ int64_t scale_at(int64_t M) const {
    return (int64_t)((uint64_t)g * (uint32_t)M + row);
  }
};

// Threads of a CTA, and CTAs that share an SM.  With a gate three (85 registers a
// thread: the next tile's operands wait in registers; 16384 x 14336 in 260 us
// forward and 231 backward, 287 and 281 on four, which spill); without one four
// (silu 158 us forward and 149 backward, 181 and 160 on three).
constexpr int kTileThreads = 256;
constexpr int ctas_per_sm(bool gate) { return gate ? 3 : 4; }

// 16 values from p, or zeros
__device__ __forceinline__ Words16 load16(const __nv_bfloat16 *p, bool in) {
  Words16 v{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (in) {
    v.a = __ldcs(reinterpret_cast<const uint4 *>(p));
    v.b = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
  }
  return v;
}

__device__ __forceinline__ float max_abs16(const F2 (&y)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_abs2(m, y[i]);
  return m;
}
__device__ __forceinline__ void pairs_of(const Words16 &v, F2 (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = v.pair(i);
}
__device__ __forceinline__ void put16(uint8_t *q, const uint4 &c, bool in) {
  if (in) *reinterpret_cast<uint4 *>(q) = c;
}

// The kernels' loops hold the common case: scales far from the ends of fp32
// (GroupScale::fast) and, backward, checkpoints of values below 2^49.  A warp with
// another case in its four rows of a tile notes the tile and does the four again behind
// its loop, out of line: the groups that need them with IEEE quotients and bounded
// activations, the others as in the loop, so that what a group's bytes are depends on
// that group alone.  (The same code inside the loop cost the backward pass 30 us of 262:
// registers kept across its calls.  16384 x 14336, gated silu, forward and backward: no
// such group 264 and 231 us, one 273 and 240, one in a hundred rows 371 and 341, all 1740
// and 1940.)
//
// A bit per tile of the walk, 32 on each lane; no CTA walks over more than kMostTiles.
constexpr uint32_t kMostTiles = 1024;
__device__ __forceinline__ void note_tile(uint32_t &noted, uint32_t step) {
  if ((threadIdx.x & 31u) == step >> 5) noted |= 1u << (step & 31u);
}
__device__ __forceinline__ bool tile_noted(uint32_t noted, uint32_t step) {
  return __shfl_sync(0xffffffffu, noted, step >> 5) >> (step & 31u) & 1u;
}

// Codes of 16 results under the scale of their group (group: 8 lanes), stored
// with it; false where the scale is not of the common case (what is stored does
// not hold then).
template <int F>
__device__ __forceinline__ bool put_group(const F2 (&y)[8], float amax, int sfmt, uint8_t *q,
                                          void *scales, int64_t at, bool in, bool owner) {
  const float top = __uint_as_float(group8_max(__float_as_uint(amax)));
  const GroupScale g = group_scale<F>(top, sfmt);
  if (owner) store_scale(scales, at, g.stored, sfmt);
  put16(q, codes16_times<F>(y, g.inv), in);
  return g.fast;
}
// The same for a group of any scale.
template <int F>
__device__ __forceinline__ void put_group_any(const F2 (&y)[8], float amax, int sfmt, uint8_t *q,
                                              void *scales, int64_t at, bool in, bool owner) {
  const float top = __uint_as_float(group8_max(__float_as_uint(amax)));
  GroupScale g = group_scale<F>(top, sfmt);
  if (g.fast) {
    put16(q, codes16_times<F>(y, g.inv), in);
  } else {
    g = group_scale_any<F>(top, sfmt);
    put16(q, codes16_any<F>(y, g.s), in);
  }
  if (owner) store_scale(scales, at, g.stored, sfmt);
}
// Two results of the same group at once: the first step of the reduction leaves
// the maximum of y to even lanes and that of z to odd ones, so that each lane
// forms one scale instead of two.
template <int F>
__device__ __forceinline__ bool put_groups(const F2 (&y)[8], const F2 (&z)[8], int sfmt,
                                           uint8_t *qy, uint8_t *qz, void *sy, void *sz, int64_t at,
                                           bool in, bool live) {
  const bool odd = threadIdx.x & 1u;
  const uint32_t ky = __float_as_uint(max_abs16(y)), kz = __float_as_uint(max_abs16(z));
  uint32_t key = odd ? kz : ky;
  key = max(key, __shfl_xor_sync(0xffffffffu, odd ? ky : kz, 1));
  key = max(key, __shfl_xor_sync(0xffffffffu, key, 2));
  key = max(key, __shfl_xor_sync(0xffffffffu, key, 4));
  const GroupScale g = group_scale<F>(__uint_as_float(key), sfmt);
  if (!__all_sync(0xffffffffu, g.fast)) return false;
  const float other = __shfl_xor_sync(0xffffffffu, g.inv, 1);
  if (live && (threadIdx.x & 7u) < 2u) store_scale(odd ? sz : sy, at, g.stored, sfmt);
  put16(qy, codes16_times<F>(y, odd ? other : g.inv), in);
  put16(qz, codes16_times<F>(z, odd ? g.inv : other), in);
  return true;
}
// Under the tensor's scale d, the maximum into `top`.
template <int F>
__device__ __forceinline__ void put_tensor(const F2 (&y)[8], const CodeScale &d, float &top,
                                           uint8_t *q, bool in) {
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_abs2(top, y[i]);
  put16(q, codes16_times<F>(y, d.inv), in);
}
template <int F>
__device__ __forceinline__ void put_tensor_any(const F2 (&y)[8], const CodeScale &d, float &top,
                                               uint8_t *q, bool in) {
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_abs2(top, y[i]);
  put16(q, d.fast ? codes16_times<F>(y, d.inv) : codes16_any<F>(y, d.s), in);
}

// The activation by its number: the loops' forms, and those for any argument.
__device__ __noinline__ uint64_t act_of_word_any(uint32_t w, int act) {
  F2 r(bf16_pair(w));
  with_act(act, [&](auto a) { r = act_of_word<a.value>(w); });
  return r.v;
}
struct BothBits {
  uint64_t value, slope;
};
__device__ __noinline__ BothBits act_both_any(uint64_t z, int act, bool common) {
  F2 value(z), slope(1.0f);
  with_act(act, [&](auto a) {
    if (common) {
      act_both2<a.value>(F2(z), value, slope);
    } else {
      value = act_value2<a.value>(F2(z));
      slope = act_slope2<a.value>(F2(z));
    }
  });
  return BothBits{value.v, slope.v};
}

// The tiles that this warp has noted, again.
template <int F>
__device__ __noinline__ float act_slow_walk(const ActArgs &a, uint32_t rows, float top,
                                             uint32_t noted) {
  const __nv_bfloat16 *h = static_cast<const __nv_bfloat16 *>(a.h);
  const __nv_bfloat16 *u = static_cast<const __nv_bfloat16 *>(a.u);
  const uint32_t N = (uint32_t)a.N;
  const CodeScale d(a.scale != nullptr ? *a.scale : 1.0f);
  uint32_t step = 0u;
#pragma unroll 1
  for (TileWalk t(rows, N); t.left > 0; t.next(), ++step) {
    if (!tile_noted(noted, step)) continue;
    const int64_t at = t.scale_at(a.M), flat = t.at(a.N);
    const bool in = t.row < rows && t.col() < N, owner = t.row < rows && (threadIdx.x & 7u) == 0u;
    const Words16 hv = load16(h + t.at(a.ldh), in);
    Words16 uv = hv;
    if (u != nullptr) uv = load16(u + t.at(a.ldu), in);
    F2 y[8], x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = F2(act_of_word_any(hv.word(i), a.act));
      if (u != nullptr) y[i] = y[i] * uv.pair(i);
    }
    if (a.hq != nullptr) {
      pairs_of(hv, x);
      put_group_any<0>(x, hv.max_abs(), a.keep_sfmt, a.hq + flat, a.hs, at, in, owner);
    }
    if (a.uq != nullptr) {
      pairs_of(uv, x);
      put_group_any<0>(x, uv.max_abs(), a.keep_sfmt, a.uq + flat, a.us, at, in, owner);
    }
    if (a.out != nullptr && in)
      store16(static_cast<__nv_bfloat16 *>(a.out) + t.at(a.ld_out), y);
    if (a.scale != nullptr)
      put_tensor_any<F>(y, d, top, a.q + flat, in);
    else
      put_group_any<F>(y, max_abs16(y), a.sfmt, a.q + flat, a.scales, at, in, owner);
  }
  return top;
}

template <int A, bool GATE, int F>
__global__ void __launch_bounds__(kTileThreads, ctas_per_sm(GATE))
    act_checkpoint_kernel(const __grid_constant__ ActArgs a) {
  launch_dependents();
  grid_dependency_wait();
  const __nv_bfloat16 *h = static_cast<const __nv_bfloat16 *>(a.h);
  const __nv_bfloat16 *u = static_cast<const __nv_bfloat16 *>(a.u);
  const uint32_t rows = live_rows(a.valid, a.M), N = (uint32_t)a.N;
  const CodeScale d(a.scale != nullptr ? *a.scale : 1.0f);
  float top = 0.0f;
  uint32_t noted = 0u;
  TileWalk w(rows, N);
  if (!d.fast) {
    noted = ~0u;
    w.left = 0;
  }
  Words16 hn, un;  // the next tile's
  auto fetch = [&]() {
    const bool in = w.left > 0 && w.row < rows && w.col() < N;
    hn = load16(h + w.at(a.ldh), in);
    if constexpr (GATE) un = load16(u + w.at(a.ldu), in);
  };
  fetch();
  while (w.left > 0) {
    const TileWalk t = w;
    const int64_t at = t.scale_at(a.M), flat = t.at(a.N);
    const bool in = t.row < rows && t.col() < N, owner = t.row < rows && (threadIdx.x & 7u) == 0u;
    const Words16 hv = hn;
    Words16 uv;
    if constexpr (GATE) uv = un;
    w.next();
    fetch();
    // (the checkpoints first: the results' registers are not needed for them)
    F2 y[8];
    bool fast = true;
    if (a.hq != nullptr) {
      pairs_of(hv, y);
      fast = put_group<0>(y, hv.max_abs(), a.keep_sfmt, a.hq + flat, a.hs, at, in, owner);
      if constexpr (GATE) {
        if (a.uq != nullptr) {
          pairs_of(uv, y);
          fast &= put_group<0>(y, uv.max_abs(), a.keep_sfmt, a.uq + flat, a.us, at, in, owner);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = act_of_word<A>(hv.word(i));
      if constexpr (GATE) y[i] = y[i] * uv.pair(i);
    }
    if (a.out != nullptr && in)
      store16(static_cast<__nv_bfloat16 *>(a.out) + t.at(a.ld_out), y);
    if (a.scale != nullptr)
      put_tensor<F>(y, d, top, a.q + flat, in);
    else
      fast &= put_group<F>(y, max_abs16(y), a.sfmt, a.q + flat, a.scales, at, in, owner);
    if (!__all_sync(0xffffffffu, fast)) note_tile(noted, t.step(rows));
  }
  if (__any_sync(0xffffffffu, noted != 0u)) top = act_slow_walk<F>(a, rows, top, noted);
  if (a.amax != nullptr) block_max_to(__float_as_uint(top), a.amax);
}

// The loop's forms hold for checkpoints of values up to this.
constexpr float kKeptScaleMax = 0x1p40f;

// The tiles that this warp has noted, again.
template <int F>
__device__ __noinline__ void act_grad_slow_walk(const ActGradArgs &a, uint32_t rows, uint32_t noted,
                                                float &top_h, float &top_u) {
  const __nv_bfloat16 *da = static_cast<const __nv_bfloat16 *>(a.da);
  const uint32_t N = (uint32_t)a.N;
  const bool gate = a.uq != nullptr;
  const CodeScale dh(a.scale_h != nullptr ? *a.scale_h : 1.0f);
  const CodeScale du(a.scale_u != nullptr ? *a.scale_u : 1.0f);
  uint32_t step = 0u;
#pragma unroll 1
  for (TileWalk t(rows, N); t.left > 0; t.next(), ++step) {
    if (!tile_noted(noted, step)) continue;
    const int64_t at = t.scale_at(a.M), flat = t.at(a.N);
    const bool in = t.row < rows && t.col() < N, owner = t.row < rows && (threadIdx.x & 7u) == 0u;
    const Words16 v = load16(da + t.at(a.ld_da), in);
    Vec16<uint8_t> hc, uc;
    hc.zero();
    uc.zero();
    float hs = 0.0f, us = 0.0f;
    if (in) {
      hc.load(a.hq + flat);
      if (gate) uc.load(a.uq + flat);
      hs = a.keep_sfmt == 0 ? kept_scale<0>(kept_bits<0>(a.hs, at))
                            : kept_scale<1>(kept_bits<1>(a.hs, at));
      if (gate)
        us = a.keep_sfmt == 0 ? kept_scale<0>(kept_bits<0>(a.us, at))
                              : kept_scale<1>(kept_bits<1>(a.us, at));
    }
    F2 yh[8], yu[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const F2 z = kept_pair(hc.w[0], i, F2(hs)), g = v.pair(i);
      const BothBits both = act_both_any(z.v, a.act, hs <= kKeptScaleMax);
      yu[i] = g * F2(both.value);
      yh[i] = gate ? g * kept_pair(uc.w[0], i, F2(us)) * F2(both.slope) : g * F2(both.slope);
    }
    if (a.dh != nullptr && in) store16(static_cast<__nv_bfloat16 *>(a.dh) + t.at(a.ld_d), yh);
    if (a.du != nullptr && in) store16(static_cast<__nv_bfloat16 *>(a.du) + t.at(a.ld_d), yu);
    const int64_t qat = t.at(a.ld_q);
    if (a.tensor != 0) {
      if (a.qh != nullptr) put_tensor_any<F>(yh, dh, top_h, a.qh + qat, in);
      if (a.qu != nullptr) put_tensor_any<F>(yu, du, top_u, a.qu + qat, in);
    } else {
      if (a.qh != nullptr)
        put_group_any<F>(yh, max_abs16(yh), a.sfmt, a.qh + qat, a.sh, at, in, owner);
      if (a.qu != nullptr)
        put_group_any<F>(yu, max_abs16(yu), a.sfmt, a.qu + qat, a.su, at, in, owner);
    }
  }
}

template <int A, bool GATE, int F, int KEPT>
__global__ void __launch_bounds__(kTileThreads, ctas_per_sm(GATE))
    act_checkpoint_grad_kernel(const __grid_constant__ ActGradArgs a) {
  launch_dependents();
  grid_dependency_wait();
  const __nv_bfloat16 *da = static_cast<const __nv_bfloat16 *>(a.da);
  const uint32_t rows = live_rows(a.valid, a.M), N = (uint32_t)a.N;
  const bool tensor = a.tensor != 0;
  const CodeScale dh(a.scale_h != nullptr ? *a.scale_h : 1.0f);
  const CodeScale du(a.scale_u != nullptr ? *a.scale_u : 1.0f);
  float top_h = 0.0f, top_u = 0.0f;
  uint32_t noted = 0u;
  TileWalk w(rows, N);
  if (!(dh.fast && du.fast)) {
    noted = ~0u;
    w.left = 0;
  }
  Words16 vn;  // the next tile's operands
  Vec16<uint8_t> hn, un;
  uint32_t hsn = 0u, usn = 0u;
  auto fetch = [&]() {
    const int64_t at = w.scale_at(a.M), flat = w.at(a.N);
    const bool in = w.left > 0 && w.row < rows && w.col() < N;
    vn = load16(da + w.at(a.ld_da), in);
    hn.zero();
    un.zero();
    hsn = usn = 0u;
    if (in) {
      hn.load(a.hq + flat);
      hsn = kept_bits<KEPT>(a.hs, at);
      if constexpr (GATE) {
        un.load(a.uq + flat);
        usn = kept_bits<KEPT>(a.us, at);
      }
    }
  };
  fetch();
  while (w.left > 0) {
    const TileWalk t = w;
    const int64_t at = t.scale_at(a.M);
    const bool in = t.row < rows && t.col() < N;
    const Words16 v = vn;
    const Vec16<uint8_t> hc = hn, uc = un;
    const float hs = kept_scale<KEPT>(hsn), us = kept_scale<KEPT>(usn);
    w.next();
    fetch();
    if (!__all_sync(0xffffffffu, hs <= kKeptScaleMax)) {
      note_tile(noted, t.step(rows));
      continue;
    }
    F2 yh[8], yu[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      act_both2<A>(kept_pair(hc.w[0], i, F2(hs)), yu[i], yh[i]);
      const F2 g = v.pair(i);
      if constexpr (GATE) {
        yh[i] = g * kept_pair(uc.w[0], i, F2(us)) * yh[i];
        yu[i] = g * yu[i];
      } else {
        yh[i] = g * yh[i];
      }
    }
    if (a.dh != nullptr && in) store16(static_cast<__nv_bfloat16 *>(a.dh) + t.at(a.ld_d), yh);
    if (GATE && a.du != nullptr && in)
      store16(static_cast<__nv_bfloat16 *>(a.du) + t.at(a.ld_d), yu);
    const int64_t qat = t.at(a.ld_q);
    const bool live = t.row < rows;
    bool fast = true;
    if (tensor) {
      if (a.qh != nullptr) put_tensor<F>(yh, dh, top_h, a.qh + qat, in);
      if (GATE && a.qu != nullptr) put_tensor<F>(yu, du, top_u, a.qu + qat, in);
    } else if (GATE && a.qh != nullptr && a.qu != nullptr) {
      fast = put_groups<F>(yh, yu, a.sfmt, a.qh + qat, a.qu + qat, a.sh, a.su, at, in, live);
    } else {
      const bool owner = live && (threadIdx.x & 7u) == 0u;
      if (a.qh != nullptr)
        fast = put_group<F>(yh, max_abs16(yh), a.sfmt, a.qh + qat, a.sh, at, in, owner);
      if (GATE && a.qu != nullptr)
        fast &= put_group<F>(yu, max_abs16(yu), a.sfmt, a.qu + qat, a.su, at, in, owner);
      fast = __all_sync(0xffffffffu, fast);
    }
    if (!fast) note_tile(noted, t.step(rows));
  }
  if (__any_sync(0xffffffffu, noted != 0u)) {
    float th = top_h, tu = top_u;
    act_grad_slow_walk<F>(a, rows, noted, th, tu);
    top_h = th;
    top_u = tu;
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

// Resident CTAs, times as many as keep each walk within kMostTiles.
static int64_t tile_blocks(int64_t M, int64_t N, int64_t most) {
  const int64_t tiles = (M + 31) / 32 * ((N + 127) / 128), full = most * kMostTiles;
  return tiles < most ? tiles : most * ((tiles + full - 1) / full);
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
  const int64_t blocks = tile_blocks(a.M, a.N, (int64_t)sms * ctas_per_sm(a.u != nullptr));
  each_act(a.act, [&](auto act) {
    with_gate(a.u != nullptr, a.fmt, [&](auto gate, auto fmt) {
      e = launch_serial(act_checkpoint_kernel<act.value, gate.value, fmt.value>, blocks,
                        kTileThreads, st, a);
    });
  });
  return e;
}

cudaError_t launch_act_checkpoint_grad(const ActGradArgs &a, int sms, cudaStream_t st) {
  cudaError_t e = clear_maxima(a.amax_h, a.amax_u, st);
  if (e != cudaSuccess || a.M == 0) return e;
  const int64_t blocks = tile_blocks(a.M, a.N, (int64_t)sms * ctas_per_sm(a.uq != nullptr));
  each_act(a.act, [&](auto act) {
    with_gate(a.uq != nullptr, a.fmt, [&](auto gate, auto fmt) {
      e = a.keep_sfmt == 0
              ? launch_serial(act_checkpoint_grad_kernel<act.value, gate.value, fmt.value, 0>, blocks,
                              kTileThreads, st, a)
              : launch_serial(act_checkpoint_grad_kernel<act.value, gate.value, fmt.value, 1>, blocks,
                              kTileThreads, st, a);
    });
  });
  return e;
}

}  // namespace fp8k
