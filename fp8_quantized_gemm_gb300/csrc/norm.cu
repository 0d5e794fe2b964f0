// Root-mean-square norm around the FP8 products of a transformer block.
//
// Forward: r = T(x + residual), inv = 1 / sqrt(mean(r^2) + eps), y = r inv w,
// and the FP8 codes of y.  The sum is rounded to the stream's type T before
// it is normalised, so that the row the backward pass reads from memory is
// the row that was normalised; y itself is rounded once, from fp32 to its
// code (and once to bf16 where the caller wants that copy too).
//
// Backward (y's quantization passes the gradient through): with g = dy w and
// xhat = r inv,
//   dx = inv (g - xhat mean(g xhat)) + d_residual,   dw = sum over rows of dy xhat.
//
// Both are bound by HBM: every operand is touched once, the row stays in
// registers between the reduction and the scaling.  A CTA takes one row at a
// time (thread t owns the 8-element vectors t, t + T, ...: 16-byte accesses,
// and a 1x128 group is 16 neighbouring lanes, a 1x32 block four), reduces it
// with one barrier (the partial sums alternate between two buffers), and has
// the loads of its next row in flight meanwhile.  Measured (HBM's copy rate
// 6690 GB/s): forward 16384 x 4096 with residual and per-tensor codes 75.4 us,
// 93% of it; 1x128 groups 76-78 us, one-level MX 82 (their scales go out a few
// bytes at a time, a row of the group-major layout each); an fp32 stream 143-151
// (86-91%: two vectors of fp32 per thread spill a few registers of the 64).
// Backward with codes and dw 102-103 us, 88%; an fp32 stream 180 (95%).  Rows of
// more than 8192 elements take four vectors per thread, which leaves no
// registers to prefetch the next row: 4096 x 14336 126-128 us (62%), fp32 235
// (64%).  For the backward pass
// a ring of rows in shared memory filled by bulk copies measured 101-104 us
// at 4096 columns and 135 at 2048 (a row's chain of reduction, barrier and
// second pass bounds it, not the bytes in flight).
#include "common.cuh"
#include "kernels.h"
#include "norm.h"
#include "pairs.cuh"
#include "quant_common.cuh"

namespace fp8k {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the CTA, the same bits in every thread.  `red` is this row's
// buffer of the two: a thread that writes it again has passed the next row's
// barrier, behind every read of it.
__device__ __forceinline__ float block_sum(float v, float *red) {
  v = warp_sum(v);
  const uint32_t nw = blockDim.x >> 5;
  if (nw == 1) return v;
  if (lane_id() == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane_id() < nw ? red[lane_id()] : 0.0f);
}

// The four pairs of a raw vector.
template <typename T>
__device__ __forceinline__ F2 pair_of(const Raw8<T> &r, int i) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
    return bf16_pair(w[i]);
  } else {
    const uint4 &u = r.w[i >> 1];
    return i & 1 ? F2(__uint_as_float(u.z), __uint_as_float(u.w))
                 : F2(__uint_as_float(u.x), __uint_as_float(u.y));
  }
}

// Four pairs rounded to T, as stored.
template <typename T>
__device__ __forceinline__ Raw8<T> pack(const F2 (&v)[4]) {
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

// x + y, each sum rounded once to T (bf16: packed bf16 additions, exact up to
// that rounding).
template <typename T>
__device__ __forceinline__ Raw8<T> add(const Raw8<T> &x, const Raw8<T> &y) {
  if constexpr (sizeof(T) == 2) {
    auto sum = [](uint32_t a, uint32_t b) {
      const __nv_bfloat162 h = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                          *reinterpret_cast<const __nv_bfloat162 *>(&b));
      return *reinterpret_cast<const uint32_t *>(&h);
    };
    Raw8<T> r;
    r.w[0] = make_uint4(sum(x.w[0].x, y.w[0].x), sum(x.w[0].y, y.w[0].y),
                        sum(x.w[0].z, y.w[0].z), sum(x.w[0].w, y.w[0].w));
    return r;
  } else {
    const F2 v[4] = {pair_of(x, 0) + pair_of(y, 0), pair_of(x, 1) + pair_of(y, 1),
                     pair_of(x, 2) + pair_of(y, 2), pair_of(x, 3) + pair_of(y, 3)};
    return pack<T>(v);
  }
}

template <typename T>
__device__ __forceinline__ void store_raw8(T *p, const Raw8<T> &r) {
#pragma unroll
  for (int i = 0; i < Raw8<T>::kWords; ++i) reinterpret_cast<uint4 *>(p)[i] = r.w[i];
}

// Eight gains as pairs (w null: ones).  They are re-read per row: K values
// that stay in L1.  (Plain loads here and of inv: the previous kernel, still
// running when this one starts, may write them, and what
// grid_dependency_wait() makes visible does not cover the read-only path.)
__device__ __forceinline__ void load_gain8(const void *w, int w_dt, int64_t c, F2 (&g)[4]) {
  if (w == nullptr) {
#pragma unroll
    for (int j = 0; j < 4; ++j) g[j] = F2(1.0f);
  } else if (w_dt == 0) {
    const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(w) + c);
    g[0] = bf16_pair(u.x); g[1] = bf16_pair(u.y); g[2] = bf16_pair(u.z); g[3] = bf16_pair(u.w);
  } else {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(w) + c);
    const float4 a = p[0], b = p[1];
    g[0] = F2(a.x, a.y); g[1] = F2(a.z, a.w); g[2] = F2(b.x, b.y); g[3] = F2(b.z, b.w);
  }
}

__device__ __forceinline__ uint2 codes8(const F2 (&y)[4], const CodeScale &d, int fmt) {
  float z[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) d.quotient(y[j]).get(z[2 * j], z[2 * j + 1]);
  return pack8(fmt, z);
}

// Codes of eight values under the power of two 2^e.
__device__ __forceinline__ uint2 codes8_pow2(const F2 (&y)[4], int e, int fmt) {
  const F2 inv(exp2_int(-e));
  float z[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) (y[j] * inv).get(z[2 * j], z[2 * j + 1]);
  return pack8(fmt, z);
}

// Exponent of the smallest power of two not below amax / MAX, clamped to a
// UE8M0 byte's range (0 for an all-zero or NaN amax: scale 1).
__device__ __forceinline__ int ue8m0_exp(float amax, float mx) {
  return amax > 0.0f ? min(max(ceil_log2_pos(__fdiv_rn(amax, mx)), -127), 127) : 0;
}

// The CTA's max |x|: whole into *slot where one is given, else into *dst,
// cleared before the launch.
__device__ __forceinline__ void put_amax(float amax, uint32_t *dst, uint32_t *slot) {
  if (slot != nullptr) {
    __shared__ uint32_t top;
    if (threadIdx.x == 0) top = 0u;
    __syncthreads();
    const uint32_t k = warp_max_u32(__float_as_uint(amax));
    if (lane_id() == 0) atomicMax(&top, k);
    __syncthreads();
    if (threadIdx.x == 0) *slot = top;
  } else {
    block_max_to(__float_as_uint(amax), dst);
  }
}

// ---------------------------------------------------------------- forward --
template <typename T, int MODE, int V>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormArgs a) {
  __shared__ float red[2][32];
  launch_dependents();
  grid_dependency_wait();
  const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
  T *sum = static_cast<T *>(a.sum);
  const float mx = fmt_max(a.fmt);
  const CodeScale dt(MODE == kNormTensor ? *a.scale : 1.0f);
  float top = 0.0f;  // kNormTensor: running max |y|
  // the block-scaled layout also holds words for the rows that pad M to 128
  const int64_t rows = MODE == kNormMx ? (a.M + 127) / 128 * 128 : a.M;

  int64_t col[V];
#pragma unroll
  for (int i = 0; i < V; ++i) col[i] = 8 * ((int64_t)i * blockDim.x + threadIdx.x);
  Raw8<T> xr[V], rr[V];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      xr[i].zero();
      rr[i].zero();
      if (col[i] < a.K) {
        xr[i].load_stream(x + row * a.ldx + col[i]);
        if (res != nullptr) rr[i].load_stream(res + row * a.ldr + col[i]);
      }
    }
  };
  int64_t row = blockIdx.x;
  if (row < a.M) fetch(row);
  for (int phase = 0; row < rows; row += gridDim.x, phase ^= 1) {
    if (MODE == kNormMx && row >= a.M) {  // a padding row (the same branch in every thread)
      uint32_t *words = static_cast<uint32_t *>(a.scales);
      for (int64_t g = threadIdx.x; g < a.K / 128; g += blockDim.x)
        words[g * rows + (row & ~127) + 4 * (row % 32) + (row % 128) / 32] = 0x7F7F7F7Fu;
      continue;
    }
    Raw8<T> r[V];
    F2 ss(0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      r[i] = res != nullptr ? add(xr[i], rr[i]) : xr[i];
      if (sum != nullptr && col[i] < a.K) store_raw8(sum + row * a.ld_sum + col[i], r[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) ss = fma2(pair_of(r[i], j), pair_of(r[i], j), ss);
    }
    if (row + gridDim.x < a.M) fetch(row + gridDim.x);
    float s0, s1;
    ss.get(s0, s1);
    const float inv = rsqrtf(fmaf(block_sum(s0 + s1, red[phase]), a.inv_k, a.eps));
    if (a.inv_rms != nullptr && threadIdx.x == 0) a.inv_rms[row] = inv;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      // (every lane of a warp takes part in the group reductions; a lane past
      // the row's end holds zeros)
      const bool in = col[i] < a.K;
      if (MODE == kNormTensor && !in) continue;
      F2 y[4];
      if (in) {
        load_gain8(a.w, a.w_dt, col[i], y);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = (pair_of(r[i], j) * F2(inv)) * y[j];
      }
      uint2 c;
      if constexpr (MODE == kNormTensor) {
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max_abs2(top, y[j]);
        c = codes8(y, dt, a.fmt);
      } else {
        float m8 = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) m8 = max_abs2(m8, y[j]);
        uint32_t k8 = __float_as_uint(m8);
        constexpr int kLanes = MODE == kNormGroup ? 16 : 4;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
          k8 = max(k8, __shfl_xor_sync(0xffffffffu, k8, o));
        const float amax = __uint_as_float(k8);
        if constexpr (MODE == kNormGroup) {
          const bool owner = (threadIdx.x & 15u) == 0 && in;
          const int64_t at = (col[i] >> 7) * a.M + row;
          if (a.sfmt == 0) {
            const float s = scale_from_amax(amax, mx);
            if (owner) static_cast<float *>(a.scales)[at] = s;
            c = codes8(y, CodeScale(s), a.fmt);
          } else {
            const int e = ue8m0_exp(amax, mx);
            if (owner) static_cast<uint8_t *>(a.scales)[at] = (uint8_t)(e + 127);
            c = codes8_pow2(y, e, a.fmt);
          }
        } else {
          const int e = ue8m0_exp(amax, mx);
          uint32_t word = (uint32_t)(e + 127) << (8 * ((threadIdx.x >> 2) & 3u));
          word |= __shfl_xor_sync(0xffffffffu, word, 4);
          word |= __shfl_xor_sync(0xffffffffu, word, 8);
          if ((threadIdx.x & 15u) == 0 && in)
            static_cast<uint32_t *>(a.scales)[(col[i] >> 7) * rows + (row & ~127) +
                                              4 * (row % 32) + (row % 128) / 32] = word;
          c = codes8_pow2(y, e, a.fmt);
        }
        if (!in) continue;
      }
      *reinterpret_cast<uint2 *>(a.q + row * a.K + col[i]) = c;
      if (a.y != nullptr)
        store_raw8(static_cast<__nv_bfloat16 *>(a.y) + row * a.ld_y + col[i], pack<__nv_bfloat16>(y));
    }
  }
  if (MODE == kNormTensor && a.amax != nullptr)
    put_amax(top, a.amax, gridDim.x == 1 ? a.amax : nullptr);
}

// --------------------------------------------------------------- backward --
// Thread t's columns are the same for every row, so its share of dw stays in
// registers over all the rows its CTA takes; each CTA then writes one row of
// partial sums, and column_sum_kernel adds those in a fixed order (no atomic:
// the same bits on every run).
template <typename T, typename DY, int V>
__global__ void __launch_bounds__(512, 1) rmsnorm_grad_kernel(const NormGradArgs a) {
  // next row in flight while this one is reduced, where the registers allow
  // (4096 x 14336: 130 us without, 140 with)
  constexpr bool kPrefetch = V <= 2;
  __shared__ float red[2][32];
  launch_dependents();
  grid_dependency_wait();
  const T *r = static_cast<const T *>(a.r), *dres = static_cast<const T *>(a.dres);
  const DY *dy = static_cast<const DY *>(a.dy);
  T *dx = static_cast<T *>(a.dx);
  const CodeScale d(a.q != nullptr ? *a.scale : 1.0f);
  float top = 0.0f;  // running max |dx|
  int64_t col[V];
  F2 dw[V][4];
#pragma unroll
  for (int i = 0; i < V; ++i) col[i] = 8 * ((int64_t)i * blockDim.x + threadIdx.x);
  // the gains of this thread's columns stay in registers (read again in both
  // passes of every row they cost 5 us of 109)
  F2 gain[V][4];
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (col[i] < a.K) load_gain8(a.w, a.w_dt, col[i], gain[i]);
  Raw8<DY> yr[V];
  Raw8<T> rr[V], er[V];
  float inv = 0.0f;
  auto fetch = [&](int64_t row) {
    inv = a.inv_rms[row];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      yr[i].zero();
      rr[i].zero();
      er[i].zero();
      if (col[i] < a.K) {
        yr[i].load_stream(dy + row * a.ld_dy + col[i]);
        rr[i].load_stream(r + row * a.ld_r + col[i]);
        if (dres != nullptr) er[i].load_stream(dres + row * a.ld_dres + col[i]);
      }
    }
  };
  int64_t row = blockIdx.x;
  if (kPrefetch && row < a.M) fetch(row);
  for (int phase = 0; row < a.M; row += gridDim.x, phase ^= 1) {
    if (!kPrefetch) fetch(row);
    // the row stays in registers as loaded (half the size of its products)
    Raw8<DY> y0[V];
    Raw8<T> r0[V], e0[V];
    const float inv0 = inv;
    F2 dot(0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      y0[i] = yr[i];
      r0[i] = rr[i];
      e0[i] = er[i];
      if (col[i] >= a.K) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 t = pair_of(y0[i], j) * (pair_of(r0[i], j) * F2(inv0));  // dy xhat
        dw[i][j] = dw[i][j] + t;
        dot = fma2(t, gain[i][j], dot);
      }
    }
    if (kPrefetch && row + gridDim.x < a.M) fetch(row + gridDim.x);
    float d0, d1;
    dot.get(d0, d1);
    const float c = block_sum(d0 + d1, red[phase]) * a.inv_k;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (col[i] >= a.K) continue;
      F2 g[4];
      const F2 mc(-c), i2(inv0);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        g[j] = fma2(i2, fma2(pair_of(r0[i], j) * i2, mc, pair_of(y0[i], j) * gain[i][j]),
                    pair_of(e0[i], j));
      if (a.q != nullptr) {
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max_abs2(top, g[j]);
        *reinterpret_cast<uint2 *>(a.q + row * a.K + col[i]) = codes8(g, d, a.fmt);
      }
      store_raw8(dx + row * a.ld_dx + col[i], pack<T>(g));
    }
  }
  if (a.parts != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (col[i] >= a.K) continue;
      store_raw8(a.parts + (int64_t)blockIdx.x * a.K + col[i], pack<float>(dw[i]));
    }
  }
  if (a.q != nullptr && a.amax != nullptr)
    put_amax(top, a.amax, a.tops != nullptr ? a.tops + blockIdx.x : nullptr);
}

// out[n] (+)= sum over p < P of parts[p][n], in a fixed order: 32 columns per
// CTA, warp w adds rows w, w + 32, ..., then the 32 warps' sums are added.
// The first CTA also finishes a maximum: *top_out = max of tops[0 .. ntops)
// (keys of non-negative floats; nullable).  (parts and tops are not declared
// __restrict__: the previous kernel may still be writing them when this one
// starts, and const __restrict__ data may be read through the read-only path.)
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *parts, int64_t P, int64_t N,
                                                          int accumulate, float *out,
                                                          const uint32_t *tops, int ntops,
                                                          uint32_t *top_out) {
  __shared__ float s[32][33];
  __shared__ uint32_t top;
  if (threadIdx.x == 0) top = 0u;
  launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * 32 + lane;
  float acc = 0.0f;
  if (n < N) {
#pragma unroll 8
    for (int64_t p = w; p < P; p += 32) acc += __ldcg(parts + p * N + n);
  }
  s[w][lane] = acc;
  __syncthreads();
  if (blockIdx.x == 0 && top_out != nullptr) {
    uint32_t k = 0u;
    for (int i = threadIdx.x; i < ntops; i += 1024) k = max(k, __ldcg(tops + i));
    k = warp_max_u32(k);
    if (lane == 0) atomicMax(&top, k);
    __syncthreads();
    if (threadIdx.x == 0) *top_out = top;
  }
  acc = warp_sum(s[lane][w]);  // column w of this CTA
  const int64_t m = (int64_t)blockIdx.x * 32 + w;
  if (lane == 0 && m < N) out[m] = accumulate ? out[m] + acc : acc;
}

// *p = 0 between two kernels that are launched with programmatic stream
// serialization (a memset node would end that chain: 3 us of a call against
// 1.5).
__global__ void clear_word_kernel(uint32_t *p) {
  launch_dependents();
  grid_dependency_wait();
  if (threadIdx.x == 0) *p = 0u;
}

// A launch with programmatic stream serialization (the kernels wait for the
// previous one before they touch memory).
template <typename... KArgs, typename... Args>
static cudaError_t launch_serial(void (*kern)(KArgs...), int64_t blocks, int threads,
                                 cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

static int round32(int64_t n) { return (int)((n + 31) / 32 * 32); }

cudaError_t launch_column_sum(const float *parts, int64_t P, int64_t N, int accumulate, float *out,
                              const float *tops, int ntops, uint32_t *top_out, cudaStream_t st) {
  return launch_serial(column_sum_kernel, (N + 31) / 32, 1024, st, parts, P, N, accumulate, out,
                       reinterpret_cast<const uint32_t *>(tops), ntops, top_out);
}

cudaError_t launch_clear_word(uint32_t *p, cudaStream_t st) {
  return launch_serial(clear_word_kernel, 1, 32, st, p);
}

// Vectors per thread of a K-element row: with a row per SM or fewer the row
// is spread over as many threads as it has vectors; otherwise two vectors
// each, so that several CTAs share an SM and one's loads cover another's
// barrier.
static int forward_vectors(int64_t M, int64_t K, int sms) {
  const int64_t vecs = K / 8;
  if (vecs > 1024) return 2;
  return M <= sms || vecs < 64 ? 1 : 2;
}

template <typename T, int MODE>
static cudaError_t run_norm(const NormArgs &a, int sms, cudaStream_t st) {
  const int v = forward_vectors(a.M, a.K, sms);
  const int threads = round32((a.K / 8 + v - 1) / v);
  const int64_t rows = MODE == kNormMx ? (a.M + 127) / 128 * 128 : a.M;
  // resident at once: 1024 threads of 64 registers
  int64_t blocks = (int64_t)sms * (1024 / threads);
  if (blocks > rows) blocks = rows;
  return v == 1 ? launch_serial(rmsnorm_kernel<T, MODE, 1>, blocks, threads, st, a)
                : launch_serial(rmsnorm_kernel<T, MODE, 2>, blocks, threads, st, a);
}

cudaError_t launch_rmsnorm(const NormArgs &a, int dt, int mode, int sms, cudaStream_t st) {
  if (a.amax != nullptr && a.M != 1) {  // one row is one CTA, which writes it whole
    const cudaError_t e = launch_clear_word(a.amax, st);
    if (e != cudaSuccess) return e;
  }
  if (a.M == 0) return cudaSuccess;
  if (dt == 0) {
    if (mode == kNormTensor) return run_norm<__nv_bfloat16, kNormTensor>(a, sms, st);
    if (mode == kNormGroup) return run_norm<__nv_bfloat16, kNormGroup>(a, sms, st);
    return run_norm<__nv_bfloat16, kNormMx>(a, sms, st);
  }
  if (mode == kNormTensor) return run_norm<float, kNormTensor>(a, sms, st);
  if (mode == kNormGroup) return run_norm<float, kNormGroup>(a, sms, st);
  return run_norm<float, kNormMx>(a, sms, st);
}

static int grad_vectors(int64_t K) {
  const int64_t vecs = K / 8;
  return vecs <= 64 ? 1 : vecs <= 1024 ? 2 : 4;
}

// CTAs (and rows of dw partials) of the backward pass on `sms` SMs: 512
// threads of 128 registers resident per SM.
int64_t rmsnorm_grad_blocks(int64_t M, int64_t K, int sms) {
  const int v = grad_vectors(K);
  const int64_t blocks = (int64_t)sms * max(1, 512 / round32((K / 8 + v - 1) / v));
  return blocks < M ? blocks : M;
}

template <typename T, typename DY>
static cudaError_t run_norm_grad(const NormGradArgs &a, int64_t blocks, cudaStream_t st) {
  const int v = grad_vectors(a.K);
  const int threads = round32((a.K / 8 + v - 1) / v);
  switch (v) {
    case 1: return launch_serial(rmsnorm_grad_kernel<T, DY, 1>, blocks, threads, st, a);
    case 2: return launch_serial(rmsnorm_grad_kernel<T, DY, 2>, blocks, threads, st, a);
    default: return launch_serial(rmsnorm_grad_kernel<T, DY, 4>, blocks, threads, st, a);
  }
}

cudaError_t launch_rmsnorm_grad(const NormGradArgs &a, int dt, int dy_dt, float *dw,
                                int accumulate, int sms, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  // the maximum: finished by the column sums' kernel, or by atomics
  if (a.q != nullptr && a.amax != nullptr && (a.M == 0 || a.tops == nullptr) &&
      (e = launch_clear_word(a.amax, st)) != cudaSuccess)
    return e;
  if (a.M == 0) {
    if (dw != nullptr && !accumulate) return cudaMemsetAsync(dw, 0, (size_t)a.K * 4, st);
    return cudaSuccess;
  }
  const int64_t blocks = rmsnorm_grad_blocks(a.M, a.K, sms);
  if (dt == 0)
    e = dy_dt == 0 ? run_norm_grad<__nv_bfloat16, __nv_bfloat16>(a, blocks, st)
                   : run_norm_grad<__nv_bfloat16, float>(a, blocks, st);
  else
    e = dy_dt == 0 ? run_norm_grad<float, __nv_bfloat16>(a, blocks, st)
                   : run_norm_grad<float, float>(a, blocks, st);
  if (e != cudaSuccess || dw == nullptr) return e;
  return launch_column_sum(a.parts, blocks, a.K, accumulate, dw,
                           reinterpret_cast<const float *>(a.tops), (int)blocks,
                           a.tops != nullptr ? a.amax : nullptr, st);
}

}  // namespace fp8k
