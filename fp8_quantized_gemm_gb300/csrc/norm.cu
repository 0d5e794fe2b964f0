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
// time (thread t owns the 8-element vectors t, t + T, ...: 16-byte loads, and
// a 1x128 group is 16 neighbouring lanes, an 1x32 block four), reduces it
// with one barrier (the partial sums alternate between two buffers), and has
// the loads of its next row in flight meanwhile.
#include "common.cuh"
#include "kernels.h"
#include "norm.h"
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

// Round eight values to T, in place, and pack them as stored.
template <typename T>
__device__ __forceinline__ Raw8<T> round_pack(float (&v)[8]) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    r.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
    r.decode(v);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r.w[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                          __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void store_raw8(T *p, const Raw8<T> &r) {
#pragma unroll
  for (int i = 0; i < Raw8<T>::kWords; ++i) reinterpret_cast<uint4 *>(p)[i] = r.w[i];
}

// Eight gains (w null: ones).  They are re-read per row: K values that stay
// in L1.
__device__ __forceinline__ void load_gain8(const void *w, int w_dt, int64_t c, float (&g)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = 1.0f;
  } else if (w_dt == 0) {
    Vec8<__nv_bfloat16>::load(static_cast<const __nv_bfloat16 *>(w) + c, g);
  } else {
    Vec8<float>::load(static_cast<const float *>(w) + c, g);
  }
}

__device__ __forceinline__ uint32_t max_key8(const float (&y)[8]) {
  uint32_t k = abs_key(y[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) k = max(k, abs_key(y[j]));
  return k;
}

__device__ __forceinline__ uint2 codes8(const float (&y)[8], const ScaleDiv &d, int fmt) {
  float z[8];
  div8(d, y, z);
  return pack8(fmt, z);
}

// Codes of eight values under the power of two 2^e.
__device__ __forceinline__ uint2 codes8_pow2(const float (&y)[8], int e, int fmt) {
  const float inv = exp2_int(-e);
  float z[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) z[j] = __fmul_rn(y[j], inv);
  return pack8(fmt, z);
}

// Exponent of the smallest power of two not below amax / MAX, clamped to a
// UE8M0 byte's range (0 for an all-zero or NaN amax: scale 1).
__device__ __forceinline__ int ue8m0_exp(float amax, float mx) {
  return amax > 0.0f ? min(max(ceil_log2_pos(__fdiv_rn(amax, mx)), -127), 127) : 0;
}

// ---------------------------------------------------------------- forward --
template <typename T, int MODE, int V>
__global__ void __launch_bounds__(V == 4 ? 512 : 1024) rmsnorm_kernel(const NormArgs a) {
  __shared__ float red[2][32];
  launch_dependents();
  grid_dependency_wait();
  const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
  T *sum = static_cast<T *>(a.sum);
  const float mx = fmt_max(a.fmt);
  const ScaleDiv dt(MODE == kNormTensor ? *a.scale : 1.0f);
  uint32_t key = 0;
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
    float r[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      xr[i].decode(r[i]);
      if (res != nullptr) {
        float b[8];
        rr[i].decode(b);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] += b[j];
        const Raw8<T> packed = round_pack<T>(r[i]);
        if (sum != nullptr && col[i] < a.K) store_raw8(sum + row * a.ld_sum + col[i], packed);
      } else if (sum != nullptr && col[i] < a.K) {
        store_raw8(sum + row * a.ld_sum + col[i], xr[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(r[i][j], r[i][j], ss);
    }
    if (row + gridDim.x < a.M) fetch(row + gridDim.x);
    const float inv = rsqrtf(fmaf(block_sum(ss, red[phase]), a.inv_k, a.eps));
    if (a.inv_rms != nullptr && threadIdx.x == 0) a.inv_rms[row] = inv;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      // (every lane of a warp takes part in the group reductions; a lane past
      // the row's end holds zeros)
      if constexpr (MODE == kNormTensor) {
        if (col[i] >= a.K) continue;
      }
      float y[8];
      if (col[i] < a.K) {
        load_gain8(a.w, a.w_dt, col[i], y);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(__fmul_rn(r[i][j], inv), y[j]);
      uint32_t k8 = max_key8(y);
      uint2 c;
      if constexpr (MODE == kNormTensor) {
        key = max(key, k8);
        c = codes8(y, dt, a.fmt);
      } else {
        constexpr int kLanes = MODE == kNormGroup ? 16 : 4;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
          k8 = max(k8, __shfl_xor_sync(0xffffffffu, k8, o));
        const float amax = __uint_as_float(k8);
        if constexpr (MODE == kNormGroup) {
          const bool owner = (threadIdx.x & 15u) == 0 && col[i] < a.K;
          const int64_t at = (col[i] >> 7) * a.M + row;
          if (a.sfmt == 0) {
            const float s = scale_from_amax(amax, mx);
            if (owner) static_cast<float *>(a.scales)[at] = s;
            c = codes8(y, ScaleDiv(s), a.fmt);
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
          if ((threadIdx.x & 15u) == 0 && col[i] < a.K)
            static_cast<uint32_t *>(a.scales)[(col[i] >> 7) * rows + (row & ~127) +
                                              4 * (row % 32) + (row % 128) / 32] = word;
          c = codes8_pow2(y, e, a.fmt);
        }
        if (col[i] >= a.K) continue;
      }
      *reinterpret_cast<uint2 *>(a.q + row * a.K + col[i]) = c;
      if (a.y != nullptr) {
        const Raw8<__nv_bfloat16> p = round_pack<__nv_bfloat16>(y);
        store_raw8(static_cast<__nv_bfloat16 *>(a.y) + row * a.ld_y + col[i], p);
      }
    }
  }
  if (MODE == kNormTensor && a.amax != nullptr) block_max_to(key, a.amax);
}

// --------------------------------------------------------------- backward --
// Thread t's columns are the same for every row, so its share of dw stays in
// registers over all the rows its CTA takes; each CTA then writes one row of
// partial sums, and column_sum_kernel adds those in a fixed order (no atomic:
// the same bits on every run).
template <typename T, typename DY, int V>
__global__ void __launch_bounds__(512, 1) rmsnorm_grad_kernel(const NormGradArgs a) {
  // next row in flight while this one is reduced, where the registers allow
  constexpr bool kPrefetch = V * (2 * sizeof(T) + sizeof(DY)) <= 16;
  __shared__ float red[2][32];
  launch_dependents();
  grid_dependency_wait();
  const T *r = static_cast<const T *>(a.r), *dres = static_cast<const T *>(a.dres);
  const DY *dy = static_cast<const DY *>(a.dy);
  T *dx = static_cast<T *>(a.dx);
  const ScaleDiv d(a.q != nullptr ? *a.scale : 1.0f);
  uint32_t key = 0;
  int64_t col[V];
  float dw[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    col[i] = 8 * ((int64_t)i * blockDim.x + threadIdx.x);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  Raw8<DY> yr[V];
  Raw8<T> rr[V], er[V];
  float inv = 0.0f;
  auto fetch = [&](int64_t row) {
    inv = __ldg(a.inv_rms + row);
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
    float g[V][8], xh[V][8];
    Raw8<T> er0[V];
    const float inv0 = inv;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float t[8];
      yr[i].decode(t);
      rr[i].decode(xh[i]);
      er0[i] = er[i];
      if (col[i] < a.K) {
        load_gain8(a.w, a.w_dt, col[i], g[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[i][j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] *= inv0;
        dw[i][j] = fmaf(t[j], xh[i][j], dw[i][j]);
        g[i][j] *= t[j];
        dot = fmaf(g[i][j], xh[i][j], dot);
      }
    }
    if (kPrefetch && row + gridDim.x < a.M) fetch(row + gridDim.x);
    const float c = block_sum(dot, red[phase]) * a.inv_k;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (col[i] >= a.K) continue;
      float e[8];
      er0[i].decode(e);
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = fmaf(inv0, fmaf(-xh[i][j], c, g[i][j]), e[j]);
      if (a.q != nullptr) {
        key = max(key, max_key8(e));
        *reinterpret_cast<uint2 *>(a.q + row * a.K + col[i]) = codes8(e, d, a.fmt);
      }
      store_raw8(dx + row * a.ld_dx + col[i], round_pack<T>(e));
    }
  }
  if (a.parts != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (col[i] >= a.K) continue;
      float4 *p = reinterpret_cast<float4 *>(a.parts + (int64_t)blockIdx.x * a.K + col[i]);
      p[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
      p[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
    }
  }
  if (a.q != nullptr && a.amax != nullptr) block_max_to(key, a.amax);
}

// out[n] (+)= sum over p < P of parts[p][n], in a fixed order: 32 columns per
// CTA, warp w adds rows w, w + 32, ..., then the 32 warps' sums are added.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *__restrict__ parts,
                                                          int64_t P, int64_t N, int accumulate,
                                                          float *__restrict__ out) {
  __shared__ float s[32][33];
  launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * 32 + lane;
  float acc = 0.0f;
  if (n < N) {
#pragma unroll 4
    for (int64_t p = w; p < P; p += 32) acc += __ldcg(parts + p * N + n);
  }
  s[w][lane] = acc;
  __syncthreads();
  acc = warp_sum(s[lane][w]);  // column w of this CTA
  const int64_t m = (int64_t)blockIdx.x * 32 + w;
  if (lane == 0 && m < N) out[m] = accumulate ? out[m] + acc : acc;
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
                              cudaStream_t st) {
  return launch_serial(column_sum_kernel, (N + 31) / 32, 1024, st, parts, P, N, accumulate, out);
}

// Vectors per thread of a K-element row: with a row per SM or fewer the row
// is spread over as many threads as it has vectors; otherwise two vectors
// each, so that several CTAs share an SM and one's loads cover another's
// barrier.
static int forward_vectors(int64_t M, int64_t K, int sms) {
  const int64_t vecs = K / 8;
  if (M <= sms) return vecs <= 1024 ? 1 : 2;
  if (vecs < 64) return 1;
  return vecs <= 1024 ? 2 : 4;
}

template <typename T, int MODE>
static cudaError_t run_norm(const NormArgs &a, int sms, cudaStream_t st) {
  const int v = forward_vectors(a.M, a.K, sms);
  const int threads = round32((a.K / 8 + v - 1) / v);
  const int64_t rows = MODE == kNormMx ? (a.M + 127) / 128 * 128 : a.M;
  // resident at once: 1024 threads of 64 registers (V 1, 2), 512 of 128 (V 4)
  int64_t blocks = (int64_t)sms * max(1, (v == 4 ? 512 : 1024) / threads);
  if (blocks > rows) blocks = rows;
  switch (v) {
    case 1: return launch_serial(rmsnorm_kernel<T, MODE, 1>, blocks, threads, st, a);
    case 2: return launch_serial(rmsnorm_kernel<T, MODE, 2>, blocks, threads, st, a);
    default: return launch_serial(rmsnorm_kernel<T, MODE, 4>, blocks, threads, st, a);
  }
}

cudaError_t launch_rmsnorm(const NormArgs &a, int dt, int mode, int sms, cudaStream_t st) {
  if (a.amax != nullptr) {
    const cudaError_t e = cudaMemsetAsync(a.amax, 0, sizeof(uint32_t), st);
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
  return vecs <= 256 ? 1 : vecs <= 1024 ? 2 : 4;
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
  if (a.q != nullptr && a.amax != nullptr &&
      (e = cudaMemsetAsync(a.amax, 0, sizeof(uint32_t), st)) != cudaSuccess)
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
  return launch_column_sum(a.parts, blocks, a.K, accumulate, dw, st);
}

}  // namespace fp8k
