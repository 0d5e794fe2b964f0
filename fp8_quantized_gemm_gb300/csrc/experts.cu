// Tokens to their experts' rows and back, around the expert-grouped products.
//
// A token t has S choices; pair (t, s) owns one row of the products' operands.
// Rows are ordered by expert, and within one by (t, s):
//   sort      row(t, s) by a stable counting sort of the chosen experts
//   gather    row(t, s) <- codes of x[t] in 1x128 groups
//   combine   out[t] = residual[t] + sum over s of w[t, s] x[row(t, s)]
//   its gradient: row(t, s) <- codes of w[t, s] dy[t], dw[t, s] = <dy[t], x[row(t, s)]>
// A pair whose row lies outside [0, M) is dropped: nothing is read or written
// for it, and its dw is zero.  (The gradient of gather is combine with weights
// of one.)
//
// All but the sort are bound by HBM.  They walk the tokens, not the rows: what
// belongs to a token (x, dy, its groups' maxima) is read and formed once for
// its S rows.
#include "common.cuh"
#include "experts.h"
#include "kernels.h"
#include "launch.h"
#include "pairs.cuh"
#include "quant_common.cuh"
#include "rowvec.cuh"

namespace fp8k {

// ------------------------------------------------------------------- sort --
// One cluster of up to eight CTAs of 32 warps; warp g of it owns the g-th run
// of consecutive pairs.  A pass counts each warp's pairs per expert in shared
// memory, two prefix sums (over the warps of the cluster, the CTAs' totals
// exchanged through distributed shared memory, and over the experts) turn the
// counts into first rows, and a second pass hands the rows out in order: the
// lanes of 32 pairs that chose the same expert find each other with one match
// instruction.  No atomic decides an order, no scratch, one launch.
constexpr int kSortWarps = 32, kSortCluster = 8;

__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

template <typename ID>
__global__ void __launch_bounds__(32 * kSortWarps)
    experts_sort_kernel(const ID *ids, uint32_t P, int E, int32_t *offsets, int32_t *rows,
                        int32_t *pairs) {
  // (the odd pitch keeps the four rows that a warp reads in the prefix sum on
  // different banks)
  __shared__ uint32_t count[kSortWarps][kMaxExperts + 1];
  __shared__ uint32_t total[kMaxExperts];  // of this CTA; read by the whole cluster
  __shared__ uint32_t first[kMaxExperts];  // row of this CTA's first pair of each expert
  __shared__ uint32_t sums[kMaxExperts / 32];
  __shared__ uint32_t kept;                // pairs that have an expert
  launch_dependents();
  grid_dependency_wait();
  const uint32_t l = lane_id(), w = threadIdx.x >> 5;
  const uint32_t ctas = gridDim.x, rank = ctas > 1 ? cluster_ctarank() : 0u;
  const uint32_t warps = ctas * kSortWarps;
  const uint32_t per = (P + warps * 32 - 1) / (warps * 32) * 32;
  const uint32_t begin = min((rank * kSortWarps + w) * per, P), end = min(begin + per, P);
  uint32_t *const mine = count[w];
  // the expert of pair i; E for a dropped one
  auto expert = [&](uint32_t i) -> uint32_t {
    const ID id = ids[i];
    return id >= 0 && id < (ID)E ? (uint32_t)id : (uint32_t)E;
  };

  for (int e = l; e < E; e += 32) mine[e] = 0u;
  __syncwarp();
#pragma unroll 4
  for (uint32_t i = begin + l; i < end; i += 32) {
    const uint32_t e = expert(i);
    if (e < (uint32_t)E) atomicAdd(mine + e, 1u);
  }
  __syncthreads();

  {  // exclusive sums over the CTA's warps: four lanes per expert, eight warps each
    const int e = threadIdx.x >> 2, part = threadIdx.x & 3;
    uint32_t c[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = e < E ? count[8 * part + i][e] : 0u;
      sum += c[i];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o, 4);
      if (part >= o) incl += v;
    }
    uint32_t run = incl - sum;
    if (e < E) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        count[8 * part + i][e] = run;
        run += c[i];
      }
      if (part == 3) total[e] = incl;
    }
  }
  if (ctas > 1)
    cluster_sync();
  else
    __syncthreads();

  uint32_t all = 0, before = 0, incl = 0;
  if (threadIdx.x < kMaxExperts) {
    const int e = threadIdx.x;
    if (e < E) {
      if (ctas > 1) {
        const uint32_t at = smem_u32(total + e);
        for (uint32_t r = 0; r < ctas; ++r) {
          const uint32_t v = ld_shared_cluster_u32(mapa_shared(at, r));
          if (r < rank) before += v;
          all += v;
        }
      } else {
        all = total[e];
      }
    }
    incl = all;  // inclusive sum over the experts of this warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (l >= (uint32_t)o) incl += v;
    }
    if (l == 31) sums[w] = incl;
  }
  __syncthreads();
  if (threadIdx.x < kMaxExperts) {
    const int e = threadIdx.x;
    for (uint32_t i = 0; i < w; ++i) incl += sums[i];
    if (e < E) {
      first[e] = incl - all + before;
      if (rank == 0) offsets[e] = (int32_t)(incl - all);
      if (e == E - 1) {
        kept = incl;
        if (rank == 0) offsets[E] = (int32_t)incl;
      }
    }
  }
  __syncthreads();

  const uint32_t below = (1u << l) - 1u;
  uint32_t next = begin + l < end ? expert(begin + l) : (uint32_t)E;
  for (uint32_t i0 = begin; i0 < end; i0 += 32) {
    const uint32_t i = i0 + l, e = next;
    next = i + 32 < end ? expert(i + 32) : (uint32_t)E;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    uint32_t row = 0;
    if (e < (uint32_t)E) {
      row = first[e] + mine[e] + __popc(same & below);
      if (pairs != nullptr) pairs[row] = (int32_t)i;
    }
    if (i < end) rows[i] = e < (uint32_t)E ? (int32_t)row : -1;
    __syncwarp();
    if (e < (uint32_t)E && (same & below) == 0u) mine[e] += __popc(same);
    __syncwarp();
  }
  if (pairs != nullptr)
    for (uint32_t i = kept + rank * blockDim.x + threadIdx.x; i < P; i += ctas * blockDim.x)
      pairs[i] = -1;
  if (ctas > 1) cluster_sync();  // no CTA leaves while another may read its totals
}

cudaError_t launch_experts_sort(const void *ids, bool wide, int64_t P, int E, int32_t *offsets,
                                int32_t *rows, int32_t *pairs, cudaStream_t st) {
  const int ctas = P <= 4096 ? 1 : kSortCluster;
  if (wide)
    return launch_serial_cluster(experts_sort_kernel<int64_t>, ctas, 32 * kSortWarps, ctas, st,
                                 static_cast<const int64_t *>(ids), (uint32_t)P, E, offsets, rows,
                                 pairs);
  return launch_serial_cluster(experts_sort_kernel<int32_t>, ctas, 32 * kSortWarps, ctas, st,
                               static_cast<const int32_t *>(ids), (uint32_t)P, E, offsets, rows,
                               pairs);
}

// ----------------------------------------------------------------- gather --
// A warp per (token, 512 columns): lane l holds 16 consecutive elements, so
// eight lanes form a 1x128 group and each lane stores 16 bytes of codes per
// row.  The token's rows sit in the lanes, one each; a group's scale for eight
// rows goes out in one store instruction, one row per lane of the group.
template <typename T, int F>
__global__ void __launch_bounds__(256) experts_gather_kernel(const GatherArgs a) {
  constexpr bool kCodes = sizeof(T) == 1;
  launch_dependents();
  grid_dependency_wait();
  const uint32_t l = lane_id();
  const int64_t wins = (a.K + 511) / 512, tasks = a.T * wins;
  const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  const bool narrow = tasks <= (int64_t)0xFFFFFFFFu;
  const float mx = fmt_max(F);
  for (int64_t task = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; task < tasks;
       task += warps) {
    int64_t t, win;
    split_task(task, wins, narrow, t, win);
    const int64_t k = win * 512 + l * 16, g = k >> 7;
    const bool in = k < a.K;
    Vec16<T> v;
    if (in)
      v.load(static_cast<const T *>(a.x) + t * a.ldx + k);
    else
      v.zero();
    uint4 c = make_uint4(0u, 0u, 0u, 0u);
    uint32_t scale = 0u;  // bits of the fp32 scale, or the UE8M0 byte
    if constexpr (kCodes) {
      c = v.w[0];
      if (128 * g < a.K)  // (in a ragged last group also on the lanes past the row's end)
        scale = a.sfmt == 0 ? static_cast<const uint32_t *>(a.x_scales)[g * a.T + t]
                            : static_cast<const uint8_t *>(a.x_scales)[g * a.T + t];
    } else if (a.q != nullptr) {
      const float amax = __uint_as_float(group8_max(v.max_key()));
      if (a.sfmt == 0) {
        const float s = scale_from_amax(amax, mx);
        scale = __float_as_uint(s);
        c = v.template codes<F>(ScaleDiv(s));
      } else {
        const int e = ue8m0_exponent(amax, mx);
        scale = (uint32_t)(e + 127);
        c = v.template codes_pow2<F>(exp2_int(-e));
      }
    }
    for (int64_t s0 = 0; s0 < a.S; s0 += 32) {
      const int n = (int)min((int64_t)32, a.S - s0);
      const int32_t mine = (int)l < n ? a.rows[t * a.S + s0 + l] : -1;
      for (int s = 0; s < n; ++s) {
        const int64_t row = __shfl_sync(0xffffffffu, mine, s);
        if (row < 0 || row >= a.M || !in) continue;
        if (a.q != nullptr) *reinterpret_cast<uint4 *>(a.q + row * a.K + k) = c;
        if constexpr (!kCodes)
          if (a.out != nullptr) v.store(static_cast<T *>(a.out) + row * a.ld_out + k);
      }
      if (a.q == nullptr) continue;
      for (int s = 0; s < n; s += 8) {
        const int64_t row = __shfl_sync(0xffffffffu, mine, s + (int)(l & 7u));
        if (row < 0 || row >= a.M || 128 * g >= a.K) continue;
        if (a.sfmt == 0)
          static_cast<uint32_t *>(a.scales)[g * a.M + row] = scale;
        else
          static_cast<uint8_t *>(a.scales)[g * a.M + row] = (uint8_t)scale;
      }
    }
  }
}

static int64_t grid_of(int64_t warps, int per_block, int64_t most) {
  const int64_t blocks = (warps + per_block - 1) / per_block;
  return blocks < 1 ? 1 : blocks < most ? blocks : most;
}

template <typename T>
static cudaError_t run_gather(const GatherArgs &a, int sms, cudaStream_t st) {
  const int64_t blocks = grid_of(a.T * ((a.K + 511) / 512), 8, (int64_t)sms * 64);
  return a.fmt == 0 ? launch_serial(experts_gather_kernel<T, 0>, blocks, 256, st, a)
                    : launch_serial(experts_gather_kernel<T, 1>, blocks, 256, st, a);
}

cudaError_t launch_experts_gather(const GatherArgs &a, int source, int sms, cudaStream_t st) {
  if (a.T == 0 || a.M == 0) return cudaSuccess;
  if (source == kGatherCodes) {  // the format of codes that are moved does not matter
    GatherArgs b = a;
    b.fmt = 0;
    const int64_t blocks = grid_of(a.T * ((a.K + 511) / 512), 8, (int64_t)sms * 64);
    return launch_serial(experts_gather_kernel<uint8_t, 0>, blocks, 256, st, b);
  }
  return source == kGatherBf16 ? run_gather<__nv_bfloat16>(a, sms, st) : run_gather<float>(a, sms, st);
}

// ---------------------------------------------------------------- combine --
// A warp per (token, 256 columns), eight elements per lane; up to eight rows'
// loads in flight per lane.  Sums in fp32 in the order of the choices, the
// residual last, one rounding to the output's type.
template <typename T, typename O>
__global__ void __launch_bounds__(256) experts_combine_kernel(const CombineArgs a) {
  launch_dependents();
  grid_dependency_wait();
  const uint32_t l = lane_id();
  const T *x = static_cast<const T *>(a.x);
  const O *res = static_cast<const O *>(a.residual);
  const int64_t wins = (a.K + 255) / 256, tasks = a.T * wins;
  const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  const bool narrow = tasks <= (int64_t)0xFFFFFFFFu;
  for (int64_t task = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; task < tasks;
       task += warps) {
    int64_t t, win;
    split_task(task, wins, narrow, t, win);
    const int64_t k = win * 256 + l * 8;
    const bool in = k < a.K;
    Raw8<O> r;
    r.zero();
    if (res != nullptr && in) r.load_stream(res + t * a.ldr + k);
    F2 acc[4];
    for (int64_t s0 = 0; s0 < a.S; s0 += 32) {
      const int n = (int)min((int64_t)32, a.S - s0);
      int32_t row_l = -1;
      float w_l = 0.0f;  // a dropped pair: zero times zero
      if ((int)l < n) {
        row_l = a.rows[t * a.S + s0 + l];
        if (row_l < 0 || row_l >= a.M)
          row_l = -1;
        else
          w_l = a.weights != nullptr ? a.weights[t * a.S + s0 + l] : 1.0f;
      }
      for (int s = 0; s < n; s += 8) {
        Raw8<T> v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t row = __shfl_sync(0xffffffffu, row_l, (s + j) & 31);
          if (s + j < n && row >= 0 && in)
            v[j].load_stream(x + row * a.ldx + k);
          else
            v[j].zero();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float w = __shfl_sync(0xffffffffu, w_l, (s + j) & 31);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = fma2(F2(w), raw_pair(v[j], i), acc[i]);
        }
      }
    }
    if (!in) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = acc[i] + raw_pair(r, i);
    store8(static_cast<O *>(a.out) + t * a.ld_out + k, round8<O>(acc));
  }
}

template <typename T>
static cudaError_t run_combine(const CombineArgs &a, int out_dt, int sms, cudaStream_t st) {
  const int64_t blocks = grid_of(a.T * ((a.K + 255) / 256), 8, (int64_t)sms * 64);
  return out_dt == 0 ? launch_serial(experts_combine_kernel<T, __nv_bfloat16>, blocks, 256, st, a)
                     : launch_serial(experts_combine_kernel<T, float>, blocks, 256, st, a);
}

cudaError_t launch_experts_combine(const CombineArgs &a, int x_dt, int out_dt, int sms,
                                   cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  return x_dt == 0 ? run_combine<__nv_bfloat16>(a, out_dt, sms, st)
                   : run_combine<float>(a, out_dt, sms, st);
}

// ------------------------------------------------------- combine, gradient --
// A CTA per token, a warp per 512 columns of it (16 elements per lane, groups
// of eight lanes).  |w dy| of a group peaks where |dy| does (rounding is
// monotone), so the group's maximum of dy is taken once and lane j of the
// group forms the scale of the j-th of eight rows from it.  The eight rows'
// dot products stay in registers and are reduced together: a butterfly that
// halves the rows a lane still holds at each of its first three steps.
template <typename DY, typename X, int F>
__global__ void __launch_bounds__(512) experts_combine_grad_kernel(const CombineGradArgs a) {
  __shared__ float part[2][16][8];
  launch_dependents();
  grid_dependency_wait();
  const uint32_t l = lane_id(), w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const DY *dy = static_cast<const DY *>(a.dy);
  const X *x = static_cast<const X *>(a.x);
  const float mx = fmt_max(F);
  const int64_t wins = (a.K + 511) / 512;
  int phase = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    for (int64_t s0 = 0; s0 < a.S; s0 += 8) {
      const int n = (int)min((int64_t)8, a.S - s0);
      // lane j holds row and weight of choice s0 + j % 8
      const int j_l = (int)(l & 7u);
      int32_t row_l = -1;
      float w_l = 0.0f;
      if (j_l < n) {
        row_l = a.rows[t * a.S + s0 + j_l];
        if (row_l < 0 || row_l >= a.M) row_l = -1;
        w_l = a.weights != nullptr ? a.weights[t * a.S + s0 + j_l] : 1.0f;
      }
      float dot[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) dot[j] = 0.0f;
      for (int64_t win = w; win < wins; win += nw) {
        const int64_t k = win * 512 + l * 16, g = k >> 7;
        const bool in = k < a.K;
        Vec16<DY> v;
        if (in)
          v.load(dy + t * a.ld_dy + k);
        else
          v.zero();
        float inv_l = 0.0f, s_l = 1.0f;  // row j's scale, and its reciprocal
        bool fast = true;
        if (a.q != nullptr) {
          const float amax = fabsf(w_l) * __uint_as_float(group8_max(v.max_key()));
          const bool keep = row_l >= 0 && 128 * g < a.K;
          if (a.sfmt == 0) {
            s_l = scale_from_amax(amax, mx);
            if (keep) static_cast<float *>(a.scales)[g * a.M + row_l] = s_l;
          } else {
            const int e = ue8m0_exponent(amax, mx);
            s_l = exp2_int(e);
            if (keep) static_cast<uint8_t *>(a.scales)[g * a.M + row_l] = (uint8_t)(e + 127);
          }
          const CodeScale d(s_l);
          inv_l = d.inv;
          fast = __all_sync(0xffffffffu, d.fast);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t row = __shfl_sync(0xffffffffu, row_l, j);
          const float wj = __shfl_sync(0xffffffffu, w_l, j);
          const int from = (int)(l & 24u) | j;
          const float inv = __shfl_sync(0xffffffffu, inv_l, from);
          const float s = __shfl_sync(0xffffffffu, s_l, from);
          if (row < 0 || !in) continue;
          if (a.dw != nullptr) {
            Vec16<X> xv;
            xv.load(x + row * a.ldx + k);
            F2 d2(0.0f);
#pragma unroll
            for (int i = 0; i < 8; ++i) d2 = fma2(v.pair(i), xv.pair(i), d2);
            float d0, d1;
            d2.get(d0, d1);
            dot[j] += d0 + d1;
          }
          if (a.q == nullptr && a.dx == nullptr) continue;
          F2 y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = v.pair(i) * F2(wj);
          if (a.dx != nullptr) {
            if (a.dx_dt == 0)
              store16(static_cast<__nv_bfloat16 *>(a.dx) + row * a.ld_dx + k, y);
            else
              store16(static_cast<float *>(a.dx) + row * a.ld_dx + k, y);
          }
          if (a.q != nullptr) {
            uint4 c;
            if (fast) {
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] = y[i] * F2(inv);
              c = pack16<F>(y);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] = each(y[i], [s](float z) { return __fdiv_rn(z, s); });
              c = pack16<F>(y);
            }
            *reinterpret_cast<uint4 *>(a.q + row * a.K + k) = c;
          }
        }
      }
      if (a.dw == nullptr) continue;
      // rows 4 apart, 2 apart, 1 apart: lane l ends with row (l >> 2) & 7
#pragma unroll
      for (int h = 4; h > 0; h >>= 1) {
        const bool up = (l & (uint32_t)(4 * h)) != 0u;
#pragma unroll
        for (int j = 0; j < h; ++j) {
          const float keep = up ? dot[j + h] : dot[j], give = up ? dot[j] : dot[j + h];
          dot[j] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * h);
        }
      }
      float v = dot[0];
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      // (a buffer is written again two barriers after it was read)
      if ((l & 3u) == 0u) part[phase][w][l >> 2] = v;
      __syncthreads();
      if ((int)threadIdx.x < n) {
        float sum = 0.0f;
        for (uint32_t i = 0; i < nw; ++i) sum += part[phase][i][threadIdx.x];
        a.dw[t * a.S + s0 + threadIdx.x] = sum;
      }
      phase ^= 1;
    }
  }
}

template <typename DY, typename X>
static cudaError_t run_combine_grad(const CombineGradArgs &a, int sms, cudaStream_t st) {
  const int64_t wins = (a.K + 511) / 512;
  const int warps = (int)(wins < 16 ? wins : 16);
  const int64_t most = (int64_t)sms * 32;
  const int64_t blocks = a.T < most ? a.T : most;
  return a.fmt == 0
             ? launch_serial(experts_combine_grad_kernel<DY, X, 0>, blocks, 32 * warps, st, a)
             : launch_serial(experts_combine_grad_kernel<DY, X, 1>, blocks, 32 * warps, st, a);
}

cudaError_t launch_experts_combine_grad(const CombineGradArgs &a, int dy_dt, int x_dt, int sms,
                                        cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  if (dy_dt == 0)
    return x_dt == 0 ? run_combine_grad<__nv_bfloat16, __nv_bfloat16>(a, sms, st)
                     : run_combine_grad<__nv_bfloat16, float>(a, sms, st);
  return x_dt == 0 ? run_combine_grad<float, __nv_bfloat16>(a, sms, st)
                   : run_combine_grad<float, float>(a, sms, st);
}

}  // namespace fp8k
