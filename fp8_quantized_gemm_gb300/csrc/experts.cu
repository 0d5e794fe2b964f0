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
// One cluster of up to 16 CTAs of 32 warps; warp g of it owns the g-th run of
// consecutive pairs.  A first pass ranks each pair among its warp's pairs of the
// same expert: the lanes of 32 pairs that chose the same expert find each other by
// a vote per bit of the expert's number, and the counts so far sit in shared
// memory.  Two prefix sums (over the warps of the cluster, the CTAs' totals
// exchanged through distributed shared memory, and over the experts) turn the
// counts into first rows, which a second pass adds to the ranks.  A warp's pairs
// are loaded eight per lane at once, and stay in registers between the passes
// where that is all of them.  The pairs of the rows are scattered by a kernel of
// their own on all SMs (a scattered store takes a cycle per lane of one SM).  No
// atomic, no scratch.
//
// Bound by the instructions of the passes on the cluster's SMs: 131072 pairs of 256
// experts 11.3 us (17.3 on eight CTAs; with the match instruction in the place of
// the votes and the scatter in the same kernel 25), 512 pairs 3.5 us, most of it
// launch and latency.
constexpr int kSortWarps = 32, kSortCluster = 16, kSortRun = 8;

__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// lanes whose value (below 256) equals this lane's, of those that have one (a
// lane without gets a mask that means nothing)
__device__ __forceinline__ uint32_t lanes_alike(uint32_t v, bool has) {
  uint32_t same = __ballot_sync(0xffffffffu, has);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const bool one = (v & (1u << b)) != 0u;
    const uint32_t ones = __ballot_sync(0xffffffffu, one);
    same &= ones ^ (one ? 0u : 0xffffffffu);
  }
  return same;
}

// SCATTER: also write pairs (nullable); else experts_pairs_kernel does.
template <typename ID, bool SCATTER>
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
  const uint32_t ctas = gridDim.x, cta = ctas > 1 ? cluster_ctarank() : 0u;
  const uint32_t warps = ctas * kSortWarps;
  const uint32_t per = (P + warps * 32 - 1) / (warps * 32) * 32;
  const uint32_t begin = min((cta * kSortWarps + w) * per, P), end = min(begin + per, P);
  uint32_t *const mine = count[w];
  // the expert of pair i; E for a dropped one
  auto expert = [&](uint32_t i) -> uint32_t {
    const ID id = ids[i];
    return id >= 0 && id < (ID)E ? (uint32_t)id : (uint32_t)E;
  };

  for (int e = l; e < E; e += 32) mine[e] = 0u;
  __syncwarp();
  const uint32_t below = (1u << l) - 1u;
  // the experts and ranks of a batch of pairs; a warp's only batch stays here
  // between the passes, the ranks of others wait in rows
  const bool whole = per <= 32 * kSortRun;
  uint32_t e[kSortRun];
  int32_t rank[kSortRun];
  auto load = [&](uint32_t i0) {
#pragma unroll
    for (int j = 0; j < kSortRun; ++j) {
      const uint32_t i = i0 + 32 * j + l;
      e[j] = i < end ? expert(i) : (uint32_t)E;
    }
  };
  for (uint32_t i0 = begin; i0 < end; i0 += 32 * kSortRun) {
    load(i0);
#pragma unroll
    for (int j = 0; j < kSortRun; ++j) {
      if (i0 + 32 * j >= end) break;
      const uint32_t i = i0 + 32 * j + l;
      const bool has = e[j] < (uint32_t)E;
      const uint32_t same = lanes_alike(e[j], has), ahead = same & below;
      const uint32_t seen = has ? mine[e[j]] : 0u;
      __syncwarp();
      if (has && ahead == 0u) mine[e[j]] = seen + __popc(same);
      __syncwarp();
      rank[j] = has ? (int32_t)(seen + __popc(ahead)) : -1;
      if (!whole && i < end) rows[i] = rank[j];
    }
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
          if (r < cta) before += v;
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
      if (cta == 0) offsets[e] = (int32_t)(incl - all);
      if (e == E - 1) {
        kept = incl;
        if (cta == 0) offsets[E] = (int32_t)incl;
      }
    }
  }
  __syncthreads();

  for (int e = l; e < E; e += 32) mine[e] += first[e];
  __syncwarp();
  for (uint32_t i0 = begin; i0 < end; i0 += 32 * kSortRun) {
    if (!whole) {
      load(i0);
#pragma unroll
      for (int j = 0; j < kSortRun; ++j) {
        const uint32_t i = i0 + 32 * j + l;
        rank[j] = i < end ? rows[i] : -1;  // this lane's own of the first pass
      }
    }
#pragma unroll
    for (int j = 0; j < kSortRun; ++j) {
      const uint32_t i = i0 + 32 * j + l;
      if (i >= end) break;
      const int32_t row = e[j] < (uint32_t)E ? (int32_t)mine[e[j]] + rank[j] : -1;
      rows[i] = row;
      if (SCATTER && pairs != nullptr && row >= 0) pairs[row] = (int32_t)i;
    }
  }
  if (SCATTER && pairs != nullptr)
    for (uint32_t i = kept + cta * blockDim.x + threadIdx.x; i < P; i += ctas * blockDim.x)
      pairs[i] = -1;
  if (ctas > 1) cluster_sync();  // no CTA leaves while another may read its totals
}

// pairs[rows[i]] = i, and -1 behind the last row.
__global__ void __launch_bounds__(256) experts_pairs_kernel(const int32_t *rows,
                                                            const int32_t *kept, uint32_t P,
                                                            int32_t *pairs) {
  launch_dependents();
  grid_dependency_wait();
  const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= P) return;
  const int32_t row = rows[i];
  if (row >= 0) pairs[row] = (int32_t)i;
  if (i >= (uint32_t)*kept) pairs[i] = -1;
}

// Up to 4096 pairs (128 a warp) one CTA, without the cluster's barriers, and the
// scatter in place.
template <typename ID>
static cudaError_t run_sort(const ID *ids, int64_t P, int E, int32_t *offsets, int32_t *rows,
                            int32_t *pairs, cudaStream_t st) {
  if (P <= 4096)
    return launch_serial(experts_sort_kernel<ID, true>, 1, 32 * kSortWarps, st, ids, (uint32_t)P, E,
                         offsets, rows, pairs);
  const int ctas = widest_cluster<experts_sort_kernel<ID, false>>(kSortCluster, 32 * kSortWarps);
  const cudaError_t e =
      launch_serial_cluster(experts_sort_kernel<ID, false>, ctas, 32 * kSortWarps, ctas, 0, st, ids,
                            (uint32_t)P, E, offsets, rows, pairs);
  if (e != cudaSuccess || pairs == nullptr) return e;
  return launch_serial(experts_pairs_kernel, (P + 255) / 256, 256, st,
                       static_cast<const int32_t *>(rows), static_cast<const int32_t *>(offsets + E),
                       (uint32_t)P, pairs);
}

cudaError_t launch_experts_sort(const void *ids, bool wide, int64_t P, int E, int32_t *offsets,
                                int32_t *rows, int32_t *pairs, cudaStream_t st) {
  return wide ? run_sort(static_cast<const int64_t *>(ids), P, E, offsets, rows, pairs, st)
              : run_sort(static_cast<const int32_t *>(ids), P, E, offsets, rows, pairs, st);
}

// A warp's walk over the tasks (token, window of columns) warp, warp + warps, ...
// with the windows of a token next to each other.
struct TaskWalk {
  int64_t t, step_t;
  int32_t win, wins, step_win;
  __device__ __forceinline__ TaskWalk(int64_t K, int window) {
    wins = (int32_t)((K + window - 1) / window);
    const uint32_t warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const uint32_t warps = (gridDim.x * blockDim.x) >> 5;
    t = warp / (uint32_t)wins;
    win = (int32_t)(warp % (uint32_t)wins);
    step_t = warps / (uint32_t)wins;
    step_win = (int32_t)(warps % (uint32_t)wins);
  }
  __device__ __forceinline__ void next() {
    t += step_t;
    win += step_win;
    if (win >= wins) {
      win -= wins;
      ++t;
    }
  }
};

// ----------------------------------------------------------------- gather --
// A warp per (token, W windows of 512 columns): lane l holds 16 consecutive
// elements of each, so eight lanes form a 1x128 group and each lane stores 16 bytes
// of codes per row.  The token's rows sit in the lanes, one each; a group's scale
// for eight rows goes out in one store instruction, one row per lane of the group.
//
// Bound by HBM: 4096 tokens of 7168 bf16 columns to eight rows each in 46.5 us, 95%
// of the copy rate (scattering the scales, four bytes per row and group, costs 2 to
// 6 us of it).  Codes leave L2 first (plain stores: 52 us).  A resident grid was
// slower (49 to 58 us, with the next task loaded ahead of this one's stores too),
// and so were three CTAs an SM (47.2); fp32 rows of two windows take four (spills).
template <typename T, int F, int W>
__global__ void __launch_bounds__(256, sizeof(T) * W == 8 ? 4 : 5)
    experts_gather_kernel(const GatherArgs a) {
  constexpr bool kCodes = sizeof(T) == 1;
  launch_dependents();
  grid_dependency_wait();
  const uint32_t l = lane_id(), S = (uint32_t)a.S, K = (uint32_t)a.K, M = (uint32_t)a.M;
  for (TaskWalk w(a.K, 512 * W); w.t < a.T; w.next()) {
    const uint32_t t = (uint32_t)w.t, k0 = (uint32_t)w.win * (512 * W) + l * 16;
    const int32_t *list = a.rows + (uint64_t)t * S;
    uint32_t mine = l < S ? (uint32_t)list[l] : 0xffffffffu;  // (a negative row: none)
    const T *x = static_cast<const T *>(a.x) + (uint64_t)t * (uint32_t)a.ldx + k0;
    Vec16<T> v[W];
    uint4 c[W];
    uint32_t scale[W];  // bits of the fp32 scale, or the UE8M0 byte
#pragma unroll
    for (int u = 0; u < W; ++u) {
      const uint32_t k = k0 + 512 * u, g = k >> 7;
      v[u].zero();
      scale[u] = 0u;
      if (k < K) v[u].load(x + 512 * u);
      if (kCodes && 128 * g < K) {  // (in a ragged last group also on the lanes past the row's end)
        const uint64_t at = (uint64_t)g * (uint32_t)a.T + t;
        scale[u] = a.sfmt == 0 ? static_cast<const uint32_t *>(a.x_scales)[at]
                               : static_cast<const uint8_t *>(a.x_scales)[at];
      }
    }
#pragma unroll
    for (int u = 0; u < W; ++u) {
      if constexpr (kCodes) {
        c[u] = v[u].w[0];
      } else if (a.q != nullptr) {
        const float amax = __uint_as_float(group8_max(v[u].max_key()));
        GroupScale gs = group_scale<F>(amax, a.sfmt);
        const ScaleDiv d(gs.s);
        if (__all_sync(0xffffffffu, gs.fast && (a.sfmt != 0 || d.fast))) {
          c[u] = a.sfmt == 0 ? v[u].template codes_own<F>(d) : v[u].template codes_pow2<F>(gs.inv);
        } else {
          gs = group_scale_any<F>(amax, a.sfmt);
          F2 y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = v[u].pair(i);
          c[u] = codes16_any<F>(y, gs.s);
        }
        scale[u] = gs.stored;
      }
    }
    for (uint32_t s0 = 0; s0 < S; s0 += 32) {
      const uint32_t n = min(32u, S - s0);
      if (s0 > 0) mine = l < n ? (uint32_t)list[s0 + l] : 0xffffffffu;
      for (uint32_t s = 0; s < n; s += 8) {
        const uint32_t lane_row = __shfl_sync(0xffffffffu, mine, s + (l & 7u));
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
          if (s + j >= n) break;
          const uint32_t row = __shfl_sync(0xffffffffu, mine, s + j);
          if (row >= M) continue;
#pragma unroll
          for (int u = 0; u < W; ++u) {
            const uint32_t k = k0 + 512 * u;
            if (k >= K) continue;
            if (a.q != nullptr)
              __stcs(reinterpret_cast<uint4 *>(a.q + (uint64_t)row * K + k), c[u]);
            if constexpr (!kCodes)
              if (a.out != nullptr)
                v[u].store(static_cast<T *>(a.out) + (uint64_t)row * (uint32_t)a.ld_out + k);
          }
        }
#pragma unroll
        for (int u = 0; u < W; ++u) {
          const uint32_t k = k0 + 512 * u, g = k >> 7;
          if (a.q != nullptr && lane_row < M && 128 * g < K)
            store_scale(a.scales, (uint64_t)g * M + lane_row, scale[u], a.sfmt);
        }
      }
    }
  }
}

static int64_t grid_of(int64_t warps, int per_block, int64_t most) {
  const int64_t blocks = (warps + per_block - 1) / per_block;
  return blocks < 1 ? 1 : blocks < most ? blocks : most;
}

template <typename T, int F, int W>
static cudaError_t run_gather(const GatherArgs &a, int sms, cudaStream_t st) {
  const int64_t tasks = a.T * ((a.K + 512 * W - 1) / (512 * W));
  return launch_serial(experts_gather_kernel<T, F, W>, grid_of(tasks, 8, (int64_t)sms * 64), 256, st,
                       a);
}
// Two windows at once for short lists of many tasks, whose fixed instructions bound
// them: from 100 tasks of one window an SM on (codes that are moved: 60), where codes
// are formed only if few windows are idle behind an odd last one.  us with one and
// with two, bf16: 7168 columns, 16384 tokens of one row 77 and 65, of two 87 and 77,
// of four 112 and 107, 2000 of four 14.1 and 13.7, but 500 of them 5.4 and 6.3; 2048
// columns, 4096 of one 7.0 and 6.7, but 2000 of four 5.6 and 6.7; 3584 columns, 8192
// of two 24.3 and 22.6; but 1040 columns (three windows) 16384 of one 17.2 and 18.6.
// fp32 gains less: 7168 columns, 8192 of two 56 and 55, 2000 of four 18.6 and 19.1.
// Moved, 2048 columns: 3000 of one row 3.8 and 3.0, of two 4.2 and 3.8; 2000 of four
// 4.6 and 5.4.
template <typename T>
static bool two_windows(const GatherArgs &a, int sms) {
  const int64_t wins = (a.K + 511) / 512, tasks = a.T * wins;
  if (a.S > 4 || wins < 2) return false;
  if (sizeof(T) == 1) return tasks >= (int64_t)sms * 60;
  return tasks >= (int64_t)sms * 100 && (wins % 2 == 0 || wins > 6);
}
template <typename T, int F>
static cudaError_t run_gather(const GatherArgs &a, int sms, cudaStream_t st) {
  return two_windows<T>(a, sms) ? run_gather<T, F, 2>(a, sms, st) : run_gather<T, F, 1>(a, sms, st);
}
template <typename T>
static cudaError_t run_gather(const GatherArgs &a, int sms, cudaStream_t st) {
  return a.fmt == 0 ? run_gather<T, 0>(a, sms, st) : run_gather<T, 1>(a, sms, st);
}

cudaError_t launch_experts_gather(const GatherArgs &a, int source, int sms, cudaStream_t st) {
  if (a.T == 0 || a.M == 0) return cudaSuccess;
  if (source == kGatherCodes)  // the format of codes that are moved does not matter
    return run_gather<uint8_t, 0>(a, sms, st);
  return source == kGatherBf16 ? run_gather<__nv_bfloat16>(a, sms, st) : run_gather<float>(a, sms, st);
}

// --------------------------------------------------------- rows in flight --
// Combine and its gradient read eight scattered rows (fp32: four) per step of
// 256 columns, eight elements per lane.  A warp keeps a two-deep ring of steps in
// shared memory: the rows of the next step are copied asynchronously while this
// one is added up, and the choices of the step behind it are loaded meanwhile,
// so that the warp always has 4 KB in flight and no registers hold them.  (Loads
// into registers, a batch at a time, measured 116 and 151 us on 4096 tokens of
// 7168 columns with eight rows each.)  Shorter lists of choices take W windows of
// 256 columns a step, so that as many rows' pieces are in flight: a quarter of them
// left two choices at 348 us where the copy rate allows 140 (the gradient, 16384
// tokens).  A dropped pair's row is a copy of no bytes, which leaves zeros.
template <typename T, int W>
constexpr int rows_per_step() {
  return (sizeof(T) == 2 ? 8 : 4) / W;
}
// Bytes of a stage: the rows' pieces, then those of a row of type V.
template <typename T, typename V, int W>
constexpr int ring_stage() {
  return 256 * W * (rows_per_step<T, W>() * (int)sizeof(T) + (int)sizeof(V));
}
// Warps of a CTA, of which three share an SM (74 KB of its shared memory each).
constexpr int ring_warps(int stage) {
  const int n = 74 * 1024 / (2 * stage);
  return n < 8 ? n : 8;
}
// The most windows a step (1, 2 or 4; fp32 rows 1 or 2) that still hold the whole
// list, and of which more than half exist.  us with one, two and four, 7168 columns,
// bf16: combine 16384 tokens of one row 179, 116, 114, of two 187, 139, 142, 1000 of
// one 13.2, 8.3, 6.3; gradient 16384 of one 370, 213, 134, of two 380, 226, 153, 4096
// of two 97, 60, 52; 1040 columns, 4096 of two 21, 15.2, 13.1.  What it costs: the
// gradient of 64 decoded tokens (narrow ones 3.4, 3.8, 4.1; 7168 columns 8.2, 5.8, 6.6)
// and fp32 sums of full size (16384 tokens of one row 219 and 232, two rows 277 and 280).
template <typename T, typename Fn>
static cudaError_t with_windows(int64_t S, int64_t K, Fn &&f) {
  const int64_t all = rows_per_step<T, 1>();
  int w = sizeof(T) == 2 ? 4 : 2;
  while (w > 1 && (S > all / w || K <= 128 * w)) w /= 2;
  if constexpr (sizeof(T) == 2)
    if (w == 4) return f(std::integral_constant<int, 4>{});
  return w == 2 ? f(std::integral_constant<int, 2>{}) : f(std::integral_constant<int, 1>{});
}

// 256 elements of a row, of which the first `left` exist: the row's 16-byte vectors
// in their order (lane l copies vector l, and l + 32 of fp32 rows), lane l's eight
// elements read back.  (The two lanes that share a 32-byte sector copy to one place:
// apart, as a layout without bank conflicts for fp32 has them, the copies took L2
// twice the requests: 313 us instead of 170 for the sums of 4096 x 8 rows of 7168.)
template <typename T>
struct RowCopy {
  // in bytes from a row's first element: this lane's first vector at column k0
  static __device__ __forceinline__ int64_t offset(int64_t k0) {
    return k0 * (int64_t)sizeof(T) + 16 * lane_id();
  }
  // dst and src: this lane's first vector's
  static __device__ __forceinline__ void copy(uint32_t dst, const char *src, int32_t left, bool real) {
    const int32_t l = (int32_t)lane_id(), per = 16 / (int32_t)sizeof(T);
    copy16_async(dst, src, real && per * l < left ? 16u : 0u);
    if constexpr (sizeof(T) == 4)
      copy16_async(dst + 512, src + 512, real && per * (l + 32) < left ? 16u : 0u);
  }
};
template <typename T>
__device__ __forceinline__ Raw8<T> ring_row(const uint8_t *slot) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < Raw8<T>::kWords; ++i)
    r.w[i] = reinterpret_cast<const uint4 *>(slot)[Raw8<T>::kWords * lane_id() + i];
  return r;
}

// The rows and weights of choices s0 .. s0 + C - 1 of a token, choice j's on the
// lanes with l % C == j (without a row: -1 and weight zero).
template <int C>
struct Choices {
  int32_t row;
  float wt;
  __device__ __forceinline__ void load(const int32_t *rows, const float *weights, int64_t t,
                                       int32_t s0, int64_t T, int32_t S, int64_t M) {
    const int32_t s = s0 + (int32_t)(lane_id() & (uint32_t)(C - 1));
    int32_t r = -1;
    float v = 1.0f;
    if (t < T && s < S) {
      r = rows[t * S + s];
      if (weights != nullptr) v = weights[t * S + s];
    }
    const bool has = r >= 0 && r < M;
    row = has ? r : -1;
    wt = has ? v : 0.0f;
  }
  // bit j: choice j has a row
  __device__ __forceinline__ uint32_t kept() const {
    return __ballot_sync(0xffffffffu, row >= 0) & ((1u << C) - 1u);
  }
};

// ---------------------------------------------------------------- combine --
// A warp per (token, W windows).  Sums in fp32 in the order of the choices, the
// residual last, one rounding to the output's type.  4096 tokens of 7168 columns,
// eight bf16 rows each and a residual: 86.4 us, the copy rate.
template <typename T, typename O, int W>
__global__ void __launch_bounds__(32 * ring_warps(ring_stage<T, O, W>()), 3)
    experts_combine_kernel(const CombineArgs a) {
  constexpr int kC = rows_per_step<T, W>(), kRow = 256 * sizeof(T), kRes = 256 * sizeof(O),
                kStage = ring_stage<T, O, W>();
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t *ring = smem + (threadIdx.x >> 5) * (2 * kStage);
  const uint32_t ring_at = smem_u32(ring);
  launch_dependents();
  grid_dependency_wait();
  const O *res = static_cast<const O *>(a.residual);
  const int32_t S = (int32_t)a.S;
  const uint32_t pitch = (uint32_t)a.ldx * (uint32_t)sizeof(T);
  struct Step {
    TaskWalk w;
    int32_t s0;
    __device__ __forceinline__ void next(int32_t S) {
      s0 += kC;
      if (s0 >= S) {
        s0 = 0;
        w.next();
      }
    }
  };
  auto fetch = [&](const Step &s, const Choices<kC> &c, int stage) {
    if (s.w.t < a.T) {
      const int32_t n = min(kC, S - s.s0);
      const uint32_t kept = c.kept(), at = ring_at + stage * kStage + 16 * lane_id();
      const int64_t k0 = (int64_t)s.w.win * (256 * W);
      const int32_t left = (int32_t)min((int64_t)256 * W, a.K - k0);
      const char *x = static_cast<const char *>(a.x) + RowCopy<T>::offset(k0);
      uint32_t r[kC];
#pragma unroll
      for (int j = 0; j < kC; ++j) r[j] = (uint32_t)max(__shfl_sync(0xffffffffu, c.row, j), 0);
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        if (j >= n) continue;
        const char *row = x + (uint64_t)r[j] * pitch;
#pragma unroll
        for (int u = 0; u < W; ++u)
          RowCopy<T>::copy(at + (u * kC + j) * kRow, row + u * kRow, left - 256 * u, kept >> j & 1u);
      }
      if (res != nullptr && S <= kC) {
        const char *v = reinterpret_cast<const char *>(res + s.w.t * a.ldr) + RowCopy<O>::offset(k0);
#pragma unroll
        for (int u = 0; u < W; ++u)
          RowCopy<O>::copy(at + W * kC * kRow + u * kRes, v + u * kRes, left - 256 * u, true);
      }
    }
    copies_commit();
  };
  auto choices = [&](const Step &s, Choices<kC> &c) {
    c.load(a.rows, a.weights, s.w.t, s.s0, a.T, S, a.M);
  };
  Step cur{TaskWalk(a.K, 256 * W), 0};
  Choices<kC> c_cur, c_next;
  choices(cur, c_cur);
  fetch(cur, c_cur, 0);
  Step nxt = cur;
  nxt.next(S);
  choices(nxt, c_next);
  F2 acc[W][4];
  for (int stage = 0; cur.w.t < a.T; stage ^= 1) {
    __syncwarp();  // the other lanes have read what this overwrites
    fetch(nxt, c_next, stage ^ 1);
    Step behind = nxt;
    behind.next(S);
    const float w_l = c_cur.wt;
    c_cur = c_next;
    choices(behind, c_next);
    copies_wait<1>();
    __syncwarp();
    const uint8_t *slot = ring + stage * kStage;
    const int32_t n = min(kC, S - cur.s0);
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const F2 wt(__shfl_sync(0xffffffffu, w_l, j));
      if (j >= n) continue;
#pragma unroll
      for (int u = 0; u < W; ++u) {
        const Raw8<T> v = ring_row<T>(slot + (u * kC + j) * kRow);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[u][i] = fma2(wt, raw_pair(v, i), acc[u][i]);
      }
    }
    if (cur.s0 + kC >= S) {
#pragma unroll
      for (int u = 0; u < W; ++u) {
        const int64_t k = (int64_t)cur.w.win * (256 * W) + 256 * u + lane_id() * 8;
        if (k < a.K) {
          if (res != nullptr) {
            Raw8<O> r;
            if (S <= kC)
              r = ring_row<O>(slot + W * kC * kRow + u * kRes);
            else  // (a longer list has other stages behind the first)
              r.load_stream(res + cur.w.t * a.ldr + k);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[u][i] = acc[u][i] + raw_pair(r, i);
          }
          store8(static_cast<O *>(a.out) + cur.w.t * a.ld_out + k, round8<O>(acc[u]));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[u][i] = F2(0.0f);
      }
    }
    cur = nxt;
    nxt = behind;
  }
  copies_wait<0>();
}

template <typename T, typename O>
static cudaError_t run_combine(const CombineArgs &a, int sms, cudaStream_t st) {
  return with_windows<T>(a.S, a.K, [&](auto windows) {
    constexpr int kW = windows.value, kStage = ring_stage<T, O, kW>(), kWarps = ring_warps(kStage);
    constexpr int kSmem = kWarps * 2 * kStage;
    const int64_t tasks = a.T * ((a.K + 256 * kW - 1) / (256 * kW));
    return launch_serial_smem<experts_combine_kernel<T, O, kW>, kSmem>(
        grid_of(tasks, kWarps, (int64_t)sms * 3), 32 * kWarps, kSmem, st, a);
  });
}

cudaError_t launch_experts_combine(const CombineArgs &a, int x_dt, int out_dt, int sms,
                                   cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  if (a.M == 0) {  // no row is read; the copies of no bytes have an address all the same
    CombineArgs b = a;
    b.x = a.out;
    b.ldx = 0;
    b.M = -1;
    return launch_experts_combine(b, x_dt, out_dt, sms, st);
  }
  if (x_dt == 0)
    return out_dt == 0 ? run_combine<__nv_bfloat16, __nv_bfloat16>(a, sms, st)
                       : run_combine<__nv_bfloat16, float>(a, sms, st);
  return out_dt == 0 ? run_combine<float, __nv_bfloat16>(a, sms, st)
                     : run_combine<float, float>(a, sms, st);
}

// ------------------------------------------------------- combine, gradient --
// A CTA per token, each warp every nw-th W windows of it (alone: a warp per token).
// |w dy| of a group (16 lanes) peaks where |dy| does (rounding is monotone), so the
// group's maximum of dy is taken once and lane j of the group forms the scale of
// the j-th row from it, and the factor w / scale that takes dy to that row's codes.
// The rows' dot products stay in registers and are reduced together: a butterfly
// that halves the rows a lane still holds at each of its first steps, then a sum
// over the warps in their order.  4096 tokens of 7168 columns, eight bf16 rows each,
// codes and dw: 120 us, 95% of the copy rate; with one row each (16384 tokens, 133
// us, 65%) the scales and reductions of a step serve only that row.
template <typename DY, typename X, int F, int W>
__global__ void __launch_bounds__(32 * ring_warps(ring_stage<X, DY, W>()), 3)
    experts_combine_grad_kernel(const CombineGradArgs a) {
  constexpr int kC = rows_per_step<X, W>(), kRow = 256 * sizeof(X), kDy = 256 * sizeof(DY),
                kStage = ring_stage<X, DY, W>(), kWarps = ring_warps(kStage);
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float part[2][kWarps][kC];
  launch_dependents();
  grid_dependency_wait();
  const uint32_t l = lane_id(), warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const bool alone = a.alone != 0;
  const uint32_t w = alone ? 0u : warp, nw = alone ? 1u : warps;
  const int64_t first = alone ? (int64_t)blockIdx.x * warps + warp : blockIdx.x;
  const int64_t step_t = alone ? (int64_t)gridDim.x * warps : gridDim.x;
  uint8_t *ring = smem + warp * (2 * kStage);
  const uint32_t ring_at = smem_u32(ring);
  const DY *dy = static_cast<const DY *>(a.dy);
  const int32_t wins = (int32_t)((a.K + 256 * W - 1) / (256 * W)), S = (int32_t)a.S;
  const uint32_t pitch = (uint32_t)a.ldx * (uint32_t)sizeof(X), K = (uint32_t)a.K;
  struct Step {
    int64_t t;
    int32_t s0, win;
    // true: another list of choices
    __device__ __forceinline__ bool next(int32_t wins, int32_t w, int32_t nw, int32_t S,
                                         int64_t step_t) {
      win += nw;
      if (win < wins) return false;
      win = w;
      s0 += kC;
      if (s0 >= S) {
        s0 = 0;
        t += step_t;
      }
      return true;
    }
  };
  auto fetch = [&](const Step &s, const Choices<kC> &c, int stage) {
    if (s.t < a.T) {
      const int32_t n = min(kC, S - s.s0);
      const uint32_t kept = c.kept(), at = ring_at + stage * kStage + 16 * lane_id();
      const int64_t k0 = (int64_t)s.win * (256 * W);
      const int32_t left = (int32_t)min((int64_t)256 * W, a.K - k0);
      const char *d = reinterpret_cast<const char *>(dy + s.t * a.ld_dy) + RowCopy<DY>::offset(k0);
#pragma unroll
      for (int u = 0; u < W; ++u)
        RowCopy<DY>::copy(at + W * kC * kRow + u * kDy, d + u * kDy, left - 256 * u, true);
      if (a.dw != nullptr && a.M > 0) {
        const char *x = static_cast<const char *>(a.x) + RowCopy<X>::offset(k0);
#pragma unroll
        for (int j = 0; j < kC; ++j) {
          const char *row = x + (uint64_t)max(__shfl_sync(0xffffffffu, c.row, j), 0) * pitch;
          if (j >= n) continue;
#pragma unroll
          for (int u = 0; u < W; ++u)
            RowCopy<X>::copy(at + (u * kC + j) * kRow, row + u * kRow, left - 256 * u, kept >> j & 1u);
        }
      }
    }
    copies_commit();
  };
  auto choices = [&](const Step &s, Choices<kC> &c) {
    c.load(a.rows, a.weights, s.t, s.s0, a.T, S, a.M);
  };
  Step cur{first, 0, (int32_t)w};
  Choices<kC> c_cur, c_next;
  choices(cur, c_cur);
  fetch(cur, c_cur, 0);
  Step nxt = cur;
  c_next = c_cur;
  if (nxt.next(wins, (int32_t)w, (int32_t)nw, S, step_t)) choices(nxt, c_next);
  F2 dot[kC];
  int phase = 0;
  for (int stage = 0; cur.t < a.T; stage ^= 1) {
    __syncwarp();  // the other lanes have read what this overwrites
    fetch(nxt, c_next, stage ^ 1);
    Step behind = nxt;
    const bool fresh = behind.next(wins, (int32_t)w, (int32_t)nw, S, step_t);
    const int32_t row_l = c_cur.row;
    const float w_l = c_cur.wt;
    const uint32_t kept = c_cur.kept();
    c_cur = c_next;
    if (fresh) choices(behind, c_next);
    copies_wait<1>();
    __syncwarp();
    const int32_t n = min(kC, S - cur.s0);
#pragma unroll
    for (int u = 0; u < W; ++u) {
      const uint8_t *slot = ring + stage * kStage + u * kC * kRow;
      const uint32_t k = (uint32_t)cur.win * (256 * W) + 256 * u + l * 8, g = k >> 7;
      const bool in = k < K;
      const Raw8<DY> raw = ring_row<DY>(ring + stage * kStage + W * kC * kRow + u * kDy);
      F2 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = raw_pair(raw, i);
      if (a.q != nullptr) {
        uint32_t ka = 0, kb = 0;
        raw.max_abs(ka, kb);
        uint32_t key = Raw8<DY>::merge_keys(ka, kb);
        key = max(key, __shfl_xor_sync(0xffffffffu, key, 8));
        const float amax = fabsf(w_l) * __uint_as_float(group8_max(key));
        GroupScale gs = group_scale<F>(amax, a.sfmt);
        const float f_l = w_l * gs.inv;
        const bool fast =
            __all_sync(0xffffffffu, gs.fast && (w_l == 0.0f || (fabsf(f_l) >= 0x1p-100f &&
                                                                fabsf(f_l) <= 0x1p100f)));
        if (!fast) gs = group_scale_any<F>(amax, a.sfmt);
        if (row_l >= 0 && (l & 15u) < (uint32_t)kC && 128 * g < K)
          store_scale(a.scales, (int64_t)g * a.M + row_l, gs.stored, a.sfmt);
        uint8_t *q = a.q + k;
#pragma unroll
        for (int j = 0; j < kC; ++j) {
          const uint32_t row = (uint32_t)__shfl_sync(0xffffffffu, row_l, j);
          const int from = (int)(l & 16u) | j;
          uint2 c;
          if (fast) {
            const F2 f(__shfl_sync(0xffffffffu, f_l, from));
            c = make_uint2(pack4<F>(v[0] * f, v[1] * f), pack4<F>(v[2] * f, v[3] * f));
          } else {
            const F2 wj(__shfl_sync(0xffffffffu, w_l, j));
            const float s = __shfl_sync(0xffffffffu, gs.s, from);
            c = make_uint2(codes4_ieee<F>((v[0] * wj).v, (v[1] * wj).v, s),
                           codes4_ieee<F>((v[2] * wj).v, (v[3] * wj).v, s));
          }
          if ((kept >> j & 1u) && in) *reinterpret_cast<uint2 *>(q + (uint64_t)row * K) = c;
        }
      }
      if (a.dx != nullptr) {
#pragma unroll
        for (int j = 0; j < kC; ++j) {
          const int64_t row = __shfl_sync(0xffffffffu, row_l, j);
          const F2 wj(__shfl_sync(0xffffffffu, w_l, j));
          if (row < 0 || !in) continue;
          const F2 y[4] = {v[0] * wj, v[1] * wj, v[2] * wj, v[3] * wj};
          if (a.dx_dt == 0)
            store8(static_cast<__nv_bfloat16 *>(a.dx) + row * a.ld_dx + k, round8<__nv_bfloat16>(y));
          else
            store8(static_cast<float *>(a.dx) + row * a.ld_dx + k, round8<float>(y));
        }
      }
      if (a.dw != nullptr && a.M > 0) {
#pragma unroll
        for (int j = 0; j < kC; ++j) {
          if (j >= n) continue;
          const Raw8<X> xv = ring_row<X>(slot + j * kRow);
#pragma unroll
          for (int i = 0; i < 4; ++i) dot[j] = fma2(v[i], raw_pair(xv, i), dot[j]);
        }
      }
    }
    if (a.dw != nullptr && cur.win + (int32_t)nw >= wins) {  // this warp's last columns of these rows
      float d[kC];
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        float d0, d1;
        dot[j].get(d0, d1);
        d[j] = d0 + d1;
        dot[j] = F2(0.0f);
      }
      // halves apart, quarters apart, ...: lane l ends with row l / (32 / kC)
#pragma unroll
      for (int h = kC / 2; h > 0; h >>= 1) {
        const uint32_t apart = (uint32_t)(32 / kC * h);
#pragma unroll
        for (int j = 0; j < h; ++j) {
          const float keep = l & apart ? d[j + h] : d[j], give = l & apart ? d[j] : d[j + h];
          d[j] = keep + __shfl_xor_sync(0xffffffffu, give, (int)apart);
        }
      }
      float sum = d[0];
#pragma unroll
      for (int o = 16 / kC; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      // (a dropped pair's sum would be dy's infinities times zeros)
      const uint32_t j = l / (32 / kC);
      if (alone) {
        if (l % (32 / kC) == 0 && (int32_t)j < n)
          a.dw[cur.t * S + cur.s0 + j] = kept >> j & 1u ? sum : 0.0f;
      } else {
        // (a buffer is written again two barriers after it was read)
        if (l % (32 / kC) == 0) part[phase][w][j] = sum;
        __syncthreads();
        if ((int)threadIdx.x < n) {
          float all = 0.0f;
          for (uint32_t i = 0; i < nw; ++i) all += part[phase][i][threadIdx.x];
          a.dw[cur.t * S + cur.s0 + threadIdx.x] = kept >> threadIdx.x & 1u ? all : 0.0f;
        }
      }
      phase ^= 1;
    }
    cur = nxt;
    nxt = behind;
  }
  copies_wait<0>();
}

// A CTA per token: the fewest rounds of its steps, then as few warps as they need.
// Of many tokens (two and more for each resident warp) with one or two choices a
// warp takes one alone, without the barrier.  7168 columns, us with a CTA and with a
// warp per token: 16384 tokens of one choice 167 and 133, of two 184 and 152, 8192 of
// two 98 and 79, 4096 of two 52 and 53; but of four 8192 in 134 and 161, and 16384 of
// eight choices, 4096 columns, in 265 and 328.  Between full rounds of 2736 tokens the
// last one is idle in part: 5472 of two choices 66 and 55, 6000 72 and 70, 8500 98 and
// 91, 12000 138 and 120; 2048 columns 18.4 and 17.2, 22.2 and 22.9, 32.8 and 32.4, 43
// and 42; 14336 columns 118 and 109, 131 and 133, 181 and 173, 251 and 236.  fp32, two
// choices: 2048 columns 81 and 79, 7168 columns 257 and 266 (16384 tokens; one choice
// 69 and 50, 185 and 171).
template <typename DY, typename X, int F>
static cudaError_t run_combine_grad(const CombineGradArgs &a, int sms, cudaStream_t st) {
  return with_windows<X>(a.S, a.K, [&](auto windows) {
    constexpr int kW = windows.value, kStage = ring_stage<X, DY, kW>(), kMost = ring_warps(kStage);
    const int64_t steps = (a.K + 256 * kW - 1) / (256 * kW), rounds = (steps + kMost - 1) / kMost;
    CombineGradArgs b = a;
    b.alone = rows_per_step<X, kW>() == 2 && a.T >= (int64_t)sms * 6 * kMost ? 1 : 0;
    const int warps = b.alone ? kMost : (int)((steps + rounds - 1) / rounds);
    const int64_t most = (int64_t)sms * (3 * kMost / warps);  // resident at once
    return launch_serial_smem<experts_combine_grad_kernel<DY, X, F, kW>, kMost * 2 * kStage>(
        a.T < most ? a.T : most, 32 * warps, warps * 2 * kStage, st, b);
  });
}
template <typename DY, typename X>
static cudaError_t run_combine_grad(const CombineGradArgs &a, int sms, cudaStream_t st) {
  return a.fmt == 0 ? run_combine_grad<DY, X, 0>(a, sms, st) : run_combine_grad<DY, X, 1>(a, sms, st);
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
