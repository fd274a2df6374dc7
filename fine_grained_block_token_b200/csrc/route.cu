// Router of an expert layer: top-k choice from the logits, the chosen
// experts' weights, the counts per expert, the balance loss and the gradient
// of weights and loss with respect to the logits.
//
// Mathematics, per row z of E logits (fp32 arithmetic throughout):
//   softmax: p_e = exp(z_e - max z) / sum;  score = share = p
//   sigmoid: s_e = 1 / (1 + exp(-z_e));     score = s, share = s / sum s
//   chosen: the k largest logits above -inf (both scores grow with the logit,
//   so comparing logits needs no rounding), ties to the lowest index
//   w_j = scale * score_j, or scale * score_j / sum of the chosen scores
//   loss = balance * E / (k n^2) * sum_e c_e sum_t share_te over the n rows
//   that chose anything; slope_e = balance * E * c_e / (k n^2) = dloss/dshare.
// Where every logit of a row is far below zero, sigmoid shares and renormalised
// weights are formed from scores multiplied by exp(-max z): their ratios stay
// finite where the scores themselves underflow.
//
// A row belongs to kLanes lanes of a warp and a lane holds kVals neighbouring
// logits, so one pass over the logits serves the choice, the scores and the
// per-expert sums; each lane keeps the sums of its experts in registers over
// all rows of its warp.  Sums leave the block once, in a fixed order, so
// results do not depend on scheduling.
//
// What bounds it is the instructions of the choice, not the bytes: with 256
// experts a row costs about 580 warp instructions, 340 of them apart from the k
// rounds.  16384 x 256 fp32 logits with 8 of 256: 15 us forward (17 MB, 61% of
// the issue slots), 4 us for the sums of the blocks, 11 us for the gradient (half
// the issue slots; what stalls it first are the loads of the chosen's logits and
// slopes).  One row: 5.8 us, a block of 1024 threads and its sums for one warp's
// work.
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp8bl_internal.h"
#include "ptx_sm100.cuh"

namespace fp8bl {
namespace {

// Threads of a block: as many as the registers of an SM allow, since a row is
// a long chain of short steps and only other rows can fill the gaps.
template <int kVals>
constexpr int kForward = kVals <= 8 ? 1024 : kVals == 16 ? 512 : 256;
constexpr int kThreads = 256;  // of the gradient
constexpr unsigned kFull = 0xffffffffu;

template <int kLanes>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// The lanes of this thread's row, as bits of the warp.
template <int kLanes>
__device__ __forceinline__ unsigned lanes_of_row() {
  if constexpr (kLanes == 32) return kFull;
  return ((1u << (kLanes % 32)) - 1u) << (threadIdx.x % 32 / kLanes * kLanes);
}

// Largest of the lanes of a row (no NaN among them); a whole warp has an
// instruction for it.
template <int kLanes>
__device__ __forceinline__ float max_lanes(float v) {
  if constexpr (kLanes == 32) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
  } else {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
  }
}

// A logit as the choice sees it: NaN, which is never chosen, as -inf.
__device__ __forceinline__ float choice(float z) { return fmaxf(z, -INFINITY); }

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_float(float& d, float v) { d = v; }
// the one rounding of a bf16 gradient
__device__ __forceinline__ void from_float(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }

// A lane's kVals neighbouring elements; `vec` (every lane's run lies wholly
// inside or outside the row, and starts aligned) uses the widest accesses.
template <typename T, int kVals>
__device__ __forceinline__ void load_vals(const T* p, int valid, bool vec, float (&z)[kVals]) {
  constexpr int kBytes = kVals * static_cast<int>(sizeof(T));
  if (vec) {
    if (valid <= 0) {
#pragma unroll
      for (int i = 0; i < kVals; ++i) z[i] = -INFINITY;
      return;
    }
    alignas(16) T buf[kVals];
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4*>(buf)[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(buf) = __ldg(reinterpret_cast<const uint2*>(p));
    } else if constexpr (kBytes == 4) {
      *reinterpret_cast<uint32_t*>(buf) = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
      buf[0] = p[0];
    }
#pragma unroll
    for (int i = 0; i < kVals; ++i) z[i] = to_float(buf[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kVals; ++i) z[i] = i < valid ? to_float(p[i]) : -INFINITY;
  }
}

template <typename T, int kVals>
__device__ __forceinline__ void store_vals(T* p, int valid, bool vec, const float (&d)[kVals]) {
  constexpr int kBytes = kVals * static_cast<int>(sizeof(T));
  if (vec) {
    if (valid <= 0) return;
    alignas(16) T buf[kVals];
#pragma unroll
    for (int i = 0; i < kVals; ++i) from_float(buf[i], d[i]);
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(buf)[i];
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(buf);
    } else if constexpr (kBytes == 4) {
      *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(buf);
    } else {
      p[0] = buf[0];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      if (i < valid) from_float(p[i], d[i]);
  }
}

// exp(x) and 1 / x in one instruction each (ex2 to 2^-22, rcp to 2^-23 of the
// result; results below 2^-126 are flushed to zero).  With u = 2^-24, x log2(e)
// is off by 1.22 u of itself (the constant's rounding and the product's), so
// exp(x) by 1.22 u |x| + 4 u of itself.
//
// For every number of experts: how far a gradient's terms cancel depends on a
// row's scores, not on how many there are.  Against expf and __frcp_rn, errors
// of the gradient in norm over 4096 rows, fp32, 2 chosen, softmax | sigmoid:
//   8 experts   9.2e-8 and 9.2e-8 | 9.5e-8 and 9.9e-8
//   16, 17      8.6e-8 and 8.6e-8 | 9.8e-8 and 9.6e-8
//   64          8.4e-8 and 8.4e-8 | 1.2e-7 and 9.8e-8
//   256         8.1e-8 and 8.0e-8 | 1.3e-7 and 9.6e-8
// (the same formulas in fp32 tensor operations: 0.7 to 0.9e-7 | 1.9e-7 to 2.5e-6),
// and expf takes 19.2 | 20.1 us instead of 18.4 | 18.6 for 16384 x 256.
__device__ __forceinline__ float fast_exp(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));  // log2(e)
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Scores of a row from its logits and its largest, `top`: e[i] is the score
// times a factor common to the row (softmax: its denominator; sigmoid: 1, or
// exp(-top) where every logit is below kFar), so e / sum is the share.  Below
// kFar 1 + exp(z) is 1 in fp32 and a score is exp(z): exp(z - top) keeps the
// ratios of a row down to e^-87 where the scores themselves underflow.  e is off
// by (2.22 |z - top| + 4) u of itself where the exponent is z - top (its own
// rounding comes in), and by (1.22 |z| + 7) u for a sigmoid score (the sum with 1
// and its reciprocal come in).
constexpr float kFar = -18.0f;

template <int kLanes, int kVals, bool kSigmoid>
struct RowScores {
  float shift, sum;
  bool far;

  __device__ __forceinline__ float value(float z) const {
    if (kSigmoid && !far) return fast_rcp(1.0f + fast_exp(-z));
    return fast_exp(z - shift);
  }

  __device__ __forceinline__ RowScores(float top, const float (&z)[kVals], float (&e)[kVals]) {
    shift = top;
    far = kSigmoid && top < kFar;
    float s = 0.0f;
    if (kSigmoid && !far) {
#pragma unroll
      for (int i = 0; i < kVals; ++i) e[i] = fast_rcp(1.0f + fast_exp(-z[i]));
    } else {
#pragma unroll
      for (int i = 0; i < kVals; ++i) e[i] = fast_exp(z[i] - shift);
    }
#pragma unroll
    for (int i = 0; i < kVals; ++i) s += e[i];
    sum = sum_lanes<kLanes>(s);
  }
};

constexpr int kCluster = 8;

// Shared memory of block `rank` of the cluster, at the place of `here`.
__device__ __forceinline__ int ld_cluster_int(const int* here, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];"
               : "=r"(v)
               : "r"(ptx::map_to_cta(ptx::smem_u32(here), rank))
               : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_double(const double* here, uint32_t rank, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(
                   ptx::map_to_cta(ptx::smem_u32(here), rank)),
               "d"(v)
               : "memory");
}

struct RouteArgs {
  const void* logits;
  const uint8_t* mask;
  int32_t* ids;
  float* weights;
  int32_t* counts;
  float* loss;
  float* loss_grad;
  float* part_share;   // [blocks][E]
  int32_t* part_count; // [blocks][E]
  int32_t* part_rows;  // [blocks]
  int T, E, k;
  int blocks;          // of the forward kernel: up to kCluster are one cluster
  int renorm, vec;
  float scale, balance;
};

__device__ __forceinline__ double loss_slope(float balance, int E, int k, int rows) {
  const double n = rows > 0 ? rows : 1;
  return static_cast<double>(balance) * E / (static_cast<double>(k) * n * n);
}

// A lane's largest and second largest key with their indices (the lower index
// of two equal keys first).  A lane seldom wins more than one of the k rounds,
// so the second is at hand when it does, and a scan for more is rare: key2 is
// NaN while it is not known.
template <int kVals>
struct Best {
  float key, key2;
  int at, at2;

  __device__ __forceinline__ void take(float v, int i) {
    const bool first = v > key, second = v > key2;
    key2 = fmaxf(key2, fminf(v, key));
    at2 = first ? at : second ? i : at2;
    key = fmaxf(v, key);
    at = first ? i : at;
  }

  // Of the keys that come after (m, from) in the order of choice; at0 is the
  // index of k[0].
  __device__ __forceinline__ void scan(const float (&k)[kVals], int at0, float m, int from) {
    key = key2 = -INFINITY;
    at = at2 = 0;
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      take(k[i] < m || (k[i] == m && at0 + i > from) ? k[i] : -INFINITY, at0 + i);
  }

  __device__ __forceinline__ Best(const float (&k)[kVals], int at0) {
    key = key2 = -INFINITY;
    at = at2 = 0;
#pragma unroll
    for (int i = 0; i < kVals; ++i) take(k[i], at0 + i);
  }
};

template <typename T, int kLanes, int kVals, bool kSigmoid>
__global__ void __launch_bounds__(kForward<kVals>, 1) route_kernel(const RouteArgs a) {
  constexpr int kBlock = kForward<kVals>, kWarps = kBlock / 32;
  constexpr int kRows = kBlock / kLanes;  // rows in flight per block
  constexpr int kSlots = kMaxTopK / kLanes;  // of the chosen, per lane
  extern __shared__ __align__(16) unsigned char smem_raw[];
  int* counts = reinterpret_cast<int*>(smem_raw);     // [E]
  float* sums = reinterpret_cast<float*>(counts + a.E);  // [kWarps][E]
  __shared__ int rows_used;
  __shared__ double red[kWarps];
  __shared__ double terms[kCluster];  // of the loss, block 0's copy

  for (int e = threadIdx.x; e < a.E; e += kBlock) counts[e] = 0;
  if (threadIdx.x == 0) rows_used = 0;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  __syncthreads();

  const int g = threadIdx.x / kLanes, l = threadIdx.x % kLanes;
  const int lane = threadIdx.x % 32;
  const unsigned group = lanes_of_row<kLanes>();
  const int first = l * kVals, valid = a.E - first;
  float acc[kVals];
#pragma unroll
  for (int i = 0; i < kVals; ++i) acc[i] = 0.0f;
  int my_rows = 0;

  // every lane of a warp takes the same number of turns: the shuffles below
  // name the whole warp
  const int turns = (a.T + gridDim.x * kRows - 1) / (gridDim.x * kRows);
  for (int turn = 0; turn < turns; ++turn) {
    const int row = (turn * gridDim.x + blockIdx.x) * kRows + g;
    const bool live = row < a.T && (!a.mask || a.mask[row]);
    if (!__any_sync(kFull, live)) {  // no row of this warp chooses
      if (row < a.T)
        for (int j = l; j < a.k; j += kLanes) {
          a.ids[static_cast<int64_t>(row) * a.k + j] = -1;
          a.weights[static_cast<int64_t>(row) * a.k + j] = 0.0f;
        }
      continue;
    }
    float z[kVals];
    if (live) {
      load_vals<T, kVals>(static_cast<const T*>(a.logits) + static_cast<int64_t>(row) * a.E + first,
                          valid, a.vec, z);
    } else {
#pragma unroll
      for (int i = 0; i < kVals; ++i) z[i] = -INFINITY;
    }
    float key[kVals];
#pragma unroll
    for (int i = 0; i < kVals; ++i) key[i] = choice(z[i]);

    // k rounds of: the largest key left, in the lowest lane that holds it
    // (lanes hold rising indices, so that is the lowest index).  Lane l keeps
    // the slots l, l + kLanes, ...
    Best<kVals> best(key, first);
    int id[kSlots];
    float zc[kSlots];
    float top = -INFINITY;
#pragma unroll
    for (int t = 0; t < kSlots; ++t) {
      id[t] = -1;
      zc[t] = -INFINITY;
      const int n = min(a.k - t * kLanes, kLanes);
#pragma unroll 2
      for (int j = 0; j < n; ++j) {
        const float m = max_lanes<kLanes>(best.key);
        if (t == 0 && j == 0) top = m;
        unsigned holders = __ballot_sync(kFull, best.key == m);
        if (kLanes < 32) holders &= group;
        const int holder = __ffs(holders) - 1;
        const int won = __shfl_sync(kFull, best.at, holder);
        if (l == j) id[t] = won, zc[t] = m;
        if (lane == holder) {
          best.key = best.key2, best.at = best.at2;
          best.key2 = __int_as_float(0x7fffffff);
        }
        if (best.key != best.key) best.scan(key, first, m, won);
      }
      if (!(zc[t] > -INFINITY)) id[t] = -1;  // nothing was left
    }

    float e[kVals];
    const RowScores<kLanes, kVals, kSigmoid> sc(top, z, e);
    const bool used = top > -INFINITY;
    if (used) {
      const float inv = fast_rcp(sc.sum);
#pragma unroll
      for (int i = 0; i < kVals; ++i) acc[i] += e[i] * inv;
      my_rows += l == 0;
    }
    // weights of the chosen
    float v[kSlots], part = 0.0f;
#pragma unroll
    for (int t = 0; t < kSlots; ++t) {
      v[t] = id[t] >= 0 ? sc.value(zc[t]) : 0.0f;
      part += v[t];
    }
    if (a.renorm) {
      part = sum_lanes<kLanes>(part);
      if (sc.sum != sc.sum) part = sc.sum;  // a NaN logit beside the chosen
    } else {
      part = kSigmoid ? 1.0f : sc.sum;
    }
    if (row < a.T) {
#pragma unroll
      for (int t = 0; t < kSlots; ++t) {
        const int j = l + t * kLanes;
        if (j >= a.k) break;
        float w = 0.0f;
        if (id[t] >= 0) {
          // divided exactly: the weight of a single chosen expert is `scale`
          w = a.scale * __fdiv_rn(v[t], part);
          // a score on its own, not times the row's factor
          if (kSigmoid && sc.far && !a.renorm) w = a.scale * fast_exp(zc[t]);
          atomicAdd(&counts[id[t]], 1);
        }
        const int64_t o = static_cast<int64_t>(row) * a.k + j;
        a.ids[o] = id[t];
        a.weights[o] = w;
      }
    }
  }

  // block sums: the row groups of a warp, then the warps in order
  const bool want_share = a.loss != nullptr;
  if (want_share) {
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(kFull, acc[i], o);
      if (lane < kLanes && i < valid) sums[threadIdx.x / 32 * a.E + first + i] = acc[i];
    }
  }
  if (my_rows) atomicAdd(&rows_used, my_rows);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kBlock) {
    float s = 0.0f;
    if (want_share)
      for (int w = 0; w < kWarps; ++w) s += sums[w * a.E + e];
    if (a.blocks <= kCluster) {
      sums[e] = s;  // this thread alone reads and writes column e
    } else {
      a.part_share[static_cast<int64_t>(blockIdx.x) * a.E + e] = s;
      a.part_count[static_cast<int64_t>(blockIdx.x) * a.E + e] = counts[e];
    }
  }
  if (a.blocks > kCluster) {
    if (threadIdx.x == 0) a.part_rows[blockIdx.x] = rows_used;
    return;
  }
  // One block, or one cluster whose blocks add up a share of the experts each
  // over all blocks, in order.
  __syncwarp();
  ptx::cluster_sync();
  const uint32_t rank = ptx::cluster_ctarank();
  int rows = 0;
  for (int b = 0; b < a.blocks; ++b) rows += ld_cluster_int(&rows_used, b);
  const double slope = loss_slope(a.balance, a.E, a.k, rows);
  double term = 0.0;
  const int per = (a.E + a.blocks - 1) / a.blocks;
  for (int i = threadIdx.x; i < per; i += kBlock) {
    const int e = static_cast<int>(rank) * per + i;
    if (e >= a.E) break;
    int c = 0;
    double s = 0.0;
    for (int b = 0; b < a.blocks; ++b) {
      c += ld_cluster_int(&counts[e], b);
      s += __int_as_float(ld_cluster_int(reinterpret_cast<const int*>(&sums[e]), b));
    }
    a.counts[e] = c;
    if (a.loss_grad) a.loss_grad[e] = static_cast<float>(slope * c);
    term += slope * c * s;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(kFull, term, o);
  if (lane == 0) red[threadIdx.x / 32] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int w = 0; w < kWarps; ++w) t += red[w];
    st_cluster_double(&terms[rank], 0, t);
  }
  __syncwarp();
  ptx::cluster_sync();  // also: the others have read this block's sums
  if (rank == 0 && threadIdx.x == 0 && want_share) {
    double t = 0.0;
    for (int b = 0; b < a.blocks; ++b) t += terms[b];
    *a.loss = static_cast<float>(t);
  }
}

// Adds up the blocks' sums.  One cluster of kFinalCtas blocks: block c owns
// every kFinalCtas-th group of 32 experts, a warp strides over the partials
// of 32 experts (a lane each), and the loss terms meet in block 0.
constexpr int kFinalCtas = 8;
constexpr int kFinalThreads = 512;

__global__ void __launch_bounds__(kFinalThreads) route_final_kernel(const RouteArgs a, int blocks) {
  constexpr int kWarps = kFinalThreads / 32;
  __shared__ double terms[kFinalCtas];  // block 0's copy collects
  __shared__ int s_count[kWarps][32];
  __shared__ float s_share[kWarps][32];
  __shared__ int s_rows[kWarps];
  const int w = threadIdx.x / 32, l = threadIdx.x % 32;
  const uint32_t rank = ptx::cluster_ctarank();
  __syncwarp();
  ptx::cluster_sync();  // block 0's shared memory may be written only once it runs
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  int rows = 0;
  for (int b = threadIdx.x; b < blocks; b += kFinalThreads) rows += a.part_rows[b];
  double slope = 0.0, term = 0.0;
  bool first = true;  // the rows are added up with the first experts
  for (int e0 = static_cast<int>(rank) * 32; first || e0 < a.E; e0 += kFinalCtas * 32) {
    const int e = e0 + l;
    int c = 0;
    float s = 0.0f;
    if (e < a.E) {
#pragma unroll 10
      for (int b = w; b < blocks; b += kWarps) {
        c += a.part_count[static_cast<int64_t>(b) * a.E + e];
        s += a.part_share[static_cast<int64_t>(b) * a.E + e];
      }
    }
    if (first) {
      rows = __reduce_add_sync(kFull, rows);
      if (l == 0) s_rows[w] = rows;
    }
    s_count[w][l] = c;
    s_share[w][l] = s;
    __syncthreads();
    if (w == 0) {
      if (first) {
        rows = __reduce_add_sync(kFull, l < kWarps ? s_rows[l] : 0);
        slope = loss_slope(a.balance, a.E, a.k, rows);
      }
      if (e < a.E) {
        int ct = 0;
        double st = 0.0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) ct += s_count[i][l], st += s_share[i][l];
        a.counts[e] = ct;
        if (a.loss_grad) a.loss_grad[e] = static_cast<float>(slope * ct);
        term += slope * ct * st;
      }
    }
    first = false;
    __syncthreads();
  }
  if (!a.loss) return;  // the same for every block of the cluster
  if (w == 0) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(kFull, term, o);
    if (l == 0) st_cluster_double(&terms[rank], 0, term);
  }
  __syncwarp();
  ptx::cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    double t = 0.0;
    for (int i = 0; i < kFinalCtas; ++i) t += terms[i];
    *a.loss = static_cast<float>(t);
  }
}

struct RouteBackArgs {
  const void* logits;
  const int32_t* ids;
  const float* d_weights;
  const float* loss_grad;
  const float* d_loss;
  void* d_logits;
  int T, E, k;
  int renorm, vec;
  float scale;
};

// Gradient of one row per group of lanes: the scores again from the logits
// (cheaper to recompute than to keep T * E of them), then
//   softmax: dz = p (up - <p, up>)            up = slope * d_loss
//   sigmoid: dz = q (1 - s) (up - <q, up>)
// and, for the chosen, the weights' part.  The chosen few are written again
// over the row's stores by the lane that owns the slot.
template <typename T, int kLanes, int kVals, bool kSigmoid>
__global__ void __launch_bounds__(kThreads, kVals <= 8 ? 4 : 1) route_backward_kernel(const RouteBackArgs a) {
  constexpr int kRows = kThreads / kLanes;
  constexpr int kSlots = kMaxTopK / kLanes;  // of the chosen, per lane
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int g = threadIdx.x / kLanes, l = threadIdx.x % kLanes;
  const unsigned group = lanes_of_row<kLanes>();
  const int first = l * kVals, valid = a.E - first;
  const float d_loss = a.loss_grad ? (a.d_loss ? *a.d_loss : 1.0f) : 0.0f;
  float up[kVals];
#pragma unroll
  for (int i = 0; i < kVals; ++i)
    up[i] = a.loss_grad && i < valid ? a.loss_grad[first + i] * d_loss : 0.0f;

  const int turns = (a.T + gridDim.x * kRows - 1) / (gridDim.x * kRows);
  for (int turn = 0; turn < turns; ++turn) {
    const int row = (turn * gridDim.x + blockIdx.x) * kRows + g;
    const int64_t base = static_cast<int64_t>(row) * a.E;
    const T* zr = static_cast<const T*>(a.logits) + base;
    T* dr = static_cast<T*>(a.d_logits) + base;
    const int64_t slot0 = static_cast<int64_t>(row) * a.k;
    // the chosen of this lane's slots, and whether the row has any
    int id[kSlots];
    bool any = false;
#pragma unroll
    for (int t = 0; t < kSlots; ++t) {
      const int j = l + t * kLanes;
      id[t] = row < a.T && j < a.k ? a.ids[slot0 + j] : -1;
      if (id[t] < 0 || id[t] >= a.E) id[t] = -1;
      any = any || id[t] >= 0;
    }
    const bool used = (__ballot_sync(kFull, any) & group) != 0;
    float z[kVals];
    if (used) {
      load_vals<T, kVals>(zr + first, valid, a.vec, z);
    } else {
#pragma unroll
      for (int i = 0; i < kVals; ++i) z[i] = -INFINITY;
    }
    // the chosen's logits on their way early
    float zc[kSlots], down[kSlots];
#pragma unroll
    for (int t = 0; t < kSlots; ++t) {
      const bool in = a.d_weights && id[t] >= 0;
      down[t] = in ? a.d_weights[slot0 + l + t * kLanes] * a.scale : 0.0f;
      zc[t] = in ? to_float(zr[id[t]]) : -INFINITY;
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVals; ++i) top = fmaxf(top, z[i]);
    top = max_lanes<kLanes>(top);
    float e[kVals];
    const RowScores<kLanes, kVals, kSigmoid> sc(top, z, e);
    const float inv = fast_rcp(sc.sum);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      e[i] *= inv;  // the share
      dot += e[i] * up[i];
    }
    dot = sum_lanes<kLanes>(dot);

    // The chosen: v their scores or, renormalised, their parts of the sum of
    // the chosen scores (divided exactly, so that the part of a single one is 1
    // and its gradient 0), mix = sum of v * d_weight.
    float v[kSlots], part = 0.0f, mix = 0.0f;
    if (a.d_weights) {
#pragma unroll
      for (int t = 0; t < kSlots; ++t) {
        v[t] = id[t] >= 0 ? sc.value(zc[t]) : 0.0f;
        part += v[t];
      }
      if (a.renorm) part = sum_lanes<kLanes>(part);
      if (sc.sum != sc.sum) part = sc.sum;  // a NaN logit beside the chosen
#pragma unroll
      for (int t = 0; t < kSlots; ++t) {
        if (a.renorm && id[t] >= 0) v[t] = __fdiv_rn(v[t], part);
        mix += v[t] * down[t];
      }
      mix = sum_lanes<kLanes>(mix);
    }
    // without a gradient through the shares a NaN logit reaches the chosen alone
    const bool shares = a.loss_grad || (!kSigmoid && !a.renorm && a.d_weights);
    // softmax without renormalisation: every expert's score loses
    // p_e * sum_j p_j d_w_j; with it, the chosen share that among themselves
    const float all = dot + (!kSigmoid && !a.renorm ? mix * inv : 0.0f);
    if (row < a.T) {
      float d[kVals];
#pragma unroll
      for (int i = 0; i < kVals; ++i) {
        float x = e[i] * (up[i] - all);
        // 1 - s = 1 / (1 + exp(z))
        if constexpr (kSigmoid) x *= fast_rcp(1.0f + fast_exp(z[i]));
        d[i] = used && shares ? x : 0.0f;
      }
      store_vals<T, kVals>(dr + first, valid, a.vec, d);
    }
    __syncwarp();
    if (a.d_weights) {
#pragma unroll
      for (int t = 0; t < kSlots; ++t) {
        if (id[t] < 0) continue;
        const float u = a.loss_grad ? a.loss_grad[id[t]] * d_loss : 0.0f;
        const float score = sc.value(zc[t]);
        float dz = shares ? score * inv * (u - all) : 0.0f;
        if (a.renorm)
          dz += v[t] * (down[t] - mix);
        else if (kSigmoid)
          dz += down[t] * (sc.far ? fast_exp(zc[t]) : score);
        else
          dz += score * inv * down[t];
        if constexpr (kSigmoid) dz *= fast_rcp(1.0f + fast_exp(zc[t]));
        from_float(dr[id[t]], dz);
      }
    }
    __syncwarp();
  }
}

// Widths: kLanes * kVals >= E.  Up to 64 experts eight lanes serve a row, so
// that a warp handles four rows and its shuffles have three steps.
template <typename T, bool kSigmoid, typename F>
cudaError_t by_width(int64_t E, F f) {
  if (E <= 8) return f.template operator()<T, 8, 1, kSigmoid>();
  if (E <= 16) return f.template operator()<T, 8, 2, kSigmoid>();
  if (E <= 32) return f.template operator()<T, 8, 4, kSigmoid>();
  if (E <= 64) return f.template operator()<T, 8, 8, kSigmoid>();
  if (E <= 128) return f.template operator()<T, 16, 8, kSigmoid>();
  if (E <= 256) return f.template operator()<T, 32, 8, kSigmoid>();
  if (E <= 512) return f.template operator()<T, 32, 16, kSigmoid>();
  return f.template operator()<T, 32, 32, kSigmoid>();
}

template <typename F>
cudaError_t by_type(bool f32, bool sigmoid, int64_t E, F f) {
  if (f32) return sigmoid ? by_width<float, true>(E, f) : by_width<float, false>(E, f);
  return sigmoid ? by_width<__nv_bfloat16, true>(E, f) : by_width<__nv_bfloat16, false>(E, f);
}

// Blocks of the forward kernel, by the time on the GPU: one for the rows that
// it takes in one turn; one cluster for those that it takes in one turn, whose
// blocks add up their sums themselves; beyond, up to one per SM, and a second
// launch for the sums.  us, fp32 sigmoid, at 16 | 64 | 256 | 1024 experts:
//   one turn of a block     one block 4.4 | 8.1 | 6.8 | 11.9, a cluster 5.5 | 9.2 | 8.1 | 12.4
//   one and a half          5.5 | 11.3 | 8.8 | 13.7 and 5.7 | 9.5 | 8.0 | 12.4
//   one turn of a cluster   5.6 | 9.6 | 7.8 | 13.3
//   one and a quarter       a cluster 7.1 | 14.5 | 10.7 | 15.9, the grid 5.2 | 9.3 | 7.6 | 15.1
//   four turns              10.1 | 23.6 | 16.6 | 24.0 and 5.8 | 9.6 | 8.2 | 17.7
// The second launch costs the host 2.4 us: calls back to back that the host
// bounds take 12.2 instead of 9.8 where 16 experts' rows would fit a cluster's two to
// four turns.
int route_blocks(int64_t T, int64_t E, int sm_count) {
  const int64_t rows = E <= 64 ? 128 : E <= 128 ? 64 : E <= 256 ? 32 : E <= 512 ? 16 : 8;
  if (T <= rows) return 1;
  if (T <= kCluster * rows) return kCluster;
  const int64_t b = (T + rows - 1) / rows;
  return static_cast<int>(b > sm_count ? sm_count : b);
}

template <typename Kernel, typename... Args>
cudaError_t launch_pdl(Kernel k, int blocks, int cluster, int threads, size_t smem,
                       cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  set_programmatic_serialization(at[0]);
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

struct LaunchForward {
  RouteArgs a;
  int blocks;
  cudaStream_t st;
  template <typename T, int kLanes, int kVals, bool kSigmoid>
  cudaError_t operator()() {
    a.vec = a.E % kVals == 0;
    constexpr int kBlock = kForward<kVals>;
    constexpr size_t kMax = kLanes * kVals * 4 * (1 + kBlock / 32);
    static_assert(kMax + 1024 <= 48 * 1024, "shared memory without an opt-in");
    const size_t smem = static_cast<size_t>(a.E) * 4 * (1 + kBlock / 32);
    return launch_pdl(route_kernel<T, kLanes, kVals, kSigmoid>, blocks,
                      blocks <= kCluster ? blocks : 1, kBlock, smem, st, a);
  }
};

struct LaunchBackward {
  RouteBackArgs a;
  int sm_count;
  cudaStream_t st;
  template <typename T, int kLanes, int kVals, bool kSigmoid>
  cudaError_t operator()() {
    a.vec = a.E % kVals == 0;
    constexpr int kRows = kThreads / kLanes;
    const int64_t need = (static_cast<int64_t>(a.T) + kRows - 1) / kRows;
    const int blocks = static_cast<int>(need < sm_count * 8 ? need : sm_count * 8);
    return launch_pdl(route_backward_kernel<T, kLanes, kVals, kSigmoid>, blocks, 1, kThreads, 0,
                      st, a);
  }
};

}  // namespace

size_t route_workspace_bytes(int64_t T, int64_t E, int sm_count) {
  const int b = route_blocks(T, E, sm_count);
  return b <= kCluster ? 0 : static_cast<size_t>(b) * (static_cast<size_t>(E) * 8 + 4);
}

cudaError_t launch_route(const void* logits, bool f32, int64_t T, int64_t E, int64_t k,
                         bool sigmoid, bool renorm, float scale, float balance,
                         const uint8_t* mask, int32_t* ids, float* weights, int32_t* counts,
                         float* loss, float* loss_grad, void* workspace, int sm_count,
                         cudaStream_t st) {
  RouteArgs a = {};
  const int blocks = route_blocks(T, E, sm_count);
  a.logits = logits;
  a.mask = mask;
  a.ids = ids;
  a.weights = weights;
  a.counts = counts;
  a.loss = loss;
  a.loss_grad = loss_grad;
  a.part_share = static_cast<float*>(workspace);
  a.part_count = static_cast<int32_t*>(workspace) + static_cast<int64_t>(blocks) * E;
  a.part_rows = static_cast<int32_t*>(workspace) + 2 * static_cast<int64_t>(blocks) * E;
  a.T = static_cast<int>(T);
  a.E = static_cast<int>(E);
  a.k = static_cast<int>(k);
  a.blocks = blocks;
  a.renorm = renorm;
  a.scale = scale;
  a.balance = balance;
  cudaError_t e = by_type(f32, sigmoid, E, LaunchForward{a, blocks, st});
  if (e != cudaSuccess || blocks <= kCluster) return e;
  return launch_pdl(route_final_kernel, kFinalCtas, kFinalCtas, kFinalThreads, 0, st, a, blocks);
}

cudaError_t launch_route_backward(const void* logits, bool f32, const int32_t* ids,
                                  const float* d_weights, const float* loss_grad,
                                  const float* d_loss, int64_t T, int64_t E, int64_t k,
                                  bool sigmoid, bool renorm, float scale, void* d_logits,
                                  int sm_count, cudaStream_t st) {
  RouteBackArgs a = {};
  a.logits = logits;
  a.ids = ids;
  a.d_weights = d_weights;
  a.loss_grad = loss_grad;
  a.d_loss = d_loss;
  a.d_logits = d_logits;
  a.T = static_cast<int>(T);
  a.E = static_cast<int>(E);
  a.k = static_cast<int>(k);
  a.renorm = renorm;
  a.scale = scale;
  return by_type(f32, sigmoid, E, LaunchBackward{a, sm_count, st});
}

}  // namespace fp8bl
