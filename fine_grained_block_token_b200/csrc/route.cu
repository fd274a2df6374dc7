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
// Sigmoid shares and renormalised weights are formed from scores multiplied
// by exp(-m), m = min(max z, 0): their ratios stay finite where every score
// of a row underflows.
//
// A row belongs to kLanes lanes of a warp and a lane holds kVals neighbouring
// logits, so one pass over the logits serves the choice, the scores and the
// per-expert sums; each lane keeps the sums of its experts in registers over
// all rows of its warp.  Sums leave the block once, in a fixed order, so
// results do not depend on scheduling.
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp8bl_internal.h"
#include "ptx_sm100.cuh"

namespace fp8bl {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kFull = 0xffffffffu;

// Logit as a 32-bit key that orders like the float; 0 = never chosen (-inf,
// NaN).  z + 0 turns -0 into +0 so that the two compare equal.
__device__ __forceinline__ uint32_t choice_key(float z) {
  if (!(z > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(z + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

template <int kLanes>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

template <int kLanes>
__device__ __forceinline__ uint32_t max_lanes(uint32_t v) {
  if constexpr (kLanes == 32) {
    return __reduce_max_sync(kFull, v);
  } else {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
    return v;
  }
}

template <int kLanes>
__device__ __forceinline__ uint32_t min_lanes(uint32_t v) {
  if constexpr (kLanes == 32) {
    return __reduce_min_sync(kFull, v);
  } else {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(kFull, v, o));
    return v;
  }
}

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

// Scores of a row from its logits.  e[i] is the score times a factor common
// to the row (softmax: 1 / p's denominator; sigmoid: exp(-m)), inv_sum the
// reciprocal of their sum over the row, so e * inv_sum is the share.
template <int kLanes, int kVals, bool kSigmoid>
struct RowScores {
  float shift, sum;

  __device__ __forceinline__ float value(float z) const {
    if constexpr (kSigmoid) {
      // exp(-m) / (1 + exp(-z)) = exp(z - m) / (1 + exp(z)) where m < 0
      return shift < 0.0f ? expf(z - shift) / (1.0f + expf(z)) : 1.0f / (1.0f + expf(-z));
    } else {
      return expf(z - shift);
    }
  }

  __device__ __forceinline__ RowScores(uint32_t top, const float (&z)[kVals], float (&e)[kVals]) {
    const float m = key_logit(top);
    shift = kSigmoid ? fminf(m, 0.0f) : m;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      e[i] = value(z[i]);
      s += e[i];
    }
    sum = sum_lanes<kLanes>(s);
  }
};

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
  int renorm, vec;
  float scale, balance;
};


__device__ __forceinline__ double loss_slope(float balance, int E, int k, int rows) {
  const double n = rows > 0 ? rows : 1;
  return static_cast<double>(balance) * E / (static_cast<double>(k) * n * n);
}

template <typename T, int kLanes, int kVals, bool kSigmoid>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a) {
  constexpr int kRows = kThreads / kLanes;  // rows in flight per block
  extern __shared__ __align__(16) unsigned char smem_raw[];
  // [kRows][32] chosen ids and logits, then [E] counts, then sums [kRows][E]
  int* ch_id = reinterpret_cast<int*>(smem_raw);
  float* ch_z = reinterpret_cast<float*>(ch_id + kRows * 32);
  int* counts = reinterpret_cast<int*>(ch_z + kRows * 32);
  float* sums = reinterpret_cast<float*>(counts + a.E);
  __shared__ int rows_used;
  __shared__ double red[kThreads / 32];

  for (int e = threadIdx.x; e < a.E; e += kThreads) counts[e] = 0;
  if (threadIdx.x == 0) rows_used = 0;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  __syncthreads();

  const int g = threadIdx.x / kLanes, l = threadIdx.x % kLanes;
  const int first = l * kVals, valid = a.E - first;
  int* my_id = ch_id + g * 32;
  float* my_z = ch_z + g * 32;
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
    float z[kVals];
    if (live) {
      load_vals<T, kVals>(static_cast<const T*>(a.logits) + static_cast<int64_t>(row) * a.E + first,
                          valid, a.vec, z);
    } else {
#pragma unroll
      for (int i = 0; i < kVals; ++i) z[i] = -INFINITY;
    }
    uint32_t key[kVals];
#pragma unroll
    for (int i = 0; i < kVals; ++i) key[i] = choice_key(z[i]);

    // k rounds of: largest key left among the lanes, lowest index among
    // equals; the lane that held it looks up its next.
    uint32_t best = 0, at = 0;
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      if (key[i] > best) best = key[i], at = i;
    uint32_t top = 0;
    for (int j = 0; j < a.k; ++j) {
      const uint32_t m = max_lanes<kLanes>(best);
      const uint32_t id = min_lanes<kLanes>(best == m ? first + at : 0xffffffffu);
      if (j == 0) top = m;
      if (l == 0) {
        my_id[j] = m ? static_cast<int>(id) : -1;
        my_z[j] = key_logit(m);
      }
      if (m != 0 && id == first + at) {
        uint32_t nb = 0, na = 0;
#pragma unroll
        for (int i = 0; i < kVals; ++i) {
          const bool left = key[i] < m || (key[i] == m && i > static_cast<int>(at));
          if (left && key[i] > nb) nb = key[i], na = i;
        }
        best = nb, at = na;
      }
    }
    __syncwarp();

    float e[kVals];
    const RowScores<kLanes, kVals, kSigmoid> sc(top, z, e);
    const bool used = top != 0;
    if (used) {
      const float inv = 1.0f / sc.sum;
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if (i < valid) acc[i] += e[i] * inv;
      my_rows += l == 0;
    }
    // weights of the chosen
    float part = 0.0f;
    for (int j = l; j < a.k; j += kLanes)
      if (my_id[j] >= 0) part += sc.value(my_z[j]);
    part = sum_lanes<kLanes>(part);
    if (row < a.T) {
      for (int j = l; j < a.k; j += kLanes) {
        const int id = my_id[j];
        float w = 0.0f;
        if (id >= 0) {
          if (a.renorm) {
            w = sc.value(my_z[j]) / part;
            if (sc.sum != sc.sum) w = sc.sum;  // a NaN logit beside the chosen
          } else if (kSigmoid) {
            w = 1.0f / (1.0f + expf(-my_z[j]));
          } else {
            w = sc.value(my_z[j]) / sc.sum;
          }
          w *= a.scale;
          atomicAdd(&counts[id], 1);
        }
        const int64_t o = static_cast<int64_t>(row) * a.k + j;
        a.ids[o] = id;
        a.weights[o] = w;
      }
    }
    __syncwarp();
  }

  // block sums: each row group's registers, then over the groups in order
  if (a.loss || a.loss_grad) {
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      if (i < valid) sums[g * a.E + first + i] = acc[i];
  }
  if (my_rows) atomicAdd(&rows_used, my_rows);
  __syncthreads();
  const bool alone = gridDim.x == 1;
  const double slope = loss_slope(a.balance, a.E, a.k, rows_used);
  double term = 0.0;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    float s = 0.0f;
    if (a.loss || a.loss_grad)
      for (int r = 0; r < kRows; ++r) s += sums[r * a.E + e];
    if (alone) {
      a.counts[e] = counts[e];
      if (a.loss_grad) a.loss_grad[e] = static_cast<float>(slope * counts[e]);
      term += slope * counts[e] * static_cast<double>(s);
    } else {
      a.part_share[static_cast<int64_t>(blockIdx.x) * a.E + e] = s;
      a.part_count[static_cast<int64_t>(blockIdx.x) * a.E + e] = counts[e];
    }
  }
  if (!alone) {
    if (threadIdx.x == 0) a.part_rows[blockIdx.x] = rows_used;
    return;
  }
  if (!a.loss) return;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(kFull, term, o);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) t += red[w];
    *a.loss = static_cast<float>(t);
  }
}

// Adds up the blocks' sums.  One cluster of kFinalCtas blocks: block c owns
// every kFinalCtas-th group of 32 experts, a warp strides over the partials
// of 32 experts (a lane each), and the loss terms meet in block 0.
constexpr int kFinalCtas = 8;
constexpr int kFinalThreads = 512;

__global__ void __cluster_dims__(kFinalCtas, 1, 1) __launch_bounds__(kFinalThreads)
    route_final_kernel(const RouteArgs a, int blocks) {
  constexpr int kWarps = kFinalThreads / 32;
  __shared__ double terms[kFinalCtas];  // block 0's copy collects
  __shared__ int s_count[kWarps][32];
  __shared__ float s_share[kWarps][32];
  __shared__ int s_rows[kWarps];
  const int w = threadIdx.x / 32, l = threadIdx.x % 32;
  const uint32_t rank = ptx::cluster_ctarank();
  ptx::cluster_sync();  // block 0's shared memory may be written only once it runs
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  int rows = 0;
  for (int b = threadIdx.x; b < blocks; b += kFinalThreads) rows += a.part_rows[b];
  rows = __reduce_add_sync(kFull, rows);
  if (l == 0) s_rows[w] = rows;
  __syncthreads();
  rows = 0;
  for (int i = 0; i < kWarps; ++i) rows += s_rows[i];
  const double slope = loss_slope(a.balance, a.E, a.k, rows);
  double term = 0.0;
  for (int e0 = static_cast<int>(rank) * 32; e0 < a.E; e0 += kFinalCtas * 32) {
    const int e = e0 + l;
    int c = 0;
    float s = 0.0f;
    if (e < a.E) {
#pragma unroll 4
      for (int b = w; b < blocks; b += kWarps) {
        c += a.part_count[static_cast<int64_t>(b) * a.E + e];
        s += a.part_share[static_cast<int64_t>(b) * a.E + e];
      }
    }
    s_count[w][l] = c;
    s_share[w][l] = s;
    __syncthreads();
    if (w == 0 && e < a.E) {
      int ct = 0;
      double st = 0.0;
      for (int i = 0; i < kWarps; ++i) ct += s_count[i][l], st += s_share[i][l];
      a.counts[e] = ct;
      if (a.loss_grad) a.loss_grad[e] = static_cast<float>(slope * ct);
      term += slope * ct * st;
    }
    __syncthreads();
  }
  if (!a.loss) return;  // the same for every block of the cluster
  if (w == 0) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(kFull, term, o);
    if (l == 0) {
      const uint32_t dst = ptx::map_to_cta(ptx::smem_u32(&terms[rank]), 0);
      asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(dst), "d"(term) : "memory");
    }
  }
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
__global__ void __launch_bounds__(kThreads) route_backward_kernel(const RouteBackArgs a) {
  constexpr int kRows = kThreads / kLanes;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int g = threadIdx.x / kLanes, l = threadIdx.x % kLanes;
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
    const bool used = row < a.T && a.ids[slot0] >= 0;  // chose anything
    float z[kVals];
    if (used) {
      load_vals<T, kVals>(zr + first, valid, a.vec, z);
    } else {
#pragma unroll
      for (int i = 0; i < kVals; ++i) z[i] = -INFINITY;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kVals; ++i) top = max(top, choice_key(z[i]));
    top = max_lanes<kLanes>(top);
    float e[kVals];
    const RowScores<kLanes, kVals, kSigmoid> sc(top, z, e);
    const float inv = 1.0f / sc.sum;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      e[i] *= inv;  // the share
      if (i < valid) dot += e[i] * up[i];
    }
    dot = sum_lanes<kLanes>(dot);

    // sums over the chosen: part = their scores, mix = score * d_weight
    float part = 0.0f, mix = 0.0f;
    if (used && a.d_weights) {
      for (int j = l; j < a.k; j += kLanes) {
        const int id = a.ids[slot0 + j];
        if (id < 0 || id >= a.E) continue;
        const float v = sc.value(to_float(zr[id]));
        part += v;
        mix += v * a.d_weights[slot0 + j];
      }
    }
    part = sum_lanes<kLanes>(part);
    mix = sum_lanes<kLanes>(mix) * a.scale;
    // softmax without renormalisation: every expert's score loses
    // p_e * sum_j p_j d_w_j; with it, the chosen share `part` instead
    const bool plain_soft = !kSigmoid && !a.renorm;
    const float all = dot + (plain_soft ? mix * inv : 0.0f);
    const float mean = a.renorm ? mix / part : 0.0f;
    if (row < a.T) {
      float d[kVals];
#pragma unroll
      for (int i = 0; i < kVals; ++i) {
        float v = e[i] * (up[i] - all);
        if (kSigmoid) v *= 1.0f / (1.0f + expf(z[i]));  // 1 - s
        d[i] = used ? v : 0.0f;
      }
      store_vals<T, kVals>(dr + first, valid, a.vec, d);
    }
    __syncwarp();
    if (used && a.d_weights) {
      for (int j = l; j < a.k; j += kLanes) {
        const int id = a.ids[slot0 + j];
        if (id < 0 || id >= a.E) continue;
        const float zj = to_float(zr[id]);
        const float v = sc.value(zj), down = a.d_weights[slot0 + j] * a.scale;
        const float u = a.loss_grad ? a.loss_grad[id] * d_loss : 0.0f;
        float dz = v * inv * (u - all);
        if (a.renorm)
          dz += v / part * (down - mean);
        else if (kSigmoid)
          dz += down / (1.0f + expf(-zj));
        else
          dz += v * inv * down;
        if (kSigmoid) dz *= 1.0f / (1.0f + expf(zj));
        from_float(dr[id], dz);
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

// Blocks of the forward kernel: one while its rows take few turns, then as
// many as give every group of lanes at least two rows, up to one per SM.
int route_blocks(int64_t T, int64_t E, int sm_count) {
  const int lanes = E <= 64 ? 8 : E <= 128 ? 16 : 32;
  const int64_t rows = kThreads / lanes;
  const int64_t b = (T + 2 * rows - 1) / (2 * rows);
  return static_cast<int>(b < 1 ? 1 : b > sm_count ? sm_count : b);
}

template <typename Kernel, typename... Args>
cudaError_t launch_pdl(Kernel k, int blocks, int threads, size_t smem, cudaStream_t st,
                       Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  set_programmatic_serialization(at[0]);
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

struct LaunchForward {
  RouteArgs a;
  int blocks;
  cudaStream_t st;
  template <typename T, int kLanes, int kVals, bool kSigmoid>
  cudaError_t operator()() {
    a.vec = a.E % kVals == 0;
    constexpr int kRows = kThreads / kLanes;
    // 34 KB at most (E = 1024: 8 rows): below the 48 KB that need no opt-in
    const size_t smem = kRows * 32 * 8 + static_cast<size_t>(a.E) * 4 * (1 + kRows);
    return launch_pdl(route_kernel<T, kLanes, kVals, kSigmoid>, blocks, kThreads, smem, st, a);
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
    return launch_pdl(route_backward_kernel<T, kLanes, kVals, kSigmoid>, blocks, kThreads, 0, st,
                      a);
  }
};

}  // namespace

size_t route_workspace_bytes(int64_t T, int64_t E, int sm_count) {
  const int b = route_blocks(T, E, sm_count);
  return b == 1 ? 0 : static_cast<size_t>(b) * (static_cast<size_t>(E) * 8 + 4);
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
  a.renorm = renorm;
  a.scale = scale;
  a.balance = balance;
  cudaError_t e = by_type(f32, sigmoid, E, LaunchForward{a, blocks, st});
  if (e != cudaSuccess || blocks == 1) return e;
  return launch_pdl(route_final_kernel, kFinalCtas, kFinalThreads, 0, st, a, blocks);
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
