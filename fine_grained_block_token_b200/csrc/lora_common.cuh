// Shared by the low-rank adapter kernels: arguments, the map from tile
// numbers to rows, and the split of an fp32 value into two bf16 terms.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp8bl_internal.h"
#include "ptx_bf16.cuh"

namespace fp8bl {
namespace lora {

struct Args {
  const __nv_bfloat16* x;
  const __nv_bfloat16* a;
  const __nv_bfloat16* b;
  const float* scales;
  const int32_t* offsets;
  const int32_t* order;
  const __nv_bfloat16* y;
  __nv_bfloat16* out;
  // u of the sorted rows, rank padded to RP.  Small batches: fp32 [parts of K]
  // [M][RP]; long ones: bf16 [M][hi RP | lo RP], scaled.
  __nv_bfloat16* u;
  int M, N, K, R, L;
  int max_splits;       // parts of K at most (long batches: exactly)
  int shrink_blocks;    // blocks of the shrink kernel
  int copy_rest;        // rows without an adapter are copied from y to out
  int* err;
};

// Launch sizes; rt = rank / 16, rounded up to 1, 2, 4 or 8.
struct Plan {
  int rt;
  int shrink_blocks, expand_blocks;
  int max_splits;
  int few_clusters = 0;  // both products in one launch of so many clusters
  size_t u_bytes;
};
inline int rank_tiles(int64_t R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

// The form for long batches (lora_tiles.cu).
Plan plan_tiles(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L, int sm_count);
cudaError_t launch_tiles(const Args& a, const Plan& pl, cudaStream_t st);

// Parts of K for `tiles` tiles: as many as the shrink kernel's blocks can
// work on at once.  Both kernels derive the number from the offsets.
__device__ __forceinline__ int parts_of_k(int blocks, int tiles, int max_splits) {
  const int s = tiles > 0 ? blocks / tiles : 1;
  return s < 1 ? 1 : s > max_splits ? max_splits : s;
}

// Tiles are up to `bm` consecutive sorted rows of one adapter, numbered
// adapter by adapter; the rows without an adapter follow as group L.
struct Tile {
  int group;
  int pos;    // first sorted row
  int rows;
};

struct TileMap {
  int start[kMaxExperts + 2];   // first sorted row of each group
  int before[kMaxExperts + 2];  // tiles before each group
  int warp_sum[32];

  // By all kThreads threads of the block.  Offsets are clamped to [0, M], so
  // malformed ones cannot lead outside the tensors.
  template <int kThreads>
  __device__ void build(const int32_t* offsets, int M, int L, int bm) {
    const int t = threadIdx.x, lane = t % 32, w = t / 32;
    for (int g = t; g <= L + 1; g += kThreads) {
      const int v = g <= L ? offsets[g] : M;
      start[g] = v < 0 ? 0 : v > M ? M : v;
    }
    __syncthreads();
    const int own = (L + 1 + kThreads - 1) / kThreads;
    int mine = 0;
    for (int i = 0; i < own; ++i) {
      const int g = t * own + i;
      if (g <= L) {
        const int n = start[g + 1] - start[g];
        mine += n > 0 ? (n + bm - 1) / bm : 0;
      }
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[w] = incl;
    __syncthreads();
    int at = incl - mine;
    for (int i = 0; i < w; ++i) at += warp_sum[i];
    for (int i = 0; i < own; ++i) {
      const int g = t * own + i;
      if (g <= L) {
        before[g] = at;
        const int n = start[g + 1] - start[g];
        at += n > 0 ? (n + bm - 1) / bm : 0;
        if (g == L) before[L + 1] = at;
      }
    }
    __syncthreads();
  }

  // The last group that starts at or before tile t (it has rows, or the next
  // would start there too).  groups = L, or L + 1 with the rows of no adapter.
  __device__ __forceinline__ Tile find(int t, int groups, int bm) const {
    int lo = 0, hi = groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int r = (t - before[lo]) * bm, n = start[lo + 1] - start[lo] - r;
    return Tile{lo, start[lo] + r, n < bm ? n : bm};
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// a and b as the nearest finite bf16 pair and the bf16 pair nearest to the rest:
// fp32's last values above bf16's largest keep a finite rest, an infinity goes
// into it whole.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
  lo = pack_bf16(a - lo_f(hi), b - hi_f(hi));
}

// y + c of two neighbouring columns, rounded once
__device__ __forceinline__ uint32_t add2(uint32_t y, float c0, float c1) {
  return pack_bf16(lo_f(y) + c0, hi_f(y) + c1);
}

}  // namespace lora
}  // namespace fp8bl
