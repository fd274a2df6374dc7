// Rows of several groups (experts or adapters): sorting them by group, and
// the weighted sum that brings experts' rows back to their tokens, with its
// gradient.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp8bl_internal.h"
#include "ptx_sm100.cuh"

namespace fp8bl {
namespace {

constexpr unsigned kFull = 0xffffffffu;

template <typename Kernel, typename... Args>
cudaError_t launch_pdl(Kernel k, int64_t blocks, int threads, size_t smem, cudaStream_t st,
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

// ------------------------------------------------------------ group_rows
//
// A stable counting sort.  Entry i with id g < G goes to position
//   (entries of groups < g) + (entries of g in earlier blocks, warps, turns)
//   + (entries of g in earlier lanes);
// ids outside [0, G) count as group G, behind all others.  Blocks take
// contiguous pieces of the entries and warps contiguous parts of a piece, so
// the order within a group is the order of the entries.  Lanes with the same
// id find one another by ballots over the id's bits; the first of them adds
// their number to the warp's own counter, so nothing depends on the order of
// atomics.
//
// Bound by latency, not bytes: one launch up to 2048 entries (64 entries: 3 us
// on the GPU), two beyond (131072 entries into 256 groups: 10 us, of which the
// counts of 64 blocks per key and the scattered order are 5).  Beyond 131072 a
// block takes its pieces one after another, 1.7 us each: 524288 entries 20 us,
// 2097152 58.

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortTurns = 4;                              // entries per lane and piece
constexpr int kPiece = kSortThreads * kSortTurns;          // 2048
constexpr int kMaxSortBlocks = 64;
constexpr int kKeysPerThread = (kMaxExperts + 1 + kSortThreads - 1) / kSortThreads;  // 3

__device__ __forceinline__ int group_key(int id, int G) { return id >= 0 && id < G ? id : G; }

__global__ void __launch_bounds__(kSortThreads)
    group_count_kernel(const int32_t* ids, int n, int G, int per_block, int32_t* hist) {
  __shared__ int count[kMaxExperts + 1];
  for (int k = threadIdx.x; k <= G; k += kSortThreads) count[k] = 0;
  __syncthreads();
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * per_block;
  const int64_t end = begin + per_block < n ? begin + per_block : n;
  for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads)
    atomicAdd(&count[group_key(ids[i], G)], 1);
  __syncthreads();
  for (int k = threadIdx.x; k <= G; k += kSortThreads)
    hist[static_cast<int64_t>(blockIdx.x) * (G + 1) + k] = count[k];
}

// hist == nullptr: the one block holds all entries in one piece.  Otherwise the
// launch before this one is the count, whose blocks have all waited for the
// work before it: ids are final, so the first piece is counted while the
// count still runs.
__global__ void __launch_bounds__(kSortThreads)
    group_place_kernel(const int32_t* ids, int n, int G, int per_block, const int32_t* hist,
                       int32_t* offsets, int32_t* order, int32_t* slot) {
  __shared__ int base[kMaxExperts + 1];                         // next row of each key
  __shared__ int total[kMaxExperts + 1];                        // of the piece; first: of all
  __shared__ uint16_t warp_count[kSortWarps][kMaxExperts + 1];  // <= 128 entries per warp
  __shared__ int scan[kSortWarps];
  const int w = threadIdx.x / 32, l = threadIdx.x % 32;
  const int bits = 32 - __clz(G);  // of a key, 0 .. G
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * per_block;
  const int64_t end = begin + per_block < n ? begin + per_block : n;
  int key[kSortTurns], rank[kSortTurns];

  // Keys and ranks of a piece's entries: each warp counts its own, then every
  // key's counts become the counts of the warps before, and total the sum.
  auto count = [&](int64_t p) {
    const int64_t at = p + w * (32 * kSortTurns) + l;
#pragma unroll
    for (int t = 0; t < kSortTurns; ++t)
      key[t] = at + t * 32 < end ? group_key(ids[at + t * 32], G) : -1;
    for (int k = l; k <= G; k += 32) warp_count[w][k] = 0;
    __syncwarp();
#pragma unroll
    for (int t = 0; t < kSortTurns; ++t) {
      // the lanes that hold the same key, bit by bit (a warp match of 16
      // warps took ten times as long: 3.3 us for 8 turns)
      unsigned same = __ballot_sync(kFull, key[t] >= 0);
      if (key[t] < 0) same = ~same;
      for (int b = 0; b < bits; ++b) {
        const bool one = key[t] >> b & 1;
        const unsigned ones = __ballot_sync(kFull, one);
        same &= one ? ones : ~ones;
      }
      const unsigned earlier = same & ((1u << l) - 1);
      int seen = 0;
      if (key[t] >= 0) seen = warp_count[w][key[t]];
      __syncwarp();
      rank[t] = seen + __popc(earlier);
      if (key[t] >= 0 && earlier == 0)
        warp_count[w][key[t]] = static_cast<uint16_t>(seen + __popc(same));
      __syncwarp();
    }
    __syncthreads();
    for (int k = threadIdx.x; k <= G; k += kSortThreads) {
      int c[kSortWarps], sum = 0;
#pragma unroll
      for (int i = 0; i < kSortWarps; ++i) c[i] = warp_count[i][k];
#pragma unroll
      for (int i = 0; i < kSortWarps; ++i) {
        warp_count[i][k] = static_cast<uint16_t>(sum);
        sum += c[i];
      }
      total[k] = sum;
    }
  };

  if (!hist) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
  }
  count(begin);
  int before[kKeysPerThread] = {};  // entries of key threadIdx + q * threads in earlier blocks
  if (hist) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
#pragma unroll
    for (int q = 0; q < kKeysPerThread; ++q) {
      const int k = threadIdx.x + q * kSortThreads;
      if (k > G) break;
      int all = 0;
      const int32_t* h = hist + k;
#pragma unroll 32
      for (int b = 0; b < static_cast<int>(gridDim.x); ++b, h += G + 1) {
        const int c = *h;
        all += c;
        if (b < static_cast<int>(blockIdx.x)) before[q] += c;
      }
      base[k] = all;
    }
  } else {
    for (int k = threadIdx.x; k <= G; k += kSortThreads) base[k] = total[k];
  }
  __syncthreads();

  // exclusive sums over the keys: a thread owns `own` neighbours
  const int own = (G + kSortThreads) / kSortThreads;
  int mine = 0;
  for (int q = 0; q < own; ++q) {
    const int k = threadIdx.x * own + q;
    if (k <= G) mine += base[k];
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, o);
    if (l >= o) incl += v;
  }
  if (l == 31) scan[w] = incl;
  __syncthreads();
  int start = incl - mine;
#pragma unroll
  for (int i = 0; i < kSortWarps; ++i)
    if (i < w) start += scan[i];
  for (int q = 0; q < own; ++q) {
    const int k = threadIdx.x * own + q;
    if (k <= G) {
      const int c = base[k];
      base[k] = start;
      if (blockIdx.x == 0) offsets[k] = start;
      start += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kKeysPerThread; ++q) {
    const int k = threadIdx.x + q * kSortThreads;
    if (k <= G) base[k] += before[q];
  }
  __syncthreads();

  for (int64_t p = begin;;) {
    const int64_t at = p + w * (32 * kSortTurns) + l;
#pragma unroll
    for (int t = 0; t < kSortTurns; ++t) {
      if (key[t] >= 0) {
        const int pos = base[key[t]] + warp_count[w][key[t]] + rank[t];
        order[pos] = static_cast<int32_t>(at + t * 32);
        slot[at + t * 32] = key[t] < G ? pos : -1;
      }
    }
    p += kPiece;
    if (p >= end) break;  // the same for the whole block
    __syncthreads();
    for (int k = threadIdx.x; k <= G; k += kSortThreads) base[k] += total[k];
    __syncthreads();
    count(p);
    __syncthreads();
  }
}

// ---------------------------------------------------------- combine_rows
//
// out_t = base_t + sum_j w_tj y[slot_tj], added in the order of j in fp32 and
// rounded once.  Bound by the bytes of the rows: a thread owns 8 neighbouring
// columns of one token and has all k rows' 16-byte loads in flight (in batches
// of 8).  4093 tokens x 8 rows of 7168: 82 us, 6.5 TB/s, the copy rate; 32
// tokens: 3 us on the GPU.

constexpr int kCombineThreads = 128;

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// base may be out: the plain (coherent) path
__device__ __forceinline__ uint4 ld_base(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ void fma8(float (&acc)[8], const uint4& v, float w) {
  acc[0] = fmaf(lo_f(v.x), w, acc[0]);
  acc[1] = fmaf(hi_f(v.x), w, acc[1]);
  acc[2] = fmaf(lo_f(v.y), w, acc[2]);
  acc[3] = fmaf(hi_f(v.y), w, acc[3]);
  acc[4] = fmaf(lo_f(v.z), w, acc[4]);
  acc[5] = fmaf(hi_f(v.z), w, acc[5]);
  acc[6] = fmaf(lo_f(v.w), w, acc[6]);
  acc[7] = fmaf(hi_f(v.w), w, acc[7]);
}

__global__ void __launch_bounds__(kCombineThreads)
    combine_kernel(const uint4* y, const float* weights, const int32_t* slot, const uint4* base,
                   uint4* out, int n, int k, int vecs, int chunks) {
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int token = blockIdx.x / chunks;
  const int v = (blockIdx.x % chunks) * kCombineThreads + threadIdx.x;
  if (v >= vecs) return;
  const int64_t o = static_cast<int64_t>(token) * vecs + v;
  float acc[8] = {};
  if (base) fma8(acc, ld_base(base + o), 1.0f);
  const int64_t t0 = static_cast<int64_t>(token) * k;
  for (int j0 = 0; j0 < k; j0 += 8) {
    uint4 r[8];
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = 0.0f;
      r[j] = make_uint4(0, 0, 0, 0);
      if (j0 + j < k) {
        const int s = slot[t0 + j0 + j];
        if (s >= 0 && s < n) {
          w[j] = weights[t0 + j0 + j];
          r[j] = ld_stream(y + static_cast<int64_t>(s) * vecs + v);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) fma8(acc, r[j], w[j]);
  }
  out[o] = make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]),
                      pack_bf16(acc[4], acc[5]), pack_bf16(acc[6], acc[7]));
}

// Gradient: d_y[slot_tj] = w_tj d_out_t and d_w_tj = <d_out_t, y[slot_tj]>.
// A block owns a token: d_out_t is read once for its k rows, and the dot
// products end in one block sum.  Blocks past the tokens write zeros to the
// rows behind the last one that a slot names (*rows_used .. n).  2048 tokens x
// 8 rows of 7168: 83 us, 6.0 TB/s; reads and writes in equal parts bound it.
constexpr int kBackThreads = 128;
constexpr int kZeroBlocks = 148;

__device__ __forceinline__ uint4 scaled(const uint4& v, float w) {
  return make_uint4(pack_bf16(lo_f(v.x) * w, hi_f(v.x) * w), pack_bf16(lo_f(v.y) * w, hi_f(v.y) * w),
                    pack_bf16(lo_f(v.z) * w, hi_f(v.z) * w), pack_bf16(lo_f(v.w) * w, hi_f(v.w) * w));
}

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float acc) {
  acc = fmaf(lo_f(a.x), lo_f(b.x), acc);
  acc = fmaf(hi_f(a.x), hi_f(b.x), acc);
  acc = fmaf(lo_f(a.y), lo_f(b.y), acc);
  acc = fmaf(hi_f(a.y), hi_f(b.y), acc);
  acc = fmaf(lo_f(a.z), lo_f(b.z), acc);
  acc = fmaf(hi_f(a.z), hi_f(b.z), acc);
  acc = fmaf(lo_f(a.w), lo_f(b.w), acc);
  return fmaf(hi_f(a.w), hi_f(b.w), acc);
}

__global__ void __launch_bounds__(kBackThreads)
    combine_backward_kernel(const uint4* d_out, const uint4* y, const float* weights,
                            const int32_t* slot, const int32_t* rows_used, uint4* d_y,
                            float* d_weights, int T, int n, int k, int vecs) {
  __shared__ float part[kBackThreads / 32][8];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  if (static_cast<int>(blockIdx.x) >= T) {
    int64_t r = *rows_used;
    r = r < 0 ? 0 : r;
    const int64_t end = static_cast<int64_t>(n) * vecs;
    const int64_t step = static_cast<int64_t>(gridDim.x - T) * kBackThreads;
    for (int64_t i = r * vecs + (blockIdx.x - T) * kBackThreads + threadIdx.x; i < end; i += step)
      d_y[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int token = blockIdx.x;
  const int64_t t0 = static_cast<int64_t>(token) * k;
  const uint4* g = d_out + static_cast<int64_t>(token) * vecs;
  for (int j0 = 0; j0 < k; j0 += 8) {
    int s[8];
    float w[8], acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[j] = j0 + j < k ? slot[t0 + j0 + j] : -1;
      if (s[j] >= n) s[j] = -1;
      w[j] = s[j] >= 0 ? weights[t0 + j0 + j] : 0.0f;
      acc[j] = 0.0f;
    }
    for (int v = threadIdx.x; v < vecs; v += kBackThreads) {
      const uint4 gv = __ldg(g + v);
      uint4 r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (s[j] >= 0) r[j] = ld_stream(y + static_cast<int64_t>(s[j]) * vecs + v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (s[j] < 0) continue;
        acc[j] = dot8(gv, r[j], acc[j]);
        d_y[static_cast<int64_t>(s[j]) * vecs + v] = scaled(gv, w[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(kFull, acc[j], o);
    if (threadIdx.x % 32 == 0)
#pragma unroll
      for (int j = 0; j < 8; ++j) part[threadIdx.x / 32][j] = acc[j];
    __syncthreads();
    if (threadIdx.x < 8 && j0 + static_cast<int>(threadIdx.x) < k) {
      float d = 0.0f;
#pragma unroll
      for (int i = 0; i < kBackThreads / 32; ++i) d += part[i][threadIdx.x];
      d_weights[t0 + j0 + threadIdx.x] = d;
    }
    __syncthreads();
  }
}

int sort_blocks(int64_t n) {
  const int64_t b = (n + kPiece - 1) / kPiece;
  return static_cast<int>(b < 1 ? 1 : b > kMaxSortBlocks ? kMaxSortBlocks : b);
}

}  // namespace

size_t group_rows_workspace_bytes(int64_t n, int64_t G) {
  const int b = sort_blocks(n);
  return b == 1 ? 0 : static_cast<size_t>(b) * static_cast<size_t>(G + 1) * 4;
}

cudaError_t launch_group_rows(const int32_t* ids, int64_t n, int64_t G, int32_t* offsets,
                              int32_t* order, int32_t* slot, void* workspace, cudaStream_t st) {
  const int blocks = sort_blocks(n);
  // whole pieces per block, so that a piece belongs to one block
  const int64_t pieces = (n + kPiece - 1) / kPiece;
  const int per_block = static_cast<int>((pieces + blocks - 1) / blocks) * kPiece;
  int32_t* hist = static_cast<int32_t*>(workspace);
  if (blocks == 1)
    return launch_pdl(group_place_kernel, 1, kSortThreads, 0, st, ids, static_cast<int>(n),
                      static_cast<int>(G), kPiece, static_cast<const int32_t*>(nullptr), offsets,
                      order, slot);
  cudaError_t e = launch_pdl(group_count_kernel, blocks, kSortThreads, 0, st, ids,
                             static_cast<int>(n), static_cast<int>(G), per_block, hist);
  if (e != cudaSuccess) return e;
  return launch_pdl(group_place_kernel, blocks, kSortThreads, 0, st, ids, static_cast<int>(n),
                    static_cast<int>(G), per_block, static_cast<const int32_t*>(hist), offsets,
                    order, slot);
}

cudaError_t launch_combine_rows(const void* y, const float* weights, const int32_t* slot,
                                const void* base, void* out, int64_t T, int64_t n, int64_t k,
                                int64_t H, cudaStream_t st) {
  const int64_t vecs = H / 8, chunks = (vecs + kCombineThreads - 1) / kCombineThreads;
  if (T * chunks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return launch_pdl(combine_kernel, T * chunks, kCombineThreads, 0, st,
                    static_cast<const uint4*>(y), weights, slot, static_cast<const uint4*>(base),
                    static_cast<uint4*>(out), static_cast<int>(n), static_cast<int>(k),
                    static_cast<int>(vecs), static_cast<int>(chunks));
}

cudaError_t launch_combine_rows_backward(const void* d_out, const void* y, const float* weights,
                                         const int32_t* slot, const int32_t* rows_used, void* d_y,
                                         float* d_weights, int64_t T, int64_t n, int64_t k,
                                         int64_t H, cudaStream_t st) {
  const int64_t zero = n < kZeroBlocks ? n : kZeroBlocks;
  if (T + zero == 0) return cudaSuccess;
  return launch_pdl(combine_backward_kernel, T + zero, kBackThreads, 0, st,
                    static_cast<const uint4*>(d_out), static_cast<const uint4*>(y), weights, slot,
                    rows_used, static_cast<uint4*>(d_y), d_weights, static_cast<int>(T),
                    static_cast<int>(n), static_cast<int>(k), static_cast<int>(H / 8));
}

}  // namespace fp8bl
