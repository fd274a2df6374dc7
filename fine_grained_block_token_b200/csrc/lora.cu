// Low-rank adapters of many requests at once, added to a shared projection:
//   out_i = y_i + s_l (x_i A_l^T) B_l^T      for the rows i of adapter l
// x [M, K], A [L, R, K], B [L, N, R], y and out [M, N], all bf16; the rows of
// adapter l are order[offsets[l] .. offsets[l+1]); rows behind offsets[L]
// have no adapter and keep y.
//
// Two kernels: the shrink u = x A^T (K is long, R short: split over K) and
// the expand out = y + s u B^T (N is long).  Both are bound by memory -- the
// shrink by x, the expand by y and out -- so the matrix products only have to
// keep out of the way.  A warp takes its operands from global memory straight
// into registers in the fragment layout of mma.m16n8k16: the sum over k (or
// r) may be taken in any order, so lane q of a row group owns 8 neighbouring
// k of every 32 and reads them with one 16-byte load, for both operands
// alike; and the columns of B are dealt to the n index so that a lane ends up
// with 8 neighbouring outputs.  Nothing is staged in shared memory.
//
// u stays in fp32 between the two; the expand splits it into the bf16 nearest
// to it and the bf16 nearest to the rest (16 significant bits together) and
// multiplies B by both, so that the one rounding of the result is that of
// out.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp8bl_internal.h"
#include "ptx_sm100.cuh"

namespace fp8bl {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
// y may be out: the plain (coherent) path
__device__ __forceinline__ uint4 ld_y(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// The block's tile: up to `bm` consecutive sorted rows of one adapter.
struct Tile {
  int group;  // adapter, or L for rows without one
  int pos;    // first sorted row
  int rows;
};

// Tiles are numbered group by group, ceil(rows / bm) each.  Every thread owns
// `own` neighbouring groups and keeps the number of tiles before them, so that
// finding one tile after another needs one scan.  Offsets are clamped to
// [0, M]: malformed ones cannot lead outside the tensors.
struct TileMap {
  const int32_t* off;
  int M, L, bm, own;
  int before;  // tiles before this thread's groups
  int total;

  __device__ __forceinline__ int bound(int g) const {
    if (g > L) return M;  // rows behind the last adapter end with the tensor
    const int v = off[g];
    return v < 0 ? 0 : v > M ? M : v;
  }

  __device__ TileMap(const int32_t* offsets, int M_, int L_, int bm_, int groups, int* scratch)
      : off(offsets), M(M_), L(L_), bm(bm_) {
    own = (groups + kThreads - 1) / kThreads;
    int mine = 0;
    for (int i = 0; i < own; ++i) {
      const int g = threadIdx.x * own + i;
      if (g >= groups) break;
      const int n = bound(g + 1) - bound(g);
      if (n > 0) mine += (n + bm - 1) / bm;
    }
    const int l = threadIdx.x % 32, w = threadIdx.x / 32;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, incl, o);
      if (l >= o) incl += v;
    }
    if (l == 31) scratch[w] = incl;
    __syncthreads();
    before = incl - mine;
    total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < w) before += scratch[i];
      total += scratch[i];
    }
  }

  // Whole block; `t` < total.
  __device__ Tile find(int t, int groups, Tile* shared) const {
    __syncthreads();
    int at = before;
    for (int i = 0; i < own; ++i) {
      const int g = threadIdx.x * own + i;
      if (g >= groups) break;
      const int b = bound(g), n = bound(g + 1) - b;
      const int tiles = n > 0 ? (n + bm - 1) / bm : 0;
      if (t >= at && t < at + tiles) {
        const int r = (t - at) * bm;
        *shared = Tile{g, b + r, n - r < bm ? n - r : bm};
      }
      at += tiles;
    }
    __syncthreads();
    return *shared;
  }
};

struct LoraArgs {
  const void* x;
  const void* a;
  const void* b;
  const float* scales;
  const int32_t* offsets;
  const int32_t* order;
  const void* y;
  void* out;
  float* u;      // [splits][M][RP]: sorted row, rank padded to 16 kRT
  int M, N, K, R, L;
  int splits;    // parts of K
};

// kMT 16-row fragments per warp, kRW warps over the rows of a tile; the other
// warps of the block share the long axis.
template <int kRT, int kMT, int kRW>
struct Shape {
  static constexpr int RP = 16 * kRT;
  static constexpr int kRows = 16 * kMT * kRW;
  static constexpr int kCW = kWarps / kRW;
};

template <int kRT, int kMT, int kRW>
__global__ void __launch_bounds__(kThreads) lora_shrink_kernel(const LoraArgs p) {
  using S = Shape<kRT, kMT, kRW>;
  extern __shared__ __align__(16) float part[];  // [kCW][kRows][RP]
  __shared__ int scratch[kWarps];
  __shared__ Tile tile_s;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const TileMap map(p.offsets, p.M, p.L, S::kRows, p.L, scratch);
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rw = w % kRW, cw = w / kRW, g = lane / 4, q = lane % 4;
  // this block's part of K, in steps of 32
  const int steps = (p.K + 31) / 32;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps) * blockIdx.y / p.splits);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (blockIdx.y + 1) / p.splits);

  for (int t = blockIdx.x; t < map.total; t += gridDim.x) {
    const Tile tile = map.find(t, p.L, &tile_s);
    const uint4* xp[kMT][2];
    bool live[kMT][2];
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = (rw * kMT + m) * 16 + h * 8 + g;
        const int row = r < tile.rows ? p.order[tile.pos + r] : -1;
        live[m][h] = row >= 0 && row < p.M;
        xp[m][h] = reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(p.x) +
            static_cast<int64_t>(live[m][h] ? row : 0) * p.K + q * 8);
      }
    const __nv_bfloat16* ap =
        static_cast<const __nv_bfloat16*>(p.a) + static_cast<int64_t>(tile.group) * p.R * p.K + q * 8;
    float acc[kMT][2 * kRT][4] = {};
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 2
    for (int s = s0 + cw; s < s1; s += S::kCW) {
      const bool in = s * 32 + q * 8 < p.K;
      uint4 xv[kMT][2], av[2 * kRT];
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          xv[m][h] = in && live[m][h] ? ld_stream(xp[m][h] + s * 4) : zero;
#pragma unroll
      for (int n = 0; n < 2 * kRT; ++n) {
        const int r = n * 8 + g;
        av[n] = in && r < p.R
                    ? __ldg(reinterpret_cast<const uint4*>(ap + static_cast<int64_t>(r) * p.K) + s * 4)
                    : zero;
      }
#pragma unroll
      for (int n = 0; n < 2 * kRT; ++n)
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
          mma_bf16(acc[m][n], xv[m][0].x, xv[m][1].x, xv[m][0].y, xv[m][1].y, av[n].x, av[n].y);
          mma_bf16(acc[m][n], xv[m][0].z, xv[m][1].z, xv[m][0].w, xv[m][1].w, av[n].z, av[n].w);
        }
    }
    // the warps that share a row meet in shared memory, added in their order
    float* mine = part + static_cast<int64_t>(cw) * S::kRows * S::RP;
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
      for (int n = 0; n < 2 * kRT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(
              &mine[((rw * kMT + m) * 16 + h * 8 + g) * S::RP + n * 8 + q * 2]) =
              make_float2(acc[m][n][2 * h], acc[m][n][2 * h + 1]);
    __syncthreads();
    float* up = p.u + (static_cast<int64_t>(blockIdx.y) * p.M + tile.pos) * S::RP;
    for (int i = threadIdx.x * 4; i < tile.rows * S::RP; i += kThreads * 4) {
      float4 v = *reinterpret_cast<const float4*>(part + i);
#pragma unroll
      for (int c = 1; c < S::kCW; ++c) {
        const float4 o = *reinterpret_cast<const float4*>(part + c * S::kRows * S::RP + i);
        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
      }
      *reinterpret_cast<float4*>(up + i) = v;
    }
  }
}

// Fragments of u for 16 rows: lane (g, q) holds, per 32 ranks, the 8 from
// 8 q on, rows g and g + 8; with 16 ranks the 4 from 4 q on.
template <int kRT>
struct UFrag {
  uint32_t hi[kRT][4], lo[kRT][4];
};

__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(a, b);
  // an infinite or NaN u has no rest
  const float ra = a - lo_f(hi), rb = b - hi_f(hi);
  lo = pack_bf16(ra == ra ? ra : 0.0f, rb == rb ? rb : 0.0f);
}

template <int kRT, int kMT, int kRW>
__global__ void __launch_bounds__(kThreads) lora_expand_kernel(const LoraArgs p, bool copy_rest) {
  using S = Shape<kRT, kMT, kRW>;
  __shared__ int scratch[kWarps];
  __shared__ Tile tile_s;
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const int groups = p.L + (copy_rest ? 1 : 0);
  const TileMap map(p.offsets, p.M, p.L, S::kRows, groups, scratch);
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rw = w % kRW, cw = w / kRW, g = lane / 4, q = lane % 4;
  // this block's part of N, in steps of 32
  const int steps = (p.N + 31) / 32;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps) * blockIdx.y / gridDim.y);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (blockIdx.y + 1) / gridDim.y);

  for (int t = blockIdx.x; t < map.total; t += gridDim.x) {
    const Tile tile = map.find(t, groups, &tile_s);
    int64_t yo[kMT][2];
    bool live[kMT][2];
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = (rw * kMT + m) * 16 + h * 8 + g;
        const int row = r < tile.rows ? p.order[tile.pos + r] : -1;
        live[m][h] = row >= 0 && row < p.M;
        yo[m][h] = static_cast<int64_t>(row) * p.N + q * 8;
      }
    const __nv_bfloat16* yp = static_cast<const __nv_bfloat16*>(p.y);
    __nv_bfloat16* op = static_cast<__nv_bfloat16*>(p.out);
    if (tile.group == p.L) {  // no adapter: out = y
      for (int s = s0 + cw; s < s1; s += S::kCW) {
        if (s * 32 + q * 8 >= p.N) continue;
#pragma unroll
        for (int m = 0; m < kMT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (live[m][h])
              *reinterpret_cast<uint4*>(op + yo[m][h] + s * 32) =
                  ld_y(reinterpret_cast<const uint4*>(yp + yo[m][h] + s * 32));
      }
      continue;
    }

    // u of the tile's rows, summed over the parts of K in order
    UFrag<kRT> f[kMT];
    const float scale = p.scales ? p.scales[tile.group] : 1.0f;
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = (rw * kMT + m) * 16 + h * 8 + g;
        const bool in = r < tile.rows;
        const float* up = p.u + static_cast<int64_t>(tile.pos + (in ? r : 0)) * S::RP;
        const int64_t stride = static_cast<int64_t>(p.M) * S::RP;
        constexpr int kRun = kRT == 1 ? 4 : 8;  // neighbouring ranks of a lane
#pragma unroll
        for (int tt = 0; tt < (kRT + 1) / 2; ++tt) {
          // ranks past R are padding (their u is NaN beside an infinite x)
          float v[kRun] = {};
          if (in && tt * 32 + q * kRun < p.R) {
            for (int c = 0; c < p.splits; ++c) {
#pragma unroll
              for (int i = 0; i < kRun; i += 4) {
                const float4 o =
                    *reinterpret_cast<const float4*>(up + c * stride + tt * 32 + q * kRun + i);
                v[i] += o.x, v[i + 1] += o.y, v[i + 2] += o.z, v[i + 3] += o.w;
              }
            }
          }
#pragma unroll
          for (int i = 0; i < kRun; i += 4) {
            // ranks i, i+1 are the fragment's first pair, i+2, i+3 its second
            const int k16 = tt * 2 + i / 4;
            split2(v[i] * scale, v[i + 1] * scale, f[m].hi[k16][h], f[m].lo[k16][h]);
            split2(v[i + 2] * scale, v[i + 3] * scale, f[m].hi[k16][2 + h], f[m].lo[k16][2 + h]);
          }
        }
      }

    const __nv_bfloat16* bp =
        static_cast<const __nv_bfloat16*>(p.b) + static_cast<int64_t>(tile.group) * p.N * p.R;
    for (int s = s0 + cw; s < s1; s += S::kCW) {
      const bool in = s * 32 + q * 8 < p.N;
      uint4 yv[kMT][2];
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (in && live[m][h])
            yv[m][h] = ld_y(reinterpret_cast<const uint4*>(yp + yo[m][h] + s * 32));
      float acc[kMT][4][4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // n index g of tile j is column (g / 2) * 8 + j * 2 + g % 2
        const int col = s * 32 + (g >> 1) * 8 + j * 2 + (g & 1);
        const __nv_bfloat16* br = bp + static_cast<int64_t>(col) * p.R;
        if constexpr (kRT == 1) {
          const uint2 bv = col < p.N && q * 4 < p.R
                               ? __ldg(reinterpret_cast<const uint2*>(br + q * 4))
                               : make_uint2(0, 0);
#pragma unroll
          for (int m = 0; m < kMT; ++m) {
            mma_bf16(acc[m][j], f[m].lo[0][0], f[m].lo[0][1], f[m].lo[0][2], f[m].lo[0][3], bv.x, bv.y);
            mma_bf16(acc[m][j], f[m].hi[0][0], f[m].hi[0][1], f[m].hi[0][2], f[m].hi[0][3], bv.x, bv.y);
          }
        } else {
          uint4 bv[kRT / 2];
#pragma unroll
          for (int tt = 0; tt < kRT / 2; ++tt)
            bv[tt] = col < p.N && tt * 32 + q * 8 < p.R
                         ? __ldg(reinterpret_cast<const uint4*>(br + tt * 32 + q * 8))
                         : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int tt = 0; tt < kRT / 2; ++tt)
#pragma unroll
            for (int m = 0; m < kMT; ++m) {
              const uint32_t(&l0)[4] = f[m].lo[2 * tt];
              const uint32_t(&h0)[4] = f[m].hi[2 * tt];
              const uint32_t(&l1)[4] = f[m].lo[2 * tt + 1];
              const uint32_t(&h1)[4] = f[m].hi[2 * tt + 1];
              mma_bf16(acc[m][j], l0[0], l0[1], l0[2], l0[3], bv[tt].x, bv[tt].y);
              mma_bf16(acc[m][j], h0[0], h0[1], h0[2], h0[3], bv[tt].x, bv[tt].y);
              mma_bf16(acc[m][j], l1[0], l1[1], l1[2], l1[3], bv[tt].z, bv[tt].w);
              mma_bf16(acc[m][j], h1[0], h1[1], h1[2], h1[3], bv[tt].z, bv[tt].w);
            }
        }
      }
      // accumulator column 2 q + i of tile j is column 8 q + 2 j + i
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (in && live[m][h]) {
            const uint4 v = yv[m][h];
            const float* c0 = acc[m][0] + 2 * h;
            const float* c1 = acc[m][1] + 2 * h;
            const float* c2 = acc[m][2] + 2 * h;
            const float* c3 = acc[m][3] + 2 * h;
            *reinterpret_cast<uint4*>(op + yo[m][h] + s * 32) =
                make_uint4(pack_bf16(lo_f(v.x) + c0[0], hi_f(v.x) + c0[1]),
                           pack_bf16(lo_f(v.y) + c1[0], hi_f(v.y) + c1[1]),
                           pack_bf16(lo_f(v.z) + c2[0], hi_f(v.z) + c2[1]),
                           pack_bf16(lo_f(v.w) + c3[0], hi_f(v.w) + c3[1]));
          }
    }
  }
}

int rank_tiles(int64_t R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

// Small batches take 16-row tiles (a tile per adapter in use, every warp of a
// block on the long axis), larger ones 64-row tiles.
constexpr int64_t kSmallM = 256;

struct Plan {
  int bm, rt;
  int64_t tiles;   // upper bound, or the number of blocks that stride over them
  int splits, nsplits;
};

Plan plan_lora(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L, int sm_count) {
  Plan p;
  p.rt = rank_tiles(R);
  p.bm = M <= kSmallM ? 16 : 64;
  const int64_t least = (M + p.bm - 1) / p.bm;
  const int64_t most = M / p.bm + (L + 1 < M ? L + 1 : M);
  // partial tiles of many small adapters: blocks stride over the rest
  p.tiles = most < 2 * least + sm_count ? most : 2 * least + sm_count;
  // about two blocks per SM on each axis' long side, at least 256 of K and
  // 256 columns each
  const int64_t want = (2 * sm_count + least - 1) / least;
  const int64_t kmax = (K + 255) / 256, nmax = (N + 255) / 256;
  int64_t s = want < kmax ? want : kmax;
  p.splits = static_cast<int>(s < 1 ? 1 : s > 16 ? 16 : s);
  int64_t n = 2 * want < nmax ? 2 * want : nmax;
  p.nsplits = static_cast<int>(n < 1 ? 1 : n > 256 ? 256 : n);
  return p;
}

template <typename Kernel, typename... Args>
cudaError_t launch_pdl(Kernel k, dim3 grid, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  set_programmatic_serialization(at[0]);
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

template <int kRT, int kMT, int kRW>
cudaError_t launch_shape(const LoraArgs& a, const Plan& pl, bool copy_rest, cudaStream_t st) {
  using S = Shape<kRT, kMT, kRW>;
  constexpr size_t smem = static_cast<size_t>(S::kCW) * S::kRows * S::RP * 4;  // <= 64 KB
  static std::once_flag once[kMaxDevices];
  static cudaError_t status[kMaxDevices];
  cudaError_t e = once_per_device(once, status, [](int) {
    return cudaFuncSetAttribute(lora_shrink_kernel<kRT, kMT, kRW>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(smem));
  });
  if (e != cudaSuccess) return e;
  e = launch_pdl(lora_shrink_kernel<kRT, kMT, kRW>,
                 dim3(static_cast<unsigned>(pl.tiles), static_cast<unsigned>(pl.splits)), smem, st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(lora_expand_kernel<kRT, kMT, kRW>,
                    dim3(static_cast<unsigned>(pl.tiles), static_cast<unsigned>(pl.nsplits)), 0, st, a,
                    copy_rest);
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L, int sm_count) {
  if (M == 0) return 0;
  const Plan p = plan_lora(M, N, K, R, L, sm_count);
  return static_cast<size_t>(p.splits) * static_cast<size_t>(M) * 16 * p.rt * 4;
}

cudaError_t launch_lora_add(const void* x, const void* a, const void* b, const float* scales,
                            const int32_t* offsets, const int32_t* order, const void* y, void* out,
                            int64_t M, int64_t N, int64_t K, int64_t R, int64_t L, void* workspace,
                            int sm_count, cudaStream_t st) {
  const Plan p = plan_lora(M, N, K, R, L, sm_count);
  LoraArgs r = {};
  r.x = x;
  r.a = a;
  r.b = b;
  r.scales = scales;
  r.offsets = offsets;
  r.order = order;
  r.y = y;
  r.out = out;
  r.u = static_cast<float*>(workspace);
  r.M = static_cast<int>(M);
  r.N = static_cast<int>(N);
  r.K = static_cast<int>(K);
  r.R = static_cast<int>(R);
  r.L = static_cast<int>(L);
  r.splits = p.splits;
  const bool rest = y != out;
  if (p.bm == 16) switch (p.rt) {
    case 1: return launch_shape<1, 1, 1>(r, p, rest, st);
    case 2: return launch_shape<2, 1, 1>(r, p, rest, st);
    case 4: return launch_shape<4, 1, 1>(r, p, rest, st);
    default: return launch_shape<8, 1, 1>(r, p, rest, st);
  }
  switch (p.rt) {
    case 1: return launch_shape<1, 2, 2>(r, p, rest, st);
    case 2: return launch_shape<2, 2, 2>(r, p, rest, st);
    case 4: return launch_shape<4, 2, 2>(r, p, rest, st);
    default: return launch_shape<8, 1, 4>(r, p, rest, st);
  }
}

}  // namespace fp8bl
