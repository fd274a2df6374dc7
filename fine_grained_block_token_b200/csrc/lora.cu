// Low-rank adapters of many requests at once, added to a shared projection:
//   out_i = y_i + s_l (x_i A_l^T) B_l^T      for the rows i of adapter l
// x [M, K], A [L, R, K], B [L, N, R], y and out [M, N], all bf16; the rows of
// adapter l are order[offsets[l] .. offsets[l+1]); rows behind offsets[L]
// have no adapter and keep y.
//
// Two kernels (for a few rows one): the shrink u = x A^T (K is long, R short)
// and the expand out = y + s u B^T (N is long), both bound by memory.  This
// file holds the form for batches of a few rows per adapter (decode): tiles of
// 16 rows, one mma.m16n8k16 fragment high (the tensor core proper multiplies 64
// or 128 rows at a time; 16 rows leave it nothing to gain while B streams by).
// A warp takes its operands from global memory straight into registers in the
// fragment layout: the sum over k (or r) may be taken in any order, so lane q
// of a row group owns 8 neighbouring k of every 32 and reads them with one
// 16-byte load, for both operands alike; and the columns of B are dealt to the
// n index so that a lane ends up with 8 neighbouring outputs.  Nothing is
// staged in shared memory.
//
// The adapters' matrices are what has to be read, so the work is dealt to
// the whole GPU whatever the number of tiles: the shrink splits K into as
// many parts as its blocks can work on, the expand gives every warp an equal
// run of (tile, 32 columns) steps.  The expand starts while the shrink runs
// (programmatic dependent launch): it finds its tile and loads B and y ahead,
// and only then waits for u.
//
// Beside 28672 x 4096 at rank 16: 64 rows of 48 adapters (58 MB) 17 us where the
// adapters are in L2 from the call before, 27 where they come from memory: the
// chain launch - offsets - x - u precedes all but the first steps of B.  One row
// beside 4096 x 4096 5.1 us.
//
// u stays in fp32 between the two; the expand splits it into the bf16 nearest
// to it and the bf16 nearest to the rest (16 significant bits together) and
// multiplies B by both, so that the one rounding of the result is that of
// out.
#include "lora_common.cuh"

namespace fp8bl {
namespace {

using lora::Args;
using lora::Plan;
using lora::Tile;
using lora::TileMap;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 16;

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}
// y may be out: the plain (coherent) path
__device__ __forceinline__ uint4 ld_y(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Parts of K at most: more shorten the shrink, and the expand has to add them
// up (in one or two batches of loads).
constexpr int kMaxParts = 8;

// Rows that this form can take (their order lies in shared memory).
constexpr int kSmallM = 2048;

// Whether both products run in one launch.  On the GPU it takes as long as two,
// us beside 28672 x 4096: rank 16, 1 row 6.0 | 5.8, 16 rows of 16 adapters 10.7 |
// 11.1, and saves the host 2 (one row beside 4096 x 4096: 12.8 -> 10.5 a call);
// at larger ranks the cluster's 64 warps are too few for B: rank 64, 1 row 7.4 |
// 8.3, but 2 rows 13.5 | 9.8, 16 rows 17 | 12.
bool few_rows(int64_t M, int64_t R) { return M == 1 || (M <= kRows && R <= 16); }

// Whether a batch goes through this form or through the 128-row tiles of
// lora_tiles.cu.  Here the time grows with the number of 16-row tiles and, as
// every tile multiplies all of B by 16 rows, with the rank; there every adapter
// costs at least one 128-row tile.  Both forms, us, beside 28672 x 4096:
//   rank 16,  1 adapter:    1024 rows 30 | 35     2048 rows  64 | 60
//   rank 16,  64 adapters:   256 rows 22 | 133    2048 rows  82 | 138
//   rank 32,  8 adapters:   1024 rows 37 | 37     2048 rows  85 | 67
//   rank 64,  1 adapter:      64 rows 16 | 17      256 rows  23 | 21
//   rank 64,  8 adapters:    256 rows 27 | 31      512 rows  36 | 33
//   rank 128, 1 adapter:      32 rows 21 | 23      256 rows  36 | 27
//   rank 128, 16 adapters:   256 rows 48 | 75     1024 rows 130 | 79
bool small_batch(int64_t M, int64_t R, int64_t L) {
  const int64_t adapters = L < M ? L : M;
  int64_t most = R <= 32 ? 64 * adapters : R <= 64 ? 128 + 48 * adapters : 32 + 32 * adapters;
  if (R <= 32 && most < 1024) most = 1024;
  return M <= most && M <= kSmallM;
}

// The batch's rows in sorted order, on their way together with the offsets
// (one dependent load less); -1 for rows outside [0, M).  The map's barriers
// follow.
__device__ __forceinline__ void load_order(const Args& p, int* order) {
  for (int i = threadIdx.x; i < p.M; i += kThreads) {
    const int row = p.order[i];
    order[i] = row >= 0 && row < p.M ? row : -1;
  }
}

// kRT = rank / 16, rounded up to 1, 2, 4 or 8; RP = 16 kRT.
//
// Products of the tile's rows of x with A over the steps [s0, s1) of 32 along
// K, dealt to the block's warps, each of which leaves its sums in part[warp]
// [kRows][RP].
template <int kRT>
__device__ __forceinline__ void shrink_tile(const Args& p, const Tile& tile, const int* order, int s0,
                                            int s1, float* part) {
  constexpr int RP = 16 * kRT;
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
  const __nv_bfloat16* xp[2];
  bool live[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = h * 8 + g;
    const int row = r < tile.rows ? order[tile.pos + r] : -1;
    live[h] = row >= 0;
    xp[h] = p.x + static_cast<int64_t>(live[h] ? row : 0) * p.K + q * 8;
  }
  const __nv_bfloat16* ap = p.a + static_cast<int64_t>(tile.group) * p.R * p.K + q * 8;
  float acc[2 * kRT][4] = {};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // kTogether steps' loads on their way together
  constexpr int kTogether = kRT == 1 ? 3 : kRT <= 4 ? 2 : 1;
  for (int s = s0 + w; s < s1; s += kTogether * kWarps) {
    uint4 xv[kTogether][2], av[kTogether][2 * kRT];
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      const int k = (s + i * kWarps) * 32;
      const bool in = s + i * kWarps < s1 && k + q * 8 < p.K;
#pragma unroll
      for (int h = 0; h < 2; ++h) xv[i][h] = in && live[h] ? ld_stream(xp[h] + k) : zero;
#pragma unroll
      for (int n = 0; n < 2 * kRT; ++n) {
        const int r = n * 8 + g;
        av[i][n] = in && r < p.R ? ld_stream(ap + static_cast<int64_t>(r) * p.K + k) : zero;
      }
    }
#pragma unroll
    for (int i = 0; i < kTogether; ++i)
#pragma unroll
      for (int n = 0; n < 2 * kRT; ++n) {
        mma_bf16(acc[n], xv[i][0].x, xv[i][1].x, xv[i][0].y, xv[i][1].y, av[i][n].x, av[i][n].y);
        mma_bf16(acc[n], xv[i][0].z, xv[i][1].z, xv[i][0].w, xv[i][1].w, av[i][n].z, av[i][n].w);
      }
  }
  float* mine = part + w * kRows * RP;
#pragma unroll
  for (int n = 0; n < 2 * kRT; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (h * 8 + g < tile.rows)
        *reinterpret_cast<float2*>(&mine[(h * 8 + g) * RP + n * 8 + q * 2]) =
            make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
}

// The warps' sums, added in their order: 4 ranks at i of the tile's [rows][RP].
template <int kRT>
__device__ __forceinline__ float4 sum_warps(const float* part, int i) {
  float4 v = *reinterpret_cast<const float4*>(part + i);
#pragma unroll
  for (int k = 1; k < kWarps; ++k) {
    const float4 o = *reinterpret_cast<const float4*>(part + k * kRows * 16 * kRT + i);
    v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
  }
  return v;
}

template <int kRT>
__global__ void __launch_bounds__(kThreads) lora_shrink_kernel(const Args p) {
  constexpr int RP = 16 * kRT;
  extern __shared__ __align__(16) float part[];  // [kWarps][kRows][RP]
  __shared__ TileMap map;
  __shared__ int order[kSmallM];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  load_order(p, order);
  map.build<kThreads>(p.offsets, p.M, p.L, kRows);
  const int tiles = map.before[p.L];
  const int parts = lora::parts_of_k(p.shrink_blocks, tiles, p.max_splits);
  const int steps = (p.K + 31) / 32;

  for (int item = blockIdx.x; item < tiles * parts; item += gridDim.x) {
    const Tile tile = map.find(item / parts, p.L, kRows);
    const int c = item % parts;
    const int s0 = static_cast<int>(static_cast<int64_t>(steps) * c / parts);
    const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (c + 1) / parts);
    shrink_tile<kRT>(p, tile, order, s0, s1, part);
    __syncthreads();
    float* up = reinterpret_cast<float*>(p.u) + (static_cast<int64_t>(c) * p.M + tile.pos) * RP;
    for (int i = threadIdx.x * 4; i < tile.rows * RP; i += kThreads * 4)
      *reinterpret_cast<float4*>(up + i) = sum_warps<kRT>(part, i);
    __syncthreads();  // the next item writes `part` again
  }
}

// Its first product: the accumulator starts from zero.
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// One step's operands: 32 columns of B (four n8 tiles) and of y.
template <int kRT>
struct Step {
  static constexpr int kB = kRT == 1 ? 2 : kRT * 2;  // 32-bit words per n8 tile
  uint32_t b[4][kB];
  uint4 y[2];
};

// n steps of 32 columns from s0 on of one tile, by one warp.  B and y of the
// first steps are loaded, then before_u() is called (by warps without steps
// too), then sum_u(row, rank, v) adds kRun neighbouring ranks of u to v.
// kExact: the rank is RP itself, so that the strides of B are constants and the
// addresses of a run of steps differ by immediates.
template <int kRT>
constexpr int kRun = kRT == 1 ? 4 : 8;  // neighbouring ranks of a lane

template <int kRT, bool kExact, typename BeforeU, typename SumU>
__device__ __forceinline__ void expand_run(const Args& p, const Tile& tile, const int* order, int s0,
                                           int n, BeforeU before_u, SumU sum_u) {
  constexpr int RP = 16 * kRT, kRun = fp8bl::kRun<kRT>;
  const int R = kExact ? RP : p.R;
  constexpr int kDepth = kRT == 1 ? 4 : kRT <= 4 ? 2 : 1;  // steps loaded ahead
  const int lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
  const bool upper = tile.rows > 8;  // any of rows 8 .. 15
  int64_t yo[2];                     // element of y and out
  bool live[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = h * 8 + g;
    const int row = r < tile.rows ? order[tile.pos + r] : -1;
    live[h] = row >= 0;
    yo[h] = static_cast<int64_t>(live[h] ? row : 0) * p.N + s0 * 32 + q * 8;
  }
  if (tile.group == p.L) {  // no adapter: out = y
    for (int i = 0; i < n; ++i)
      if ((s0 + i) * 32 + q * 8 < p.N)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (live[h])
            *reinterpret_cast<uint4*>(p.out + yo[h] + i * 32) = ld_y(p.y + yo[h] + i * 32);
    return;
  }
  // n index g of n8 tile j is column (g / 2) * 8 + j * 2 + g % 2 of a step
  const int col = s0 * 32 + (g >> 1) * 8 + (g & 1);
  const __nv_bfloat16* bp =
      p.b + (static_cast<int64_t>(tile.group) * p.N + col) * R + q * kRun;
  const bool rank_in = kExact || q * kRun < R;
  const bool whole = (s0 + n) * 32 <= p.N;  // no columns past N in this run
  const __nv_bfloat16* y0 = p.y + yo[0];
  const __nv_bfloat16* y1 = p.y + yo[1];
  // Step i (below n), d steps behind the pointers.  What is not loaded keeps
  // whatever it was: a finite or foreign B past column N meets outputs that
  // are not stored, and ranks past R stay the zeros of the start.
  auto load = [&](Step<kRT>& to, int i, int d) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!(whole || (s0 + i) * 32 + (g >> 1) * 8 + (g & 1) + 2 * j < p.N)) continue;
      const __nv_bfloat16* br = bp + (d * 32 + 2 * j) * R;
      if constexpr (kRT == 1) {
        if (rank_in) {
          const uint2 v = ld_stream8(br);
          to.b[j][0] = v.x, to.b[j][1] = v.y;
        }
      } else {
#pragma unroll
        for (int k = 0; k < kRT / 2; ++k)
          if (kExact || k * 32 + q * 8 < R) {
            const uint4 v = ld_stream(br + k * 32);
            to.b[j][4 * k] = v.x, to.b[j][4 * k + 1] = v.y;
            to.b[j][4 * k + 2] = v.z, to.b[j][4 * k + 3] = v.w;
          }
      }
    }
    if (whole || (s0 + i) * 32 + q * 8 < p.N) {
      if (live[0]) to.y[0] = ld_y(y0 + d * 32);
      if (upper && live[1]) to.y[1] = ld_y(y1 + d * 32);
    }
  };
  Step<kRT> buf[kDepth] = {};
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (d < n) load(buf[d], d, d);

  // u of the tile's rows.  Lane (g, q) holds, per 32 ranks, the 8 from 8 q on
  // (with 16 ranks the 4 from 4 q on) of rows g and g + 8.
  before_u();
  uint32_t hi[kRT][4], lo[kRT][4];
  const float scale = p.scales ? p.scales[tile.group] : 1.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = h * 8 + g;
#pragma unroll
    for (int i = 0; i < (kRT + 1) / 2; ++i) {
      // ranks past R are padding (their u is NaN beside an infinite x)
      float v[kRun] = {};
      if (r < tile.rows && (kExact || i * 32 + q * kRun < R)) sum_u(r, i * 32 + q * kRun, v);
#pragma unroll
      for (int k = 0; k < kRun; k += 4) {
        // ranks k, k+1 are the fragment's first pair, k+2, k+3 its second
        const int f = i * 2 + k / 4;
        lora::split2(v[k] * scale, v[k + 1] * scale, hi[f][h], lo[f][h]);
        lora::split2(v[k + 2] * scale, v[k + 3] * scale, hi[f][2 + h], lo[f][2 + h]);
      }
    }
  }

  __nv_bfloat16* o0 = p.out + yo[0];
  __nv_bfloat16* o1 = p.out + yo[1];
  for (int i0 = 0; i0 < n; i0 += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int i = i0 + d;
      if (i >= n) break;  // the same for the whole warp
      float acc[4][4];
#pragma unroll
      for (int f = 0; f < kRT; ++f)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t b0 = buf[d].b[j][2 * f], b1 = buf[d].b[j][2 * f + 1];
          if (f == 0)
            mma_bf16_first(acc[j], lo[f][0], lo[f][1], lo[f][2], lo[f][3], b0, b1);
          else
            mma_bf16(acc[j], lo[f][0], lo[f][1], lo[f][2], lo[f][3], b0, b1);
          mma_bf16(acc[j], hi[f][0], hi[f][1], hi[f][2], hi[f][3], b0, b1);
        }
      // accumulator column 2 q + k of tile j is column 8 q + 2 j + k
      auto store = [&](__nv_bfloat16* o, const uint4& v, int h) {
        *reinterpret_cast<uint4*>(o) =
            make_uint4(lora::add2(v.x, acc[0][2 * h], acc[0][2 * h + 1]),
                       lora::add2(v.y, acc[1][2 * h], acc[1][2 * h + 1]),
                       lora::add2(v.z, acc[2][2 * h], acc[2][2 * h + 1]),
                       lora::add2(v.w, acc[3][2 * h], acc[3][2 * h + 1]));
      };
      if (whole || (s0 + i) * 32 + q * 8 < p.N) {
        if (live[0]) store(o0 + d * 32, buf[d].y[0], 0);
        if (upper && live[1]) store(o1 + d * 32, buf[d].y[1], 1);
      }
      if (i + kDepth < n) load(buf[d], i + kDepth, d + kDepth);
    }
    bp += kDepth * 32 * R;
    y0 += kDepth * 32, y1 += kDepth * 32;
    o0 += kDepth * 32, o1 += kDepth * 32;
  }
}

template <int kRT, bool kExact>
__global__ void __launch_bounds__(kThreads, kRT <= 2 ? 2 : 1) lora_expand_kernel(const Args p) {
  constexpr int RP = 16 * kRT;
  constexpr int kRun = fp8bl::kRun<kRT>;
  constexpr int kBatch = kRT <= 2 ? 8 : 4;
  __shared__ TileMap map;
  __shared__ int order[kSmallM];
  // The launch before this one is the shrink, whose blocks have all waited
  // for the work before it: offsets, order, B and y are final, u is not yet.
  load_order(p, order);
  map.build<kThreads>(p.offsets, p.M, p.L, kRows);
  const int groups = p.L + p.copy_rest;
  const int tiles = map.before[p.L];
  const int parts = lora::parts_of_k(p.shrink_blocks, tiles, p.max_splits);
  const uint32_t steps = (p.N + 31) / 32;
  // this warp's run of steps: an equal share, the first ones one more
  const uint32_t total = static_cast<uint32_t>(map.before[groups]) * steps;
  const uint32_t warps = gridDim.x * kWarps;
  const uint32_t me = threadIdx.x / 32 * gridDim.x + blockIdx.x;
  const uint32_t share = total / warps, more = total - share * warps;
  uint32_t at = me * share + (me < more ? me : more);
  const uint32_t end = at + share + (me < more ? 1 : 0);
  bool waited = false;

  while (at < end) {
    const int t = static_cast<int>(at / steps), s0 = static_cast<int>(at - t * steps);
    const int n = min(static_cast<int>(end - at), static_cast<int>(steps) - s0);
    at += n;
    const Tile tile = map.find(t, groups, kRows);
    expand_run<kRT, kExact>(
        p, tile, order, s0, n,
        [&] {
          if (!waited) {
            ptx::grid_dep_wait();
            ptx::grid_dep_launch();
            waited = true;
          }
        },
        // the parts of K in order
        [&](int r, int rank, float (&v)[kRun]) {
          const float* up = reinterpret_cast<const float*>(p.u) +
                            static_cast<int64_t>(tile.pos + r) * RP + rank;
          const int64_t stride = static_cast<int64_t>(p.M) * RP;
        // a batch of parts on its way before the first is added
#pragma unroll
        for (int c0 = 0; c0 < kMaxParts; c0 += kBatch) {
          if (c0 >= parts) break;
          float4 o[kBatch][kRun / 4];
#pragma unroll
          for (int c = 0; c < kBatch; ++c)
#pragma unroll
            for (int k = 0; k < kRun / 4; ++k)
              o[c][k] = c0 + c < parts
                            ? *reinterpret_cast<const float4*>(up + (c0 + c) * stride +
                                                               4 * k)
                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int c = 0; c < kBatch; ++c)
#pragma unroll
            for (int k = 0; k < kRun / 4; ++k) {
              v[4 * k] += o[c][k].x, v[4 * k + 1] += o[c][k].y;
              v[4 * k + 2] += o[c][k].z, v[4 * k + 3] += o[c][k].w;
            }
        }
        });
  }
  if (!waited) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
  }
}

// Both products in one launch, for a few rows: a cluster of kFew blocks takes a
// tile (and, with few tiles, a share of its columns).  Each block shrinks over
// its part of K, the parts meet through distributed shared memory in their
// order, and every warp expands some steps.  Clusters that share a tile each
// shrink it for themselves, from L2.
constexpr int kFew = 8;

template <int kRT, bool kExact>
__global__ void __launch_bounds__(kThreads, kRT <= 2 ? 2 : 1) lora_few_kernel(const Args p) {
  constexpr int RP = 16 * kRT;
  extern __shared__ __align__(16) float part[];  // [kWarps][kRows][RP], sums, u
  float* sums = part + kWarps * kRows * RP;      // [kRows][RP] of this part of K
  float* u = sums + kRows * RP;                  // of all
  __shared__ TileMap map;
  __shared__ int order[kSmallM];
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  load_order(p, order);
  map.build<kThreads>(p.offsets, p.M, p.L, kRows);
  const int groups = p.L + p.copy_rest, tiles = map.before[groups];
  const int clusters = gridDim.x / kFew, rank = static_cast<int>(ptx::cluster_ctarank());
  const int shares = tiles > 0 && tiles < clusters ? clusters / tiles : 1;
  const int ksteps = (p.K + 31) / 32, steps = (p.N + 31) / 32;
  const int me = threadIdx.x / 32 * kFew + rank;  // of the cluster's warps

  for (int item = blockIdx.x / kFew; item < tiles * shares; item += clusters) {
    const Tile tile = map.find(item / shares, groups, kRows);
    // this warp's run of the tile's steps
    const int64_t of = static_cast<int64_t>(shares) * kFew * kWarps;
    const int64_t at = static_cast<int64_t>(item % shares) * kFew * kWarps + me;
    const int s0 = static_cast<int>(steps * at / of), n = static_cast<int>(steps * (at + 1) / of) - s0;
    if (tile.group < p.L)
      shrink_tile<kRT>(p, tile, order, static_cast<int>(static_cast<int64_t>(ksteps) * rank / kFew),
                       static_cast<int>(static_cast<int64_t>(ksteps) * (rank + 1) / kFew), part);
    expand_run<kRT, kExact>(
        p, tile, order, s0, n,
        [&] {  // not called for rows without an adapter, by none of the cluster
          __syncthreads();
          for (int i = threadIdx.x * 4; i < tile.rows * RP; i += kThreads * 4)
            *reinterpret_cast<float4*>(sums + i) = sum_warps<kRT>(part, i);
          __syncwarp();
          ptx::cluster_sync();
          for (int i = threadIdx.x * 4; i < tile.rows * RP; i += kThreads * 4) {
            float4 v[kFew];
#pragma unroll
            for (int c = 0; c < kFew; ++c)
              v[c] = ptx::ld_cluster_f4(ptx::map_to_cta(ptx::smem_u32(sums + i), c));
#pragma unroll
            for (int c = 1; c < kFew; ++c)
              v[0].x += v[c].x, v[0].y += v[c].y, v[0].z += v[c].z, v[0].w += v[c].w;
            *reinterpret_cast<float4*>(u + i) = v[0];
          }
          __syncthreads();
        },
        [&](int r, int rank0, float (&v)[kRun<kRT>]) {
#pragma unroll
          for (int k = 0; k < kRun<kRT>; k += 4) {
            const float4 o = *reinterpret_cast<const float4*>(u + r * RP + rank0 + k);
            v[k] += o.x, v[k + 1] += o.y, v[k + 2] += o.z, v[k + 3] += o.w;
          }
        });
    __syncwarp();
    ptx::cluster_sync();  // the others have read this block's sums
  }
}

Plan plan_lora(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L, int sm_count) {
  if (!small_batch(M, R, L)) return lora::plan_tiles(M, N, K, R, L, sm_count);
  Plan p;
  p.rt = lora::rank_tiles(R);
  // tiles at most: full ones, and one more for each group with rows
  const int64_t tiles = M / kRows + (L + 1 < M ? L + 1 : M);
  // a part of K is at least 256 deep: one step of 32 for each warp
  const int64_t parts = (K + 255) / 256;
  p.max_splits = static_cast<int>(parts < kMaxParts ? parts : kMaxParts);
  const int64_t sb = tiles * p.max_splits, eb = (tiles * ((N + 31) / 32) + kWarps - 1) / kWarps;
  // all blocks resident at once: registers allow two per SM, one at the
  // ranks that fill them
  const int64_t sr = sm_count * (p.rt <= 4 ? 2 : 1), er = sm_count * (p.rt <= 2 ? 2 : 1);
  p.shrink_blocks = static_cast<int>(sb < sr ? sb : sr);
  p.expand_blocks = static_cast<int>(eb < er ? eb : er);
  p.u_bytes = static_cast<size_t>(p.max_splits) * static_cast<size_t>(M) * 16 * p.rt * 4;
  p.few_clusters = 0;
  if (few_rows(M, R)) {
    // a step for every warp of a cluster before there is another one
    const int64_t want = tiles * ((N + 32 * kFew * kWarps - 1) / (32 * kFew * kWarps));
    const int64_t fit = sm_count / kFew;
    p.few_clusters = static_cast<int>(want < fit ? want : fit);
    p.u_bytes = 0;
  }
  return p;
}

template <typename Kernel>
cudaError_t launch_pdl(Kernel k, int blocks, int cluster, size_t smem, cudaStream_t st,
                       const Args& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  set_programmatic_serialization(at[0]);
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, a);
}

template <int kRT>
cudaError_t launch_rank(const Args& a, const Plan& pl, cudaStream_t st) {
  constexpr size_t smem = static_cast<size_t>(kWarps) * kRows * 16 * kRT * 4;  // <= 64 KB
  constexpr size_t smem_few = smem / kWarps * (kWarps + 2);
  static std::once_flag once[kMaxDevices];
  static cudaError_t status[kMaxDevices];
  cudaError_t e = once_per_device(once, status, [](int) {
    const auto opt_in = [](const void* k, size_t bytes) {
      return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(bytes));
    };
    cudaError_t f = opt_in(reinterpret_cast<const void*>(lora_shrink_kernel<kRT>), smem);
    if (f == cudaSuccess)
      f = opt_in(reinterpret_cast<const void*>(lora_few_kernel<kRT, true>), smem_few);
    if (f == cudaSuccess)
      f = opt_in(reinterpret_cast<const void*>(lora_few_kernel<kRT, false>), smem_few);
    return f;
  });
  if (e != cudaSuccess) return e;
  const bool exact = a.R == 16 * kRT;
  if (pl.few_clusters > 0) {
    const auto few = exact ? lora_few_kernel<kRT, true> : lora_few_kernel<kRT, false>;
    return launch_pdl(few, pl.few_clusters * kFew, kFew, smem_few, st, a);
  }
  e = launch_pdl(lora_shrink_kernel<kRT>, pl.shrink_blocks, 1, smem, st, a);
  if (e != cudaSuccess) return e;
  const auto expand = exact ? lora_expand_kernel<kRT, true> : lora_expand_kernel<kRT, false>;
  return launch_pdl(expand, pl.expand_blocks, 1, 0, st, a);
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L, int sm_count) {
  if (M == 0) return 0;
  return plan_lora(M, N, K, R, L, sm_count).u_bytes;
}

cudaError_t launch_lora_add(const void* x, const void* a, const void* b, const float* scales,
                            const int32_t* offsets, const int32_t* order, const void* y, void* out,
                            int64_t M, int64_t N, int64_t K, int64_t R, int64_t L, void* workspace,
                            const DeviceInfo& dev, cudaStream_t st) {
  const Plan p = plan_lora(M, N, K, R, L, dev.sm_count);
  Args r = {};
  r.x = static_cast<const __nv_bfloat16*>(x);
  r.a = static_cast<const __nv_bfloat16*>(a);
  r.b = static_cast<const __nv_bfloat16*>(b);
  r.scales = scales;
  r.offsets = offsets;
  r.order = order;
  r.y = static_cast<const __nv_bfloat16*>(y);
  r.out = static_cast<__nv_bfloat16*>(out);
  r.u = static_cast<__nv_bfloat16*>(workspace);
  r.M = static_cast<int>(M);
  r.N = static_cast<int>(N);
  r.K = static_cast<int>(K);
  r.R = static_cast<int>(R);
  r.L = static_cast<int>(L);
  r.max_splits = p.max_splits;
  r.shrink_blocks = p.shrink_blocks;
  r.copy_rest = y != out;
  r.err = dev.error_flag;
  if (!small_batch(M, R, L)) return lora::launch_tiles(r, p, st);
  switch (p.rt) {
    case 1: return launch_rank<1>(r, p, st);
    case 2: return launch_rank<2>(r, p, st);
    case 4: return launch_rank<4>(r, p, st);
    default: return launch_rank<8>(r, p, st);
  }
}

}  // namespace fp8bl
