// Low-rank adapters for long batches (prompts): the same two products as
// lora.cu in tiles of 128 sorted rows on the tensor core (tcgen05, bf16 in,
// fp32 in tensor memory).
//
// Shrink, u = x A^T: bound by reading x.  128 threads copy 64-deep slices of
// the tile's rows (wherever `order` says they are) and of A into a ring of
// 128-byte-swizzled shared-memory stages with cp.async; one thread issues the
// MMAs.  K is split over the blocks of a cluster so that all SMs have work;
// the blocks' sums meet through distributed shared memory, added in the order
// of the parts, and leave as two bf16 terms side by side ([hi | lo], 2 RP
// deep).  (Parts that the expand adds up instead cost 38 of 137 us beside
// 28672 x 4096 at rank 64 and 4096 rows: every block of the expand read all
// seven.)
//
// Expand, out = y + s u B^T: bound by reading y and writing out.  One
// accumulation over hi and lo with B read twice multiplies by all 16 bits of
// u.  Work is
// numbered in chunks of 64 columns, tile after tile, and every block takes an
// equal run of chunks.  Of a chunk, B comes by TMA, the MMAs run into one of
// two halves of tensor memory, and the 128 epilogue threads stream y through
// a ring of shared-memory slots: cp.async in (8 lanes per 128-byte row
// piece), add the accumulator row by row (a thread per row, as tensor memory
// hands it out), write back, and out again in whole row pieces.
//
// Every wait is bounded; a thread whose wait ran out records the error, stops
// waiting and runs its loops out (the barriers between threads still match).
#include "lora_common.cuh"

namespace fp8bl {
namespace {

using lora::Args;
using lora::Tile;
using lora::TileMap;

constexpr int kRows = 128;      // rows of a tile
constexpr int kDeep = 64;       // bf16 per 128-byte row of a shared-memory block
constexpr int kBlock = kRows * 128;  // bytes of a [128 x 64] block

__device__ __forceinline__ void record_error(int* err, int code) { atomicCAS(err, 0, code); }

// Byte offset of 16-byte chunk c of row r in a 128-byte-swizzled block.
__device__ __forceinline__ uint32_t cell(int r, int c) {
  return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) &
                                    ~static_cast<uintptr_t>(1023));
}

// ----------------------------------------------------------------- shrink

template <int kRT>
struct ShrinkShape {
  static constexpr int RP = 16 * kRT;
  static constexpr int kTmem = RP < 32 ? 32 : RP;  // columns, at least 32
  static constexpr int kQuads = RP / 4;            // 16-byte quads of a row of sums
  static constexpr int kSwizzle = kQuads < 8 ? kQuads - 1 : 7;
  static constexpr int kStages = kRT <= 2 ? 5 : kRT == 4 ? 4 : 3;
  static constexpr int kA = RP * 128;  // bytes of A per stage
  static constexpr int kStage = kBlock + kA;
  static constexpr int kAhead = kStages == 3 ? 2 : kStages - 2;  // stages on their way
  static constexpr int kSmem = kStages * kStage + 1024;
  static_assert(kRows * RP * 4 <= kStages * kStage, "the sums fit the ring");
};

constexpr int kShrinkThreads = 160;  // 4 copying warps, 1 MMA warp

template <int kRT>
__global__ void __launch_bounds__(kShrinkThreads, 2) lora_shrink_tiles_kernel(const Args p) {
  using S = ShrinkShape<kRT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  __shared__ TileMap map;
  __shared__ __align__(8) uint64_t bars[2 * S::kStages + 1];
  __shared__ uint32_t tmem_holder;
  const uint32_t base = ptx::smem_u32(smem), bar0 = ptx::smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (S::kStages + s); };
  const uint32_t done = bar0 + 8u * (2 * S::kStages);
  const int warp = threadIdx.x / 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      ptx::mbar_init(full(s), 128);
      ptx::mbar_init(empty(s), 1);
    }
    ptx::mbar_init(done, 1);
    ptx::fence_barrier_init();
  }
  if (warp == 4) {
    ptx::tmem_alloc(ptx::smem_u32(&tmem_holder), S::kTmem);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  map.build<kShrinkThreads>(p.offsets, p.M, p.L, kRows);
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_holder);
  const int tiles = map.before[p.L];
  const int parts = p.max_splits;  // blocks of a cluster, one part of K each
  const int part = static_cast<int>(ptx::cluster_ctarank());
  const int clusters = gridDim.x / parts;
  const int blocks_k = (p.K + kDeep - 1) / kDeep;
  bool ok = true;
  uint32_t n_used = 0;  // stages used so far
  uint32_t item_phase = 0;

  for (int t = blockIdx.x / parts; t < tiles; t += clusters, item_phase ^= 1) {
    const Tile tile = map.find(t, p.L, kRows);
    const int k0 = static_cast<int>(static_cast<int64_t>(blocks_k) * part / parts);
    const int n = static_cast<int>(static_cast<int64_t>(blocks_k) * (part + 1) / parts) - k0;
    if (warp < 4) {
      const int c = threadIdx.x % 8, r0 = threadIdx.x / 8;  // chunk and first of 8 rows
      const __nv_bfloat16* xp[8];
      unsigned live = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        const int row = r < tile.rows ? p.order[tile.pos + r] : -1;
        const bool in = row >= 0 && row < p.M;
        live |= static_cast<unsigned>(in) << i;
        xp[i] = p.x + static_cast<int64_t>(in ? row : 0) * p.K;
      }
      const __nv_bfloat16* ap = p.a + static_cast<int64_t>(tile.group) * p.R * p.K;
      const uint32_t dst0 = cell(r0, c);
      for (int i = 0; i < n + S::kAhead; ++i) {
        if (i < n) {
          const uint32_t u = n_used + i;
          const int s = u % S::kStages;
          if (ok && !ptx::mbar_wait(empty(s), ((u / S::kStages) & 1u) ^ 1u)) {
            record_error(p.err, kErrTimeoutProducer);
            ok = false;
          }
          const uint32_t dst = base + s * S::kStage + dst0;
          const int k = (k0 + i) * kDeep + c * 8;
          const bool in = k < p.K;
          const int ks = in ? k : 0;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            ptx::cp_async16(dst + j * 2048, xp[j] + ks, in && (live >> j & 1));
#pragma unroll
          for (int j = 0; j < kRT; ++j) {
            const int r = r0 + 16 * j;
            ptx::cp_async16(dst + kBlock + j * 2048,
                            ap + static_cast<int64_t>(r < p.R ? r : 0) * p.K + ks, in && r < p.R);
          }
        }
        ptx::cp_async_commit();
        if (i >= S::kAhead) {
          // the copies of this thread have landed: visible to the tensor core
          ptx::cp_async_wait<S::kAhead>();
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(full((n_used + i - S::kAhead) % S::kStages));
        }
      }
      if (ok && !ptx::mbar_wait(done, item_phase)) {
        record_error(p.err, kErrTimeoutEpilogue);
        ok = false;
      }
      ptx::tc_fence_after();
      // this part's sums, a row per thread, into the ring (the MMAs are
      // through with it); 16-byte quads swizzled by row against bank conflicts
      const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
      uint4* row = reinterpret_cast<uint4*>(smem) + threadIdx.x * S::kQuads;
      const int sw = threadIdx.x & S::kSwizzle;
      if constexpr (kRT == 1) {
        uint32_t v[16];
        ptx::tmem_ld_32x32b_x16(lane_base, v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          row[j ^ sw] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      } else {
#pragma unroll
        for (int h = 0; h < kRT / 2; ++h) {
          uint32_t v[32];
          ptx::tmem_ld_32x32b_x32(lane_base + 32 * h, v);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            row[(8 * h + j) ^ sw] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
      }
      // the next item's MMAs start behind these reads: they wait for stages
      // that all copying threads fill afterwards
      ptx::tc_fence_before();
    } else {
      for (int i = 0; i < n && ok; ++i) {
        const uint32_t u = n_used + i;
        const int s = u % S::kStages;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_spin(full(s), (u / S::kStages) & 1u));
        if (!ok) {
          if (threadIdx.x % 32 == 0) record_error(p.err, kErrTimeoutMma);
          break;
        }
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint64_t xd = ptx::sdesc_kmajor_sw128(base + s * S::kStage);
          const uint64_t ad = ptx::sdesc_kmajor_sw128(base + s * S::kStage + kBlock);
#pragma unroll
          for (int k = 0; k < kDeep / 16; ++k)
            ptx::mma_f16(tmem, ptx::sdesc_advance(xd, k * 32), ptx::sdesc_advance(ad, k * 32),
                         ptx::idesc_bf16_f32(kRows, S::RP), (i | k) != 0 ? 1u : 0u);
          ptx::mma_commit(empty(s));
          if (i == n - 1) ptx::mma_commit(done);
        }
        __syncwarp();
      }
    }
    n_used += n;
    __syncwarp();
    ptx::cluster_sync();
    // every block adds up its share of the rows over all parts, in order
    if (warp < 4) {
      const int share = (kRows + parts - 1) / parts, r_first = part * share;
      const float scale = p.scales ? p.scales[tile.group] : 1.0f;
      __nv_bfloat16* up = p.u + static_cast<int64_t>(tile.pos) * (2 * S::RP);
      for (int f = threadIdx.x; f < share * S::kQuads; f += 128) {
        const int r = r_first + f / S::kQuads, j = f % S::kQuads;
        if (r >= tile.rows) break;
        const uint32_t at = base + (r * S::kQuads + (j ^ (r & S::kSwizzle))) * 16;
        float4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < parts) v[c] = ptx::ld_cluster_f4(ptx::map_to_cta(at, c));
#pragma unroll
        for (int c = 1; c < 8; ++c)
          if (c < parts) v[0].x += v[c].x, v[0].y += v[c].y, v[0].z += v[c].z, v[0].w += v[c].w;
        uint2 hi, lo;
        // ranks past R are padding (their sum is NaN beside an infinite x)
        if (4 * j >= p.R) v[0] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        lora::split2(v[0].x * scale, v[0].y * scale, hi.x, lo.x);
        lora::split2(v[0].z * scale, v[0].w * scale, hi.y, lo.y);
        __nv_bfloat16* o = up + static_cast<int64_t>(r) * (2 * S::RP) + 4 * j;
        *reinterpret_cast<uint2*>(o) = hi;
        *reinterpret_cast<uint2*>(o + S::RP) = lo;
      }
    }
    __syncwarp();
    ptx::cluster_sync();  // the ring is free again, here and for the others' reads
  }
  ptx::cp_async_wait<0>();
  ptx::tc_fence_before();
  __syncthreads();  // the copying warps have read what the last MMAs wrote
  if (warp == 4) ptx::tmem_dealloc(tmem, S::kTmem);
}

// ----------------------------------------------------------------- expand

constexpr int kCols = 64;            // columns of a chunk
constexpr int kExpandThreads = 192;  // 4 epilogue warps, 1 MMA warp, 1 TMA warp

template <int kRT>
struct ExpandShape {
  static constexpr int RP = 16 * kRT;
  static constexpr int kUBlocks = (2 * RP + kDeep - 1) / kDeep;  // [hi | lo], 64 deep each
  static constexpr int kBBlocks = (RP + kDeep - 1) / kDeep;
  static constexpr int kBStage = kBBlocks * kCols * 128;
  static constexpr int kBStages = 2;
  static constexpr int kSlots = kRT == 8 ? 5 : kRT == 4 ? 3 : 4;  // y slots of 16 KB
  static constexpr int kMinBlocks = kRT == 8 ? 1 : 2;
  static constexpr int kSmem =
      kUBlocks * kBlock + kBStages * kBStage + kSlots * kBlock + 1024;
  // with the static part (the tile map) and 1 KB that the system keeps
  static_assert(kMinBlocks * (kSmem + static_cast<int>(sizeof(TileMap)) + 256 + 1024) <=
                    228 * 1024,
                "blocks per SM");
};

template <int kRT>
__global__ void __launch_bounds__(kExpandThreads, ExpandShape<kRT>::kMinBlocks)
    lora_expand_tiles_kernel(const __grid_constant__ CUtensorMap tmap_b, const Args p) {
  using S = ExpandShape<kRT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* u_s = smem;
  uint8_t* b_s = u_s + S::kUBlocks * kBlock;
  uint8_t* y_s = b_s + S::kBStages * S::kBStage;
  __shared__ TileMap map;
  __shared__ __align__(8) uint64_t bars[2 * S::kBStages + 5];
  __shared__ uint32_t tmem_holder;
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto b_full = [&](int s) { return bar0 + 8u * s; };
  auto b_empty = [&](int s) { return bar0 + 8u * (S::kBStages + s); };
  auto t_full = [&](int h) { return bar0 + 8u * (2 * S::kBStages + h); };
  auto t_empty = [&](int h) { return bar0 + 8u * (2 * S::kBStages + 2 + h); };
  const uint32_t u_full = bar0 + 8u * (2 * S::kBStages + 4);
  const int warp = threadIdx.x / 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kBStages; ++s) {
      ptx::mbar_init(b_full(s), 1);
      ptx::mbar_init(b_empty(s), 1);
    }
    for (int h = 0; h < 2; ++h) {
      ptx::mbar_init(t_full(h), 1);
      ptx::mbar_init(t_empty(h), 128);
    }
    ptx::mbar_init(u_full, 128);
    ptx::fence_barrier_init();
    ptx::prefetch_tmap(&tmap_b);
  }
  if (warp == 4) {
    ptx::tmem_alloc(ptx::smem_u32(&tmem_holder), 2 * kCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  // The launch before this one is the shrink, whose blocks have all waited
  // for the work before it: offsets, order, B and y are final, u is not yet.
  map.build<kExpandThreads>(p.offsets, p.M, p.L, kRows);
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_holder);
  const int groups = p.L + p.copy_rest;
  const int chunks = (p.N + kCols - 1) / kCols;
  const int64_t total = static_cast<int64_t>(map.before[groups]) * chunks;
  int64_t at = total * blockIdx.x / gridDim.x;
  const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
  bool ok = true, waited = false;
  uint32_t n_used = 0;   // chunks multiplied so far: B stage, half of tensor memory
  uint32_t u_phase = 0;

  while (at < end) {
    const int t = static_cast<int>(at / chunks);
    const int c0 = static_cast<int>(at - static_cast<int64_t>(t) * chunks);
    const int n = static_cast<int>(end - at < chunks - c0 ? end - at : chunks - c0);
    at += n;
    const Tile tile = map.find(t, groups, kRows);
    const bool rest = tile.group == p.L;  // rows without an adapter: out = y
    if (warp < 4) {
      const int cc = threadIdx.x % 8, r0 = threadIdx.x / 8;  // 16-byte chunk, first of 8 rows
      int64_t off[8];
      unsigned live = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        const int row = r < tile.rows ? p.order[tile.pos + r] : -1;
        const bool in = row >= 0 && row < p.M;
        live |= static_cast<unsigned>(in) << i;
        off[i] = static_cast<int64_t>(in ? row : 0) * p.N + c0 * kCols + cc * 8;
      }
      const uint32_t mine = cell(r0, cc);
      const int col0 = c0 * kCols + cc * 8;
      auto fetch = [&](int i) {  // y of chunk c0 + i
        if (i < n && col0 + i * kCols < p.N) {
          const uint32_t dst = ptx::smem_u32(y_s) + (i % S::kSlots) * kBlock + mine;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (live >> j & 1) ptx::cp_async16(dst + j * 2048, p.y + off[j] + i * kCols, true);
        }
        ptx::cp_async_commit();
      };
      constexpr int kAhead = S::kSlots - 1;
      for (int i = 0; i < kAhead; ++i) fetch(i);

      if (!waited) {
        ptx::grid_dep_wait();
        ptx::grid_dep_launch();
        waited = true;
      }
      if (!rest) {
        // u of the tile, [hi | lo] as the shrink left it.  The MMAs that read
        // the last tile's u are done: their results were read.
        constexpr int kChunks = S::RP / 4;  // 16-byte chunks of a row
        const __nv_bfloat16* up = p.u + static_cast<int64_t>(tile.pos) * (2 * S::RP);
#pragma unroll 8
        for (int i = 0; i < kChunks; ++i) {
          const int f = i * 128 + threadIdx.x, r = f / kChunks, c = f % kChunks;
          const bool in = r < tile.rows;
          ptx::cp_async16(ptx::smem_u32(u_s) + (c / 8) * kBlock + cell(r, c % 8),
                          up + (in ? f * 8 : 0), in);
        }
        ptx::cp_async_commit();
        ptx::cp_async_wait<0>();
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(u_full);
      }

      const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
      for (int i = 0; i < n; ++i) {
        fetch(i + kAhead);
        ptx::cp_async_wait<kAhead>();
        uint8_t* slot = y_s + (i % S::kSlots) * kBlock;
        if (!rest) {
          const uint32_t h = (n_used + i) & 1u;
          if (ok && !ptx::mbar_wait(t_full(h), ((n_used + i) >> 1) & 1u)) {
            record_error(p.err, kErrTimeoutEpilogue);
            ok = false;
          }
          ptx::tc_fence_after();
          uint32_t a0[32], a1[32];
          ptx::tmem_ld_32x32b_x32(lane_base + h * kCols, a0);
          ptx::tmem_ld_32x32b_x32(lane_base + h * kCols + 32, a1);
          ptx::tmem_ld_wait();
          ptx::tc_fence_before();
          ptx::mbar_arrive(t_empty(h));
          ptx::named_barrier_sync(1, 128);  // everyone's y has landed
          const int r = threadIdx.x;
          uint4 v8[8];  // all reads before the writes that might alias them
#pragma unroll
          for (int c = 0; c < 8; ++c) v8[c] = *reinterpret_cast<const uint4*>(slot + cell(r, c));
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint4* q = reinterpret_cast<uint4*>(slot + cell(r, c));
            const uint4 v = v8[c];
            auto f = [&](int k) {
              const int e = c * 8 + k;
              return __uint_as_float(e < 32 ? a0[e & 31] : a1[e & 31]);
            };
            *q = make_uint4(lora::add2(v.x, f(0), f(1)), lora::add2(v.y, f(2), f(3)),
                            lora::add2(v.z, f(4), f(5)), lora::add2(v.w, f(6), f(7)));
          }
          ptx::named_barrier_sync(1, 128);  // the slot holds out
        }
        // the cells this thread copied in are the ones it copies out, so the
        // next copy into the slot needs no barrier
        if (col0 + i * kCols < p.N) {
          uint4 o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            o[j] = *reinterpret_cast<const uint4*>(slot + mine + j * 2048);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (live >> j & 1) *reinterpret_cast<uint4*>(p.out + off[j] + i * kCols) = o[j];
        }
      }
    } else if (warp == 4 && !rest) {
      if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(u_full, u_phase));
      for (int i = 0; i < n && ok; ++i) {
        const uint32_t u = n_used + i, h = u & 1u;
        const int s = u % S::kBStages;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(b_full(s), (u / S::kBStages) & 1u) &&
                                         ptx::mbar_wait(t_empty(h), ((u >> 1) & 1u) ^ 1u));
        if (!ok) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint32_t ub = ptx::smem_u32(u_s), bb = ptx::smem_u32(b_s) + s * S::kBStage;
#pragma unroll
          for (int k = 0; k < 2 * kRT; ++k) {
            const int kb = k % kRT;  // the lo half meets the same B again
            ptx::mma_f16(tmem + h * kCols,
                         ptx::sdesc_kmajor_sw128(ub + (k / 4) * kBlock + (k % 4) * 32),
                         ptx::sdesc_kmajor_sw128(bb + (kb / 4) * kCols * 128 + (kb % 4) * 32),
                         ptx::idesc_bf16_f32(kRows, kCols), k != 0 ? 1u : 0u);
          }
          ptx::mma_commit(b_empty(s));
          ptx::mma_commit(t_full(h));
        }
        __syncwarp();
      }
      if (!ok && threadIdx.x % 32 == 0) record_error(p.err, kErrTimeoutMma);
    } else if (warp == 5 && !rest && threadIdx.x % 32 == 0) {
      for (int i = 0; i < n && ok; ++i) {
        const uint32_t u = n_used + i;
        const int s = u % S::kBStages;
        if (!ptx::mbar_wait(b_empty(s), ((u / S::kBStages) & 1u) ^ 1u)) {
          record_error(p.err, kErrTimeoutProducer);
          ok = false;
          break;
        }
        ptx::mbar_arrive_expect_tx(b_full(s), S::kBStage);
#pragma unroll
        for (int k = 0; k < S::kBBlocks; ++k)
          ptx::tma_load_2d(ptx::smem_u32(b_s) + s * S::kBStage + k * kCols * 128, &tmap_b,
                           b_full(s), k * 128, tile.group * p.N + (c0 + i) * kCols);
      }
    }
    if (!rest) {
      n_used += n;
      u_phase ^= 1;
    }
  }
  if (!waited) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
  }
  // What is still on its way when a wait ran out lands before the block ends.
  if (warp == 5 && threadIdx.x % 32 == 0)
    for (uint32_t i = 0; i < S::kBStages && i < n_used; ++i) {
      const uint32_t u = n_used - 1 - i;
      if (!ptx::mbar_wait(b_full(u % S::kBStages), (u / S::kBStages) & 1u)) break;
    }
  ptx::cp_async_wait<0>();
  ptx::tc_fence_before();
  __syncthreads();  // the epilogue has read what the last MMAs wrote
  if (warp == 4) ptx::tmem_dealloc(tmem, 2 * kCols);
}

// ------------------------------------------------------------------- host

template <typename Kernel, typename... Ts>
cudaError_t launch_pdl(Kernel k, int blocks, int threads, size_t smem, int cluster,
                       cudaStream_t st, const Ts&... args) {
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
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

template <int kRT>
cudaError_t launch_rank(const Args& a, const lora::Plan& pl, cudaStream_t st) {
  static std::once_flag once[kMaxDevices];
  static cudaError_t status[kMaxDevices];
  cudaError_t e = once_per_device(once, status, [](int) {
    const cudaError_t f = cudaFuncSetAttribute(lora_shrink_tiles_kernel<kRT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               ShrinkShape<kRT>::kSmem);
    if (f != cudaSuccess) return f;
    return cudaFuncSetAttribute(lora_expand_tiles_kernel<kRT>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                ExpandShape<kRT>::kSmem);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap tb;
  if (!make_tmap_u8(&tb, a.b, static_cast<uint64_t>(a.L) * a.N, static_cast<uint64_t>(a.R) * 2,
                    kCols, 128))
    return cudaErrorInvalidValue;
  e = launch_pdl(lora_shrink_tiles_kernel<kRT>, pl.shrink_blocks, kShrinkThreads,
                 ShrinkShape<kRT>::kSmem, pl.max_splits, st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(lora_expand_tiles_kernel<kRT>, pl.expand_blocks, kExpandThreads,
                    ExpandShape<kRT>::kSmem, 1, st, tb, a);
}

}  // namespace

namespace lora {

Plan plan_tiles(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L, int sm_count) {
  Plan p;
  p.rt = rank_tiles(R);
  const int64_t least = (M + kRows - 1) / kRows, most = M / kRows + (L + 1 < M ? L + 1 : M);
  // Blocks of a cluster: as many as keep the tiles that are likely (full ones
  // and a partial one for each adapter) resident at once, two blocks per SM,
  // with at least 256 of K each.
  const int64_t likely = least + (L < least ? L : least);
  // (Clusters of 7 in place of 4 made 36 tiles of K = 4096 slower: 121 -> 126 us.)
  p.max_splits = 1;
  while (p.max_splits < 8 && likely * p.max_splits * 2 <= 2 * sm_count &&
         K >= 512 * static_cast<int64_t>(p.max_splits))
    p.max_splits *= 2;
  const int64_t clusters = 2 * sm_count / p.max_splits;
  p.shrink_blocks = static_cast<int>((most < clusters ? most : clusters) * p.max_splits);
  const int64_t eb = most * ((N + kCols - 1) / kCols), er = sm_count * (p.rt == 8 ? 1 : 2);
  p.expand_blocks = static_cast<int>(eb < er ? eb : er);
  p.u_bytes = static_cast<size_t>(M) * 16 * p.rt * 4;  // [hi | lo] in bf16
  return p;
}

cudaError_t launch_tiles(const Args& a, const Plan& pl, cudaStream_t st) {
  switch (pl.rt) {
    case 1: return launch_rank<1>(a, pl, st);
    case 2: return launch_rank<2>(a, pl, st);
    case 4: return launch_rank<4>(a, pl, st);
    default: return launch_rank<8>(a, pl, st);
  }
}

}  // namespace lora
}  // namespace fp8bl
