// Low-rank adapters for long batches (prompts): the same two products as
// lora.cu in tiles of 128 sorted rows on the tensor core (tcgen05, bf16 in,
// fp32 in tensor memory).
//
// Shrink, u = x A^T: bound by reading x.  64-deep slices of the tile's rows and
// of A come into a ring of 128-byte-swizzled shared-memory stages, by TMA where
// a full tile's rows are one piece of memory (a request's are), else by cp.async
// of 128 threads from wherever `order` says; one thread issues the MMAs.  K is
// split over the blocks of a cluster so that all SMs have work; the blocks'
// sums meet through distributed shared memory, added in the order of the parts,
// and leave as two bf16 terms side by side ([hi | lo], 2 RP deep).  (Parts that
// the expand adds up instead cost 38 of 137 us beside 28672 x 4096 at rank 64
// and 4096 rows: every block of the expand read all seven.)
//
// Expand, out = y + s u B^T: bound by reading y and writing out.  One
// accumulation over hi and lo with B read twice multiplies by all 16 bits of
// u.  Work is numbered in chunks of 64 columns, tile after tile, and every block
// takes an equal run of chunks, or blocks share tiles evenly where that works
// out.  Of a chunk, B comes by TMA, the MMAs run into one of two halves of
// tensor memory, and y streams through a ring of shared-memory
// slots: in by TMA (full tiles of one piece) or cp.async (8 lanes per 128-byte
// row piece), the accumulator added row by row (a thread per row, as tensor
// memory hands it out) and written back, and out again the same way.
//
// 4096 rows of 8 adapters of rank 64 beside 28672 x 4096: 109 to 121 us by how
// the rows fall to the adapters, for 537 MB (75 to 68% of the copy rate): about 15
// us of shrink, then 5.5 TB/s of y and out, whose row pieces of 128 bytes lie N
// apart.  5003 rows at rank 16 beside 4096 x 14336: 56 to 58 us for 227 MB.  Alone
// and from memory its shrink takes 37 us for 145 MB and its expand 26 for 82: ten
// chunks a block are mostly the way in and out (DRAM 21%, issue 33%).
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

// The tile's first row if its rows follow one another in memory too (a request
// in one piece), else -1.  Whole warp.
__device__ __forceinline__ int first_of_run(const Args& p, const Tile& tile) {
  const int lane = threadIdx.x % 32, first = p.order[tile.pos];
  bool run = first >= 0 && first <= p.M - tile.rows;
#pragma unroll
  for (int i = 0; i < kRows / 32; ++i) {
    const int r = i * 32 + lane;
    run = run && (r >= tile.rows || p.order[tile.pos + r] == first + r);
  }
  return __all_sync(0xffffffffu, run) ? first : -1;
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
__global__ void __launch_bounds__(kShrinkThreads, 2)
    lora_shrink_tiles_kernel(const __grid_constant__ CUtensorMap tmap_x,
                             const __grid_constant__ CUtensorMap tmap_a, const Args p) {
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
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 1);
    }
    ptx::mbar_init(done, 1);
    ptx::fence_barrier_init();
    ptx::prefetch_tmap(&tmap_x);
    ptx::prefetch_tmap(&tmap_a);
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
      auto wait_empty = [&](uint32_t u) {
        if (ok && !ptx::mbar_wait(empty(u % S::kStages), ((u / S::kStages) & 1u) ^ 1u)) {
          record_error(p.err, kErrTimeoutProducer);
          ok = false;
        }
      };
      const int first = tile.rows == kRows ? first_of_run(p, tile) : -1;
      if (first >= 0) {
        // A full tile of rows in one piece: TMA.  It may bring ranks behind R,
        // of the next adapter: their sums are not used.
        if (threadIdx.x == 0)
          for (int i = 0; i < n && ok; ++i) {
            const uint32_t u = n_used + i;
            const int s = u % S::kStages, k = (k0 + i) * kDeep * 2;
            wait_empty(u);
            if (!ok) break;
            ptx::mbar_arrive_expect_tx(full(s), S::kStage);
            ptx::tma_load_2d(base + s * S::kStage, &tmap_x, full(s), k, first);
            ptx::tma_load_2d(base + s * S::kStage + kBlock, &tmap_a, full(s), k,
                             tile.group * p.R);
          }
        __syncwarp();
      } else {
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
            wait_empty(u);
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
            // everyone's copies have landed and are visible to the tensor core
            ptx::cp_async_wait<S::kAhead>();
            ptx::fence_proxy_async_smem();
            ptx::named_barrier_sync(1, 128);
            if (threadIdx.x == 0) ptx::mbar_arrive(full((n_used + i - S::kAhead) % S::kStages));
          }
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
      // TMA may write the next item over the sums, which this thread wrote into
      // its own ring and read from the others'
      ptx::fence_proxy_async_cluster();
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
// 4 epilogue warps, one for the copies of B and the MMAs, one for the copies of
// y and out (with a seventh, registers would be granted as for eight, 128 each)
constexpr int kMmaWarp = 4, kYWarp = 5, kExpandThreads = 192;

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
    lora_expand_tiles_kernel(const __grid_constant__ CUtensorMap tmap_b,
                             const __grid_constant__ CUtensorMap tmap_y,
                             const __grid_constant__ CUtensorMap tmap_out, const Args p) {
  using S = ExpandShape<kRT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* u_s = smem;
  uint8_t* b_s = u_s + S::kUBlocks * kBlock;
  uint8_t* y_s = b_s + S::kBStages * S::kBStage;
  __shared__ TileMap map;
  __shared__ __align__(8) uint64_t bars[2 * S::kBStages + 7 + 2 * S::kSlots];
  __shared__ uint32_t tmem_holder;
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto b_full = [&](int s) { return bar0 + 8u * s; };
  auto b_empty = [&](int s) { return bar0 + 8u * (S::kBStages + s); };
  auto t_full = [&](int h) { return bar0 + 8u * (2 * S::kBStages + h); };
  auto t_empty = [&](int h) { return bar0 + 8u * (2 * S::kBStages + 2 + h); };
  const uint32_t u_full = bar0 + 8u * (2 * S::kBStages + 4);
  const uint32_t run_done = u_full + 8u;  // the epilogue is through with a run's slots
  auto y_full = [&](int k) { return run_done + 8u * (1 + k); };
  auto y_ready = [&](int k) { return run_done + 8u * (1 + S::kSlots + k); };  // holds out
  // the copies' warp has seen the run before end and stored this run's slots
  const uint32_t y_idle = run_done + 8u * (1 + 2 * S::kSlots);
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
    ptx::mbar_init(run_done, 1);
    for (int k = 0; k < S::kSlots; ++k) {
      ptx::mbar_init(y_full(k), 1);
      ptx::mbar_init(y_ready(k), 128);
    }
    ptx::mbar_init(y_idle, 1);
    ptx::fence_barrier_init();
    ptx::prefetch_tmap(&tmap_b);
    ptx::prefetch_tmap(&tmap_y);
    ptx::prefetch_tmap(&tmap_out);
  }
  if (warp == kMmaWarp) {
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
  int64_t end = total * (blockIdx.x + 1) / gridDim.x;
  // Where the tiles go into the blocks with little left over, `team` blocks
  // share a tile and take its chunks in turn: what they read and write at one
  // time lies side by side in every row (112 against 118 us for 4096 rows beside
  // 28672 x 4096; with 15% of the blocks left over it loses).
  const int all_tiles = map.before[groups];
  int team = all_tiles > 0 ? static_cast<int>(gridDim.x) / all_tiles : 0;
  if (team > chunks) team = chunks;
  if (10 * static_cast<int64_t>(team) * all_tiles < 9 * static_cast<int64_t>(gridDim.x)) team = 0;
  if (team > 0) {
    at = blockIdx.x;
    end = static_cast<int>(blockIdx.x) < team * all_tiles ? at + 1 : at;
  }
  const int every = team > 0 ? team : 1;  // chunks from one of a block to its next
  bool ok = true, waited = false;
  uint32_t n_used = 0;   // chunks multiplied so far: B stage, half of tensor memory
  uint32_t u_phase = 0, runs = 0;
  uint32_t b_loads = 0;  // copies of B that were started
  uint32_t y_used = 0;   // chunks of y that came by TMA: slot and phase

  while (at < end) {
    int t, c0, n;
    if (team > 0) {
      t = blockIdx.x / team, c0 = blockIdx.x % team;
      n = (chunks - c0 + team - 1) / team;
      at = end;
    } else {
      t = static_cast<int>(at / chunks);
      c0 = static_cast<int>(at - static_cast<int64_t>(t) * chunks);
      n = static_cast<int>(end - at < chunks - c0 ? end - at : chunks - c0);
      at += n;
    }
    const Tile tile = map.find(t, groups, kRows);
    const bool rest = tile.group == p.L;  // rows without an adapter: out = y
    // A full tile of rows in one piece comes and goes by TMA.
    const int first = rest || tile.rows < kRows ? -1 : first_of_run(p, tile);
    const bool full = first >= 0;
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
        if (i < n && col0 + i * every * kCols < p.N) {
          const uint32_t dst = ptx::smem_u32(y_s) + (i % S::kSlots) * kBlock + mine;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (live >> j & 1) ptx::cp_async16(dst + j * 2048, p.y + off[j] + i * every * kCols, true);
        }
        ptx::cp_async_commit();
      };
      constexpr int kAhead = S::kSlots - 1;
      if (!full)
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
      // adds the accumulator of chunk i to this thread's row of a slot
      auto add = [&](int i, uint8_t* slot) {
        const uint32_t u = n_used + i, h = u & 1u;
        if (ok && !ptx::mbar_wait(t_full(h), (u >> 1) & 1u)) {
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
        if (!full) ptx::named_barrier_sync(1, 128);  // everyone's y has landed
        const int r = threadIdx.x;
        uint4 v[8];  // all reads before the writes that might alias them
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = *reinterpret_cast<const uint4*>(slot + cell(r, c));
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          auto f = [&](int k) {
            const int e = c * 8 + k;
            return __uint_as_float(e < 32 ? a0[e & 31] : a1[e & 31]);
          };
          *reinterpret_cast<uint4*>(slot + cell(r, c)) =
              make_uint4(lora::add2(v[c].x, f(0), f(1)), lora::add2(v[c].y, f(2), f(3)),
                         lora::add2(v[c].z, f(4), f(5)), lora::add2(v[c].w, f(6), f(7)));
        }
      };
      if (full) {
        for (int i = 0; i < n; ++i) {
          const uint32_t v = y_used + i;
          const int k = v % S::kSlots;
          if (ok && !ptx::mbar_wait(y_full(k), (v / S::kSlots) & 1u)) {
            record_error(p.err, kErrTimeoutEpilogue);
            ok = false;
          }
          add(i, y_s + k * kBlock);
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(y_ready(k));
        }
      } else {
        for (int i = 0; i < n; ++i) {
          fetch(i + kAhead);
          ptx::cp_async_wait<kAhead>();
          uint8_t* slot = y_s + (i % S::kSlots) * kBlock;
          if (!rest) {
            add(i, slot);
            ptx::named_barrier_sync(1, 128);  // the slot holds out
          }
          // the cells this thread copied in are the ones it copies out, so the
          // next copy into the slot needs no barrier
          if (col0 + i * every * kCols < p.N) {
            uint4 o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              o[j] = *reinterpret_cast<const uint4*>(slot + mine + j * 2048);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (live >> j & 1) *reinterpret_cast<uint4*>(p.out + off[j] + i * every * kCols) = o[j];
          }
        }
      }
      // The next run's plain copies may use any slot.  After every run, so that
      // run_done is at most one phase ahead of the warp that waits for it.
      if (!rest && ok && !ptx::mbar_wait(y_idle, runs & 1u)) {
        record_error(p.err, kErrTimeoutEpilogue);
        ok = false;
      }
      ptx::fence_proxy_async_smem();  // the next run's TMA may write any slot
      ptx::named_barrier_sync(1, 128);  // everyone is through with the run
      if (threadIdx.x == 0) ptx::mbar_arrive(run_done);
    } else if (warp == kMmaWarp && !rest) {
      // B of chunk i of the run, into the stage that chunk i - kBStages left
      auto load_b = [&](int i) {
        if (i >= n || !ok) return;
        const uint32_t u = n_used + i;
        const int s = u % S::kBStages;
        ok = __all_sync(0xffffffffu,
                        ptx::mbar_wait(b_empty(s), ((u / S::kBStages) & 1u) ^ 1u));
        if (!ok) return;
        if (ptx::elect_one()) {
          ptx::mbar_arrive_expect_tx(b_full(s), S::kBStage);
#pragma unroll
          for (int k = 0; k < S::kBBlocks; ++k)
            ptx::tma_load_2d(ptx::smem_u32(b_s) + s * S::kBStage + k * kCols * 128, &tmap_b,
                             b_full(s), k * 128,
                             tile.group * p.N + (c0 + i * every) * kCols);
        }
        __syncwarp();
        b_loads = u + 1;
      };
      for (int i = 0; i < S::kBStages; ++i) load_b(i);
      if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(u_full, u_phase));
      for (int i = 0; i < n && ok; ++i) {
        // the MMAs of chunk i - 1 are done by now, or soon
        if (i > 0) load_b(i - 1 + S::kBStages);
        const uint32_t u = n_used + i, h = u & 1u;
        const int s = u % S::kBStages;
        ok = ok && __all_sync(0xffffffffu, ptx::mbar_wait(b_full(s), (u / S::kBStages) & 1u) &&
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
    } else if (warp == kYWarp && !rest && threadIdx.x % 32 == 0) {
      // One thread takes a slot from its load to its store and to the next
      // load.  A run starts when the epilogue is through with the one before:
      // its slots may be in use by plain copies.  (Rows without an adapter come
      // last, so every earlier run has passed here, and the phases are waited
      // for one by one: the epilogue does not end a run before this thread has
      // seen the end of the one before.)
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok && !ptx::mbar_wait(bar, parity)) {
          record_error(p.err, kErrTimeoutProducer);
          ok = false;
        }
      };
      if (runs > 0) wait(run_done, (runs - 1) & 1u);
      if (full && ok) {
        auto load = [&](int i) {
          if (i >= n) return;
          const int k = (y_used + i) % S::kSlots;
          ptx::mbar_arrive_expect_tx(y_full(k), kBlock);
          ptx::tma_load_2d(ptx::smem_u32(y_s) + k * kBlock, &tmap_y, y_full(k),
                           (c0 + i * every) * kCols * 2, first);
        };
        for (int i = 0; i < S::kSlots; ++i) load(i);
        for (int i = 0; i < n && ok; ++i) {
          const uint32_t v = y_used + i;
          const int k = v % S::kSlots;
          wait(y_ready(k), (v / S::kSlots) & 1u);
          if (!ok) break;
          ptx::tma_store_2d(&tmap_out, ptx::smem_u32(y_s) + k * kBlock, (c0 + i * every) * kCols * 2,
                            first);
          ptx::bulk_commit_group();
          ptx::bulk_wait_group_read<0>();
          load(i + S::kSlots);
        }
      }
      ptx::mbar_arrive(y_idle);
    }
    ++runs;
    if (full) y_used += n;
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
  if (warp == kMmaWarp && threadIdx.x % 32 == 0)
    for (uint32_t i = 0; i < S::kBStages && i < b_loads; ++i) {
      const uint32_t u = b_loads - 1 - i;
      if (!ptx::mbar_wait(b_full(u % S::kBStages), (u / S::kBStages) & 1u)) break;
    }
  if (warp == kYWarp && threadIdx.x % 32 == 0) {
    for (uint32_t i = 0; i < S::kSlots && i < y_used; ++i) {
      const uint32_t v = y_used - 1 - i;
      if (!ptx::mbar_wait(y_full(v % S::kSlots), (v / S::kSlots) & 1u)) break;
    }
    ptx::bulk_wait_group<0>();
  }
  ptx::cp_async_wait<0>();
  ptx::tc_fence_before();
  __syncthreads();  // the epilogue has read what the last MMAs wrote
  if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, 2 * kCols);
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
  // 128-byte pieces of rows: of x and A along K, of B along the rank, of y and
  // out along N
  const uint64_t M = a.M, N = a.N, K = a.K, R = a.R, L = a.L;
  CUtensorMap tx, ta, tb, ty, to;
  if (!make_tmap_u8(&tx, a.x, M, K * 2, kRows, 128) ||
      !make_tmap_u8(&ta, a.a, L * R, K * 2, 16 * kRT, 128) ||
      !make_tmap_u8(&tb, a.b, L * N, R * 2, kCols, 128) ||
      !make_tmap_u8(&ty, a.y, M, N * 2, kRows, 128) ||
      !make_tmap_u8(&to, a.out, M, N * 2, kRows, 128))
    return cudaErrorInvalidValue;
  e = launch_pdl(lora_shrink_tiles_kernel<kRT>, pl.shrink_blocks, kShrinkThreads,
                 ShrinkShape<kRT>::kSmem, pl.max_splits, st, tx, ta, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(lora_expand_tiles_kernel<kRT>, pl.expand_blocks, kExpandThreads,
                    ExpandShape<kRT>::kSmem, 1, st, tb, ty, to, a);
}

}  // namespace

namespace lora {

Plan plan_tiles(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L, int sm_count) {
  Plan p;
  p.rt = rank_tiles(R);
  const int64_t least = (M + kRows - 1) / kRows, most = M / kRows + (L + 1 < M ? L + 1 : M);
  // Blocks of a cluster: as many as keep the tiles that are likely (full ones
  // and a partial one for each adapter) resident at once, two blocks per SM,
  // with at least 256 of K each.  A cluster lies within one group of SMs, so of
  // all blocks' places pairs can use all, clusters of 4 15/16 and others 5/6.
  // Measured with every size at 28 to 150 tiles, K = 4096, 7168 and 14336, rank 16
  // and 64, N = 4096: 8 blocks pay up to 32 tiles, 7 up to 36, 6 to 42, 5 to 49, 4 to
  // 70, 3 to 85 and 2 to 148, at every K alike; the largest that fits is within 4% of the
  // best, one that does not loses 10 to 25%.  us at rank 16, K = 4096 | 14336:
  //   34 tiles   6 blocks 29 | 47     7 28 | 46     8 33 | 58
  //   53         3 44 | 69            4 43 | 68     5 48 | 79
  //   80         2 58 | 99            3 58 | 93     4 65 | 111
  //   100        1 74 | 144           2 67 | 113    3 77 | 135
  const int64_t likely = least + (L < least ? L : least), places = 2 * sm_count;
  p.max_splits = 1;
  for (int s = 2; s <= 8; ++s) {
    const int64_t fit = s == 2 ? places : s == 4 ? places * 15 / 16 : places * 5 / 6;
    if (likely * s <= fit && K >= 256 * s) p.max_splits = s;
  }
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
