// int8_product.cuh -- the grouped products of int8 rows and weights, on tcgen05.
//
//   z[r, n] = xs[r] ws[n] sum_k x[r, k] w[n, k]
//
// tcgen05 has no integer products on sm_103, so the codes become fp16 on their way: a
// code is a whole number of 8 bits, which fp16 holds exactly, as it does the products
// in fp32 (sums are rounded where they pass 2^24).  Between the copies and the products
// stand eight warps that read 128-byte slices of codes.  The weights' go to tensor memory
// as fp16, the rows' to shared memory.
//
// A block makes tiles of its own: 256 features (two halves, each the 128 rows of an A
// operand and an accumulator; one half where tiles are few) by up to 192 columns, rows of
// x.  In pairs of SMs each would convert and read half of the rows, but a pair's product may
// start only when both blocks' codes are written, and a release that orders them across
// the blocks takes longer than the conversion of a slice (one expert, 8191 rows, 4096 ->
// 4096: 343 us; with tiles of 128 columns and twice the stages 320).
// 64 codes deep and 176 columns wide a tile takes 1090 cycles, 700 of products.  No unit is at
// its limit (4096 rows of that layer: tensor pipe 39% of the time, issue slots 50, shared
// memory's pipe 38), but a stage's way from the converting warps to its products and back
// takes two stages' time, and tensor memory has room for no more.  Beyond 96 columns it has none either for two tiles'
// accumulators, and the products wait for a tile's results: 60 us of that layer's with
// gelu and residual.
// On GB300, us: that layer 249 (1.10 PFLOP/s); 8 experts, 8192 rows, 14336 -> 4096 750 (1.28);
// 128 experts, 512 rows by a Zipf law, gated, 2048 -> 2 x 768 71; 256 experts, 32768 rows,
// 2048 -> 7168 1301.
//   warps 0-7    epilogue: tensor memory -> registers, scaled -> shared -> rows
//   warps 8-15   codes -> fp16
//   warp 16      TMA producer: 128 codes deep
//   warp 17      tcgen05.mma issue, tensor memory allocation
//   warps 18-19  fill up a warpgroup (setmaxnreg)
#pragma once

#include "quant_product.cuh"

namespace moe {
namespace experts {

constexpr int kRawSlice = 128;     // codes of a raw stage
constexpr int kMostRaw = 4;        // raw stages
constexpr int kMostWide = 4;       // stages of fp16, 64 deep
constexpr int kWideColumns = kSlice / 2;  // of tensor memory, for 128 rows of A
constexpr int kOverlapped = 96;    // columns up to which the accumulators of two tiles fit beside A
constexpr int kInt8Widest = 4;     // of cap_of: columns of a tile at most
constexpr int kInt8Columns = kMaxN - 16 * kInt8Widest;
constexpr int kInt8DataBytes = 192 * 1024;  // of stages
constexpr int kInt8Threads = 640;
// Registers of a thread, and whether the weights' codes are converted ahead of the wait for
// room, which takes 16 more: linear products in two halves, whose tiles of more than 160
// columns have two stages (one expert, 8191 rows, 4096 -> 4096 262 -> 248 us; gated ones, whose
// epilogue needs the registers, 141 -> 144 at 16 experts, 12288 rows, 2048 -> 2 x 1408).
template <int kUse, int kHalves>
struct Int8Registers {
  static constexpr bool kEarly = kUse == kForward && kHalves == 2;
  static constexpr int kEpilogue = kEarly ? 120 : 128, kConvert = kEarly ? 88 : 80, kOther = 64;
  static constexpr int kLaunch = 65536 / kInt8Threads / 8 * 8;
  static_assert(2 * kEpilogue + 2 * kConvert + kOther <= 5 * kLaunch, "what the block has");
  static_assert(kEpilogue >= kLaunch && kConvert <= kLaunch && kOther <= kLaunch,
                "setmaxnreg.inc gives no fewer than a thread has, .dec no more");
};

// Dynamic shared memory: stages (1024-byte aligned), staging, then each expert's rows and
// its first tile.
inline size_t int8_product_smem(int E) {
  return 1024 + kInt8DataBytes + kStagingBytes + static_cast<size_t>(E) * 12 + 4;
}
static_assert(1024 + kInt8DataBytes + kStagingBytes + MOE_MAX_LOCAL_EXPERTS * 12 + 4 + 1024 <=
                  227 * 1024,
              "shared memory of one block");

// Whether tiles have two halves, of which there would be `tiles`: unless tiles of one, twice
// as many, are one wave.  us, one half / two: 1 expert, 4096 -> 4096, 64 rows 20 / 36, 512 34 /
// 36, 768 37 / 41, 1024 60 / 43; 2048 -> 7168, 384 rows 23 / 24, 512 32 / 27; 10 experts, 1456 ->
// 1000, 1540 rows 18.8 / 19.2, 3000 27 / 21; 8 experts, 4096 -> 4096, 80 rows 56 / 43.
inline bool int8_two_halves(int64_t tiles, int sms) { return 2 * tiles > sms; }

// What tiles of `cap` columns cost, in cycles over 3: 64 codes deep they take about 600 cycles
// (one half 300) and 3 for each column, and beside that 3000, or 12000 where the products wait
// for the results.  Among equals the narrowest, which have more stages.  (128 experts, 512
// rows by a Zipf law, gated, 2048 -> 2 x 768: 70 us, 79 with 192 always.)
template <int kHalves>
__device__ __forceinline__ float int8_cap_cost(int cap, int blocks, int rows, int m_blocks,
                                               int slices, int workers) {
  const int64_t waves = (static_cast<int64_t>(blocks) * m_blocks + workers - 1) / workers;
  const float columns = static_cast<float>(rows) / static_cast<float>(max(blocks, 1));
  const float slice = 100.f * kHalves + columns + static_cast<float>(cap) * 0.05f;
  const float tile = kHalves == 2 && cap > kOverlapped ? 3600.f : 1700.f;
  return static_cast<float>(waves) * (static_cast<float>(slices) * slice + tile);
}

// How a block's memory is divided, for tiles of `cap` columns.  Tensor memory: accumulators
// of one half each, of two tiles where those of two halves are narrow; the rest stages of A.
template <int kHalves>
struct Int8Shape {
  int columns;                      // of an accumulator
  int slots, wide, raw;             // accumulators, stages of fp16, raw stages
  uint32_t wide_bytes, raw_bytes;   // of a stage, in shared memory
  __device__ __forceinline__ explicit Int8Shape(int cap) {
    constexpr int kA = kHalves * kWideColumns;
    columns = (cap + 31) / 32 * 32;
    slots = columns <= kOverlapped ? 2 * kHalves : 2;
    wide = min(kMostWide, (512 - slots * columns) / kA);
    wide_bytes = columns * kSlice * 2;
    raw_bytes = kHalves * kTileABytes + (cap + 63) / 64 * kBoxBytes;
    raw = min(kMostRaw, static_cast<int>((kInt8DataBytes - wide * wide_bytes) / raw_bytes));
  }
};

// A place in a ring of `size`, and the parity of the pass through it.
struct Int8Ring {
  int at;
  uint32_t pass;
  __device__ __forceinline__ void advance(int size, int by = 1) {
    at += by;
    if (at >= size) at -= size, pass ^= 1;
  }
  __device__ __forceinline__ void back(int size) {
    if (at == 0) at = size, pass ^= 1;
    --at;
  }
};

// 4 codes as fp16.  With the sign bit flipped a byte is the code + 128; behind the high
// byte 0x64 it is the fp16 number 1024 + that.
__device__ __forceinline__ uint2 codes_to_fp16(uint32_t c) {
  const uint32_t u = c ^ 0x80808080u;
  const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 base = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), base);
  const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), base);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// 16 codes as fp16.
struct Wide16 {
  uint2 v[4];
  Wide16() = default;
  __device__ __forceinline__ explicit Wide16(uint4 c)
      : v{codes_to_fp16(c.x), codes_to_fp16(c.y), codes_to_fp16(c.z), codes_to_fp16(c.w)} {}
  // Computed ahead of what stands behind this.
  __device__ __forceinline__ void keep() {
    asm volatile(""
                 : "+r"(v[0].x), "+r"(v[0].y), "+r"(v[1].x), "+r"(v[1].y), "+r"(v[2].x),
                   "+r"(v[2].y), "+r"(v[3].x), "+r"(v[3].y));
  }
};

// map_a: the weight's codes as TMA tiles of 128 bytes by 128 rows (gated: make_gated_map);
// map_b: the rows' by 64 rows.  A block, or (kHalves = 1) two in a cluster, which share a
// tile's contraction.
template <typename T, int kUse, int kHalves>
__global__ void __launch_bounds__(kInt8Threads, 1)
k_int8_product(const __grid_constant__ CUtensorMap map_a,
               const __grid_constant__ CUtensorMap map_b, const QuantArgs a) {
  using Registers = Int8Registers<kUse, kHalves>;
  constexpr bool kGatedForm = kUse == kGated;
  constexpr int kHalfStep = m_step<kUse>() / 2;  // features of 128 rows of A
  extern __shared__ uint8_t smem_raw[];
  // s_parts is used in the cluster's first block only.
  __shared__ __align__(8) uint64_t s_raw[kMostRaw], s_read[kMostRaw], s_wide[kMostWide],
      s_empty[kMostWide], s_done[2 * kHalves], s_free[2 * kHalves], s_parts;
  __shared__ uint32_t s_tmem;
  __shared__ int s_gave_up, s_cap;
  __shared__ uint32_t s_issued;  // slices that this block's producer has issued

  uint8_t* data = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* staging = data + kInt8DataBytes;
  Segment* segments = reinterpret_cast<Segment*>(staging + kStagingBytes);
  int* first = reinterpret_cast<int*>(segments + a.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = static_cast<int>(cluster_rank()), splits = static_cast<int>(cluster_size());
  const int worker = blockIdx.x / splits, workers = gridDim.x / splits;
  constexpr int kConvert = kEpiWarps, kProducer = 2 * kEpiWarps, kIssue = kProducer + 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMostRaw; ++i) {
      mbar_init(smem_addr(&s_raw[i]), 1);
      mbar_init(smem_addr(&s_read[i]), kEpiWarps);
    }
    for (int i = 0; i < kMostWide; ++i) {
      mbar_init(smem_addr(&s_wide[i]), kEpiWarps / 2 * kHalves);
      mbar_init(smem_addr(&s_empty[i]), 1);
    }
    for (int i = 0; i < 2 * kHalves; ++i) {
      mbar_init(smem_addr(&s_done[i]), 1);
      mbar_init(smem_addr(&s_free[i]), kEpiWarps);
    }
    mbar_init(smem_addr(&s_parts), kEpiWarps);
    mbar_init_fence();
    s_gave_up = 0;
    s_issued = 0;
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
  }
  __syncthreads();
  cluster_arrive();  // this block's barriers exist
  if (warp == kIssue) tmem_alloc_single(smem_addr(&s_tmem), 512);
  pdl_wait();
  pdl_launch_dependents();

  const int width = static_cast<int>(kGatedForm ? a.N / 2 : a.N);
  const int m_blocks = (width + kHalves * kHalfStep - 1) / (kHalves * kHalfStep);
  const int all_slices = static_cast<int>((a.K + kRawSlice - 1) / kRawSlice);
  for (int e = threadIdx.x; e < a.E; e += kInt8Threads) {
    bool bad;
    segments[e] = segment(a.offset, e, a.num_rows, &bad);
    if (bad && a.status != nullptr && blockIdx.x == 0)
      atomicOr(a.status, MOE_FLAG_OFFSET_OUT_OF_RANGE);
  }
  __syncthreads();
  if (warp == 0) {
    const int cap = scan_tiles<kInt8Widest, false>(
        a.E, segments, first, splits > 1, m_blocks, workers, [&](int cap, int blocks, int rows) {
          return int8_cap_cost<kHalves>(cap, blocks, rows, m_blocks, 2 * all_slices, workers);
        });
    if (lane == 0) s_cap = cap;
  }
  tc_fence_before();
  __syncthreads();
  cluster_wait();  // the other block's barriers exist too
  tc_fence_after();
  const int cap = s_cap;
  const Int8Shape<kHalves> shape(cap);
  int total = first[a.E];
  // (More tiles than workers only where bad offsets make segments overlap.)
  if (splits > 1) total = min(total, workers);
  const uint32_t tmem = s_tmem, tmem_a = tmem + shape.slots * shape.columns;
  const uint32_t raw = smem_addr(data), wide = raw + shape.raw * shape.raw_bytes;
  volatile int* gave_up = &s_gave_up;
  const uint32_t progress = smem_addr(&s_issued);  // of the waits that span a contraction

  auto tile_at = [&](int t) {
    Tile tile = find_tile<kUse>(a.E, segments, first, t, m_blocks, 0, 0, cap);
    if (kHalves == 1) tile.m0 /= 2;
    return tile;
  };
  const int first_slice = all_slices * split / splits;
  const int n_slices = all_slices * (split + 1) / splits - first_slice;
  // Columns of a tile's product.
  auto mma_n = [](int cols) { return (cols + 15) / 16 * 16; };

  if (warp >= kProducer) {
    fewer_registers<Registers::kOther>();
    if (warp == kProducer) {
      if (elect_one()) {
        Int8Ring ring = {0, 0};
        uint32_t issued = 0;
        bool ok = true;
        for (Walk walk(worker, workers); walk.t < total && ok; walk.next()) {
          const Tile tile = tile_at(walk.t);
          const int b_boxes = (mma_n(tile.cols) + 63) / 64;
          const uint32_t bytes = kHalves * kTileABytes + b_boxes * kBoxBytes;
          for (int s = 0; s < n_slices; ++s, ++issued) {
            const uint32_t full = smem_addr(&s_raw[ring.at]);
            if (withheld(issued) ||
                !mbar_wait_as<kWaitHere>(smem_addr(&s_read[ring.at]), ring.pass ^ 1, gave_up)) {
              ok = false;
              break;
            }
            *static_cast<volatile uint32_t*>(&s_issued) = issued + 1;
            mbar_expect(full, bytes);
            uint32_t to = raw + ring.at * shape.raw_bytes;
            ring.advance(shape.raw);
            const int k = (first_slice + s) * kRawSlice;
#pragma unroll
            for (int h = 0; h < kHalves; ++h, to += kTileABytes) {
              const int m = tile.m0 + h * kHalfStep;
              if (kGatedForm) tma_load_5d_single(to, &map_a, k, 0, 0, m / 8, tile.e, full);
              else tma_load_3d_single(to, &map_a, k, m, tile.e, full);
            }
            for (int i = 0; i < b_boxes; ++i)
              tma_load_2d_single(to + i * kBoxBytes, &map_b, k, tile.lo + i * 64, full);
          }
        }
        if (*gave_up != 0) {  // no copy may be in flight when the block ends
          const unsigned long long t0 = now_ns();
          for (int i = 0; i < shape.raw && static_cast<uint32_t>(i) < issued; ++i) {
            ring.back(shape.raw);
            while (!mbar_try_here(smem_addr(&s_raw[ring.at]), ring.pass) &&
                   now_ns() - t0 < kWaitNs) {
            }
          }
        }
      }
      __syncwarp();
    } else if (warp == kIssue) {
      if (elect_one()) {
        Int8Ring ring = {0, 0}, slot = {0, 0};  // of fp16 stages, of accumulators
        uint32_t issued = 0;
        bool ok = true;
        for (Walk walk(worker, workers); walk.t < total && ok; walk.next()) {
          const Tile tile = tile_at(walk.t);
          const uint32_t idesc = instr_desc(false, false, false, 128, mma_n(tile.cols));
          Int8Ring own[kHalves];
#pragma unroll
          for (int h = 0; h < kHalves; ++h) own[h] = slot, slot.advance(shape.slots);
          for (int s = 0; s < 2 * n_slices && ok; ++s, ++issued) {
            if (!mbar_wait_as<kWaitHere>(smem_addr(&s_wide[ring.at]), ring.pass, gave_up)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t pa = tmem_a + ring.at * kHalves * kWideColumns;
            const uint32_t pb = wide + ring.at * shape.wide_bytes;
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
              if (s == 0) {
                if (!mbar_wait_as<kWaitHere>(smem_addr(&s_free[own[h].at]), own[h].pass ^ 1, gave_up,
                                             progress)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
              }
              const uint32_t acc = tmem + own[h].at * shape.columns;
#pragma unroll
              for (int i = 0; i < kSlice / 16; ++i)
                tc_mma_tmem_single(acc, pa + h * kWideColumns + i * 8,
                                   smem_desc(pb + i * 32, 16, 1024), idesc, s > 0 || i > 0);
              if (s == 2 * n_slices - 1) tc_commit_single(smem_addr(&s_done[own[h].at]));
            }
            tc_commit_single(smem_addr(&s_empty[ring.at]));
            ring.advance(shape.wide);
          }
        }
        // The products are over before the memory they read and write is given up.
        if (*gave_up != 0) {
          const unsigned long long t0 = now_ns();
          for (int i = 0; i < shape.wide && static_cast<uint32_t>(i) < issued; ++i) {
            ring.back(shape.wide);
            while (!mbar_try_here(smem_addr(&s_empty[ring.at]), ring.pass) &&
                   now_ns() - t0 < kWaitNs) {
            }
          }
        }
      }
      __syncwarp();
    }
  } else if (warp >= kConvert) {
    fewer_registers<Registers::kConvert>();
    // A lane has one row of A, and chunks of 16 codes of B.  Two halves: warps 0-3 have the
    // first's rows, 4-7 the second's, and all work on one stage of 64 codes.  One half: warps
    // 0-3 have the first 64 codes of a slice, 4-7 the others.  Chunk c of a row lies at
    // c ^ (row % 8), and makes 8 columns of the row's lane in tensor memory, or the chunks 2 c
    // and 2 c + 1 of 8 numbers in shared memory (no access meets in a bank).
    const int w = warp - kConvert, set = w >> 2, quarter = w & 3, turn = lane & 7;
    constexpr int kSets = kHalves == 2 ? 1 : 2;          // that work on stages of their own
    constexpr int kMost = kInt8Columns / (32 * kHalves);  // of B, a lane's
    static_assert(kInt8Columns % (32 * kHalves) == 0, "every row of B is converted");
    constexpr int kRowStep = kHalves == 2 ? 64 : 32;     // between a lane's rows of B
    const int b_row = (kHalves == 2 ? (w & 1) * 32 : 0) + lane;
    const int b_chunk = kHalves == 2 ? w >> 1 : quarter;
    const uint32_t a_from =
        raw + (kHalves == 2 ? set * kTileABytes : 0) + (quarter * 32 + lane) * 128;
    const uint32_t b_from = raw + kHalves * kTileABytes + b_row * 128;
    const uint32_t a_to = tmem_a + (static_cast<uint32_t>(quarter * 32) << 16) +
                          (kHalves == 2 ? set * kWideColumns : 0);
    const uint32_t b_to = wide + b_row * 128;
    Int8Ring from = {0, 0}, ring = {0, 0};  // raw stages, stages of fp16
    if (kSets == 2) ring.advance(shape.wide, set);
    bool ok = true;
    for (Walk walk(worker, workers); walk.t < total && ok; walk.next()) {
      const int rows = mma_n(tile_at(walk.t).cols) - b_row + lane;  // a warp's, of B
      for (int s = 0; s < n_slices && ok; ++s) {
        if (!warp_wait_as<kWaitAwake>(smem_addr(&s_raw[from.at]), from.pass, gave_up)) {
          ok = false;
          break;
        }
        const uint32_t stage = from.at * shape.raw_bytes;
#pragma unroll
        for (int i = 0; i < 2 / kSets; ++i) {
          const int h = kSets == 2 ? set : i;  // which 64 codes
          uint4 x[4], y[kMost];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[j] = shared_load16(a_from + stage + (((4 * h + j) ^ turn) << 4));
#pragma unroll
          for (int j = 0; j < kMost; ++j)
            if (j * kRowStep < rows)
              y[j] = shared_load16(b_from + stage + j * kRowStep * 128 +
                                   (((4 * h + b_chunk) ^ turn) << 4));
          if (i == 2 / kSets - 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&s_read[from.at]));
          }
          Wide16 v[4];
          if (Registers::kEarly) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = Wide16(x[j]), v[j].keep();
          }
          if (!warp_wait_as<kWaitAwake>(smem_addr(&s_empty[ring.at]), ring.pass ^ 1, gave_up)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t at_a = a_to + ring.at * kHalves * kWideColumns;
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            if (!Registers::kEarly) v[j] = Wide16(x[j]), v[j + 1] = Wide16(x[j + 1]);
            tmem_store_row16(at_a + j * 8, v[j].v, v[j + 1].v);
          }
          const uint32_t at_b = b_to + ring.at * shape.wide_bytes;
#pragma unroll
          for (int j = 0; j < kMost; ++j)
            if (j * kRowStep < rows) {
              const Wide16 b(y[j]);
              const uint32_t to = at_b + j * kRowStep * 128;
              shared_store16(to + (((2 * b_chunk) ^ turn) << 4),
                             make_uint4(b.v[0].x, b.v[0].y, b.v[1].x, b.v[1].y));
              shared_store16(to + (((2 * b_chunk + 1) ^ turn) << 4),
                             make_uint4(b.v[2].x, b.v[2].y, b.v[3].x, b.v[3].y));
            }
          fence_async_shared();
          tmem_wait_store();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&s_wide[ring.at]));
          ring.advance(shape.wide, kSets);
        }
        from.advance(shape.raw);
      }
    }
    __syncwarp();
  } else {
    more_registers<Registers::kEpilogue>();
    const int quad = warp & 3, g = lane >> 2, q = lane & 3;
    const uint32_t stage = smem_addr(staging + warp * kStagingWarpBytes);
    T* out = static_cast<T*>(a.out);
    T* residual = kGatedForm ? nullptr : static_cast<T*>(const_cast<void*>(a.residual));
    Int8Ring slot = {0, 0};
    // Blocks that share a tile have one tile at most: its sums may lie over the stages,
    // which are through.  A lane's 32 values of the warp's columns c: 8 steps of 512 bytes
    // from part + 64 c on.
    const uint32_t part = raw + warp * 4 * 4096 + lane * 16;
    const uint32_t other_part = splits > 1 ? cluster_addr(part, 1) : 0;
    bool ok = true;
    for (Walk walk(worker, workers); walk.t < total && ok; walk.next()) {
      const Tile tile = tile_at(walk.t);
      const int cols = tile.cols;
      for (int half = 0; half < kHalves; ++half) {
        // The warp's 32 features, its columns c + [0, 32); the lane's four of the former,
        // 16 h + 8 s + g (gated: 8 h + g, the gate's for s = 0 and the up's).
        const int64_t m = tile.m0 + half * kHalfStep + quad * (kGatedForm ? 16 : 32);
        const int c0 = warp / 4 * 32;
        float ws[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t f = m + (kGatedForm ? j / 2 * 8 : j * 8) + g;
          ws[j] = f < width ? __ldg(a.weight_scales + static_cast<int64_t>(tile.e) * a.N + f +
                                    (kGatedForm && j % 2 == 1 ? width : 0))
                            : 0.f;
        }
        float bias[4] = {};
        if (!kGatedForm && a.bias != nullptr) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t f = m + j * 8 + g;
            if (f < a.N)
              bias[j] = to_f(static_cast<const T*>(a.bias)[static_cast<int64_t>(tile.e) * a.N + f]);
          }
        }
        // Scales of rows and the residual are loaded a block of 32 columns ahead.
        float xs[8];  // columns 8 i + 2 q + b
        uint4 x[4];
        auto fetch = [&](int c) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int col = c + j / 2 * 8 + q * 2 + j % 2;
            xs[j] = col < cols ? __ldg(a.scales + tile.lo + col) : 0.f;
          }
          if (!kGatedForm && residual != nullptr && c < cols)
            load_block(x, Block<T>(residual, a.N, tile.lo + c, cols - c, m, a.N, stage));
        };
        fetch(c0);
        if (!warp_wait_as<kWaitHere>(smem_addr(&s_done[slot.at]), slot.pass, gave_up, progress)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + slot.at * shape.columns;
        if (kHalves == 1 && splits > 1) {
          if (split > 0) {
            for (int c = c0; c < cols; c += 64) {
              float z[32];
              tmem_load_32x32(acc + c, z);
              tmem_wait_load(z);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                shared_store16(part + (c - c0) * 64 + j * 512,
                               make_uint4(__float_as_uint(z[4 * j]), __float_as_uint(z[4 * j + 1]),
                                          __float_as_uint(z[4 * j + 2]),
                                          __float_as_uint(z[4 * j + 3])));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_addr(&s_parts), 0));
            ok = false;
            break;
          }
          if (!warp_wait_as<kWaitCluster>(smem_addr(&s_parts), 0, gave_up,
                                          cluster_addr(progress, 1))) {
            ok = false;
            break;
          }
        }
        for (int c = c0; c < cols; c += 64) {
          const int64_t row = tile.lo + c;
          float z[32];
          tmem_load_32x32(acc + c, z);
          tmem_wait_load(z);
          if (kHalves == 1 && splits > 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 x = cluster_load4(other_part + (c - c0) * 64 + j * 512);
              z[4 * j] += x.x, z[4 * j + 1] += x.y, z[4 * j + 2] += x.z, z[4 * j + 3] += x.w;
            }
          }
#pragma unroll
          for (int j = 0; j < 32; ++j)  // j = 16 h + 4 i + 2 s + b
            z[j] *= ws[j / 16 * 2 + j / 2 % 2] * xs[j / 4 % 4 * 2 + j % 2];
          if (kGatedForm) {
            fetch(c + 64);
            float gate[16], up[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {  // j = 4 i + 2 h + b
              gate[j] = z[j / 2 % 2 * 16 + j / 4 * 4 + j % 2];
              up[j] = z[j / 2 % 2 * 16 + j / 4 * 4 + 2 + j % 2];
            }
            apply_act<16>(a.act, gate);
#pragma unroll
            for (int j = 0; j < 16; ++j) gate[j] *= up[j];
            write_half_block(gate, Block<T, 16>(out, width, row, cols - c, m, width, stage));
          } else {
            if (a.bias != nullptr) {
#pragma unroll
              for (int j = 0; j < 4; ++j)  // z[16 h + 4 i + 2 s + b]: feature 16 h + 8 s + g
#pragma unroll
                for (int k = 0; k < 8; ++k) z[j / 2 * 16 + k / 2 * 4 + j % 2 * 2 + k % 2] += bias[j];
            }
            uint4 r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = x[j];
            fetch(c + 64);
            apply_act<32>(a.act, z);
            if (residual != nullptr) {
              const Block<T> b(residual, a.N, row, cols - c, m, a.N, stage);
              add_block(z, r, b);
            }
            write_block(z, Block<T>(out, a.N, row, cols - c, m, a.N, stage));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(smem_addr(&s_free[slot.at]));
        slot.advance(shape.slots);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the arrivals and reads of the cluster are over
  tc_fence_after();
  if (threadIdx.x == 0 && *gave_up != 0 && a.status != nullptr)
    atomicOr(a.status, MOE_FLAG_BARRIER_TIMEOUT);
  if (warp == kIssue) tmem_free_single(tmem, 512);
}

}  // namespace experts
}  // namespace moe
