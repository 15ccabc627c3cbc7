// quant_product.cuh -- the grouped products of fp8 rows and weights, on tcgen05.
//
//   z[r, n] = sum over groups g of 128 columns of
//             xs[r, g] ws[n / 128, g] sum_{k in g} x[r, k] w[n, k]
//
// A group's sum is scaled by a number of its own before it joins the others, so each
// slice's products (128 deep: one group) go to a tensor memory buffer of their own, and
// the epilogue warps add it, scaled, to sums that stay in their registers (128 a thread)
// while the next slice is multiplied.
//
// Rows are the A operand here, so that a thread, which has one lane of tensor memory,
// has one row: its scale is one number a slice (gated: two), and what is left is one
// fused multiply-add a value.  A block makes 128 rows x 256 features (gated: 128 gate and
// 128 up features).  (With the weights as A the scales lie along a thread's registers: they
// come from shared memory, by fragments, and a slice took 1900 cycles.  Pairs of SMs with
// 256 rows load a third less, but each buffer's way from products to sums and back crosses
// between them, and few rows leave half of a pair idle.  Two blocks that load half of the
// features each for both are slower: 1115 us instead of 927 for 8 experts, 8192 rows, gated,
// 4096 -> 2 x 14336.)
//   warps 0-7    tensor memory -> registers, scaled; then the epilogue
//   warp 8       TMA producer: 128-deep slices into a ring of 4 x 48 KB
//   warp 9       tcgen05.mma issue, tensor memory allocation
//   warps 10-11  the scales, four slices at a time, into a ring of 12 slices: behind the
//                tiles' loads a scale takes longer than a slice
#pragma once

#include <type_traits>

#include "expert_product.cuh"

namespace moe {
namespace experts {

constexpr int kGroupSlice = 128;   // contraction depth of one stage: a group of scales
constexpr int kTileRows = 128;
constexpr int kTileFeatures = 256;  // rows of the weight
constexpr int kRowsBytes = kTileRows * kGroupSlice, kWeightBytes = kTileFeatures * kGroupSlice;
constexpr int kFp8StageBytes = kRowsBytes + kWeightBytes;
constexpr int kFp8Stages = 4;
constexpr int kBuffers = 2;        // of tensor memory, a slice's products each
constexpr int kScaleChunk = 4;     // slices whose scales are loaded at once
constexpr int kScaleChunks = 3;    // of the ring
constexpr int kScaleSlotBytes = kTileRows * 8;  // two numbers a row
constexpr int kScaleBytes = kScaleChunks * kScaleChunk * kScaleSlotBytes;
constexpr int kQuantProductThreads = 384;
constexpr int kQuantEpilogueRegisters = 224, kQuantOtherRegisters = 56;
static_assert(2 * kQuantEpilogueRegisters + kQuantOtherRegisters <= 65536 / 384 / 8 * 8 * 3,
              "registers at launch: 168 a thread");

struct QuantArgs {
  const int64_t* offset;
  int64_t num_rows;
  int64_t K, N;  // in and out of the weight [E, N, K]
  int E;
  int act;
  const void* codes;
  const float* scales;
  const void* weight;
  const float* weight_scales;
  const void* bias;
  const void* residual;
  void* out;
  unsigned* status;
};

// Dynamic shared memory: stages (1024-byte aligned), scales, then each expert's rows and
// its first tile.
inline size_t quant_product_smem(int E) {
  return 1024 + kFp8Stages * kFp8StageBytes + kScaleBytes + static_cast<size_t>(E) * 12 + 4;
}
static_assert(1024 + kFp8Stages * kFp8StageBytes + kScaleBytes + MOE_MAX_LOCAL_EXPERTS * 12 + 4 +
                      1024 <=
                  227 * 1024,
              "shared memory of one block");

// Up to 128 rows of one expert by the features from f0 on.
struct QuantTile {
  int e, lo, rows, f0;
};

__device__ __forceinline__ QuantTile find_quant_tile(int E, const Segment* segments,
                                                     const int* first, int t, int f_blocks,
                                                     int features) {
  int lo = 0, hi = E;  // first[lo] <= t < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first[mid] <= t) lo = mid;
    else hi = mid;
  }
  const Segment s = segments[lo];
  const int rows = s.hi - s.lo;
  int f, n;
  place_in_panels(t - first[lo], f_blocks, row_blocks(rows, kTileRows), f, n);
  return {lo, s.lo + n * kTileRows, min(kTileRows, rows - n * kTileRows), f * features};
}

// 32 bytes of a row; kWide: in one access, where rows are 32-byte aligned.
template <bool kWide>
__device__ __forceinline__ void store_32_bytes(void* at, const uint32_t (&v)[8]) {
  if (kWide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    static_cast<uint4*>(at)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(at)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// z[0, 16), rounded, to columns c + [0, 16) of the row at `row`, of `width` (a multiple
// of 8).
template <typename T>
__device__ __forceinline__ void store_16(T* row, const float* z, int64_t c, int64_t width,
                                         bool wide) {
  uint32_t p[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) p[i] = pack2<T>(z[2 * i], z[2 * i + 1]);
  if (c + 16 <= width) {
    if (wide) store_32_bytes<true>(row + c, p);
    else store_32_bytes<false>(row + c, p);
  } else if (c + 8 <= width) {
    *reinterpret_cast<uint4*>(row + c) = make_uint4(p[0], p[1], p[2], p[3]);
  }
}

__device__ __forceinline__ float2 shared_load_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void shared_store_f2(uint32_t addr, float x, float y) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}

// Each expert's first tile, of 128 rows by f_blocks blocks of features, and their number
// (one warp).  The host has made sure that the tiles of num_rows rows can be counted; where
// bad offsets make segments overlap, those beyond kMostTiles are left out.
__device__ __forceinline__ void count_quant_tiles(int E, const Segment* segments, int* first,
                                                  int f_blocks) {
  constexpr int64_t kMostTiles = INT32_MAX / 2;
  const int lane = threadIdx.x & 31;
  int64_t before = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    const int64_t n = e < E ? static_cast<int64_t>(row_blocks(
                                  segments[e].hi - segments[e].lo, kTileRows)) * f_blocks
                            : 0;
    int64_t sum = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(kFullMask, sum, d);
      if (lane >= d) sum += x;
    }
    if (e < E) first[e] = static_cast<int>(min(kMostTiles, before + sum - n));
    before += __shfl_sync(kFullMask, sum, 31);
  }
  if (lane == 0) first[E] = static_cast<int>(min(kMostTiles, before));
}

// map_rows: the rows' codes as TMA tiles of 128 bytes by 64 rows, map_weight: the
// weight's [E, N, K] by 128 rows.  A block, or two in a cluster, which share a tile's
// contraction.
template <typename T, int kUse>
__global__ void __launch_bounds__(kQuantProductThreads, 1)
k_quant_product(const __grid_constant__ CUtensorMap map_rows,
                const __grid_constant__ CUtensorMap map_weight, const QuantArgs a) {
  constexpr bool kGatedForm = kUse == kGated;
  constexpr int kFeatures = m_step<kUse>();  // of a tile
  extern __shared__ uint8_t smem_raw[];
  // s_parts is used in the cluster's first block only.
  __shared__ __align__(8) uint64_t s_full[kFp8Stages], s_empty[kFp8Stages], s_done[kBuffers],
      s_free[kBuffers], s_scaled[kScaleChunks], s_used[kScaleChunks], s_parts;
  __shared__ uint32_t s_tmem;
  __shared__ int s_gave_up;
  __shared__ uint32_t s_issued;  // slices that this block's producer has issued

  uint8_t* stages = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t scale_ring = smem_addr(stages + kFp8Stages * kFp8StageBytes);
  Segment* segments =
      reinterpret_cast<Segment*>(stages + kFp8Stages * kFp8StageBytes + kScaleBytes);
  int* first = reinterpret_cast<int*>(segments + a.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = static_cast<int>(cluster_rank()), splits = static_cast<int>(cluster_size());
  const int worker = blockIdx.x / splits, workers = gridDim.x / splits;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kFp8Stages; ++i) {
      mbar_init(smem_addr(&s_full[i]), 1);
      mbar_init(smem_addr(&s_empty[i]), 1);
    }
    for (int i = 0; i < kBuffers; ++i) {
      mbar_init(smem_addr(&s_done[i]), 1);
      mbar_init(smem_addr(&s_free[i]), kEpiWarps);
    }
    for (int i = 0; i < kScaleChunks; ++i) {
      mbar_init(smem_addr(&s_scaled[i]), 2);
      mbar_init(smem_addr(&s_used[i]), kEpiWarps);
    }
    mbar_init(smem_addr(&s_parts), kEpiWarps);
    mbar_init_fence();
    s_gave_up = 0;
    s_issued = 0;
    tma_prefetch_map(&map_rows);
    tma_prefetch_map(&map_weight);
  }
  __syncthreads();
  cluster_arrive();  // this block's barriers exist
  if (warp == kEpiWarps + 1) tmem_alloc_single(smem_addr(&s_tmem), 512);
  pdl_wait();
  pdl_launch_dependents();

  const int width = static_cast<int>(kGatedForm ? a.N / 2 : a.N);
  const int f_blocks = (width + kFeatures - 1) / kFeatures;
  const int groups = static_cast<int>((a.K + kGroupSlice - 1) / kGroupSlice);  // and slices
  for (int e = threadIdx.x; e < a.E; e += kQuantProductThreads) {
    bool bad;
    segments[e] = segment(a.offset, e, a.num_rows, &bad);
    if (bad && a.status != nullptr && blockIdx.x == 0)
      atomicOr(a.status, MOE_FLAG_OFFSET_OUT_OF_RANGE);
  }
  __syncthreads();
  if (warp == 0) count_quant_tiles(a.E, segments, first, f_blocks);
  tc_fence_before();
  __syncthreads();
  cluster_wait();  // the other block's barriers exist too
  tc_fence_after();
  int total = first[a.E];
  // (More tiles than workers only where bad offsets make segments overlap.)
  if (splits > 1) total = min(total, workers);
  const uint32_t tmem = s_tmem;
  volatile int* gave_up = &s_gave_up;

  // A place in the ring of stages: stage and parity of the pass through them.
  struct Ring {
    int at = 0;
    uint32_t pass = 0;
    __device__ __forceinline__ void advance() {
      if (++at == kFp8Stages) at = 0, pass ^= 1;
    }
  };
  // After a wait gave up: what was issued last at each stage is given the time of
  // one wait to be used up, so that nothing is in flight when the block ends.
  auto drain = [&](Ring r, uint32_t issued) {
    const unsigned long long t0 = now_ns();
    for (int i = 0; i < kFp8Stages && static_cast<uint32_t>(i) < issued; ++i) {
      if (r.at == 0) r.at = kFp8Stages, r.pass ^= 1;
      --r.at;
      while (!mbar_try_here(smem_addr(&s_empty[r.at]), r.pass) && now_ns() - t0 < kWaitNs) {
      }
    }
  };
  auto tile_at = [&](int t) {
    return find_quant_tile(a.E, segments, first, t, f_blocks, kFeatures);
  };
  const int first_slice = groups * split / splits;
  const int n_slices = groups * (split + 1) / splits - first_slice;

  if (warp >= kEpiWarps) {
    fewer_registers<kQuantOtherRegisters>();
    if (warp == kEpiWarps) {
      if (elect_one()) {
        Ring ring;
        uint32_t issued = 0;
        bool ok = true;
        for (Walk walk(worker, workers); walk.t < total && ok; walk.next()) {
          const QuantTile tile = tile_at(walk.t);
          const int loads = (tile.rows + 63) / 64;
          const uint32_t bytes = kWeightBytes + loads * kBoxBytes;
          for (int s = 0; s < n_slices; ++s, ++issued) {
            const int st = ring.at;
            const uint32_t full = smem_addr(&s_full[st]);
            if (withheld(issued) ||
                !mbar_wait_as<kWaitHere>(smem_addr(&s_empty[st]), ring.pass ^ 1, gave_up)) {
              ok = false;
              break;
            }
            *static_cast<volatile uint32_t*>(&s_issued) = issued + 1;
            ring.advance();
            mbar_expect(full, bytes);
            const uint32_t sw = smem_addr(stages + st * kFp8StageBytes), sx = sw + kWeightBytes;
            const int k = (first_slice + s) * kGroupSlice;
            tma_load_3d_single(sw, &map_weight, k, tile.f0, tile.e, full);
            tma_load_3d_single(sw + kWeightBytes / 2, &map_weight, k,
                               tile.f0 + (kGatedForm ? width : 128), tile.e, full);
            for (int i = 0; i < loads; ++i)
              tma_load_2d_single(sx + i * kBoxBytes, &map_rows, k, tile.lo + i * 64, full);
          }
        }
        if (*gave_up != 0) drain(ring, issued);
      }
      __syncwarp();
    } else if (warp == kEpiWarps + 1) {
      if (elect_one()) {
        Ring ring;
        uint32_t issued = 0;
        const uint32_t idesc = instr_desc(false, false, false, kTileRows, kTileFeatures);
        bool ok = true;
        for (Walk walk(worker, workers); walk.t < total && ok; walk.next()) {
          for (int s = 0; s < n_slices; ++s) {
            const uint32_t buf = issued & 1, acc = tmem + buf * kTileFeatures;
            const int st = ring.at;
            if (!mbar_wait_as<kWaitHere>(smem_addr(&s_full[st]), ring.pass, gave_up) ||
                !mbar_wait_as<kWaitHere>(smem_addr(&s_free[buf]), (issued / 2 & 1) ^ 1, gave_up)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t pw = smem_addr(stages + st * kFp8StageBytes), px = pw + kWeightBytes;
#pragma unroll
            for (int i = 0; i < kGroupSlice / 32; ++i)
              tc_mma_fp8_single(acc, smem_desc(px + i * 32, 16, 1024),
                                smem_desc(pw + i * 32, 16, 1024), idesc, i > 0);
            tc_commit_single(smem_addr(&s_done[buf]));
            tc_commit_single(smem_addr(&s_empty[st]));
            ++issued;
            ring.advance();
          }
        }
        // The products are over before the memory they read and write is given up.
        if (*gave_up != 0) drain(ring, issued);
      }
      __syncwarp();
    } else {
      // A row's scale times those of the weight's two blocks (gated: of gate and up).
      // Lane l has rows 64 i + l and 64 i + 32 + l of the tile; kScaleChunk slices of
      // them are in flight while those before are written.
      constexpr int kMine = kTileRows / 64;
      const int r0 = (warp - kEpiWarps - 2) * (kTileRows / 2) + lane;
      const int blocks = (width + kGroupSlice - 1) / kGroupSlice;
      const bool whole = groups % kScaleChunk == 0 && first_slice % kScaleChunk == 0 &&
                         (reinterpret_cast<uintptr_t>(a.scales) & 15) == 0;
      uint32_t step = 0;  // chunks so far
      bool ok = true;
      for (Walk walk(worker, workers); walk.t < total && ok; walk.next()) {
        const QuantTile tile = tile_at(walk.t);
        const int block = tile.f0 / kGroupSlice;
        // Lanes 0-3 load the chunk's four of the first block, 4-7 of the second.
        const float* ws = a.weight_scales + first_slice + lane % kScaleChunk +
                          (static_cast<int64_t>(tile.e) * (kGatedForm ? 2 : 1) * blocks + block) *
                              groups;
        if (lane / kScaleChunk % 2 == 1)
          ws += static_cast<int64_t>(kGatedForm ? blocks : block + 1 < blocks) * groups;
        const float* xs = a.scales + (static_cast<int64_t>(tile.lo) + r0) * groups + first_slice;
        float x[kMine][kScaleChunk], w;
        auto fetch = [&](int s) {
          w = s + lane % kScaleChunk < n_slices ? __ldg(ws + s) : 0.f;
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            const float* at = xs + static_cast<int64_t>(32 * i) * groups + s;
            const bool in = r0 + 32 * i < tile.rows;
            if (whole && s + kScaleChunk <= n_slices) {
              const float4 v = in ? __ldg(reinterpret_cast<const float4*>(at))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
              x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
            } else {
#pragma unroll
              for (int k = 0; k < kScaleChunk; ++k)
                x[i][k] = in && s + k < n_slices ? __ldg(at + k) : 0.f;
            }
          }
        };
        fetch(0);
        for (int s = 0; s < n_slices; s += kScaleChunk, ++step) {
          const uint32_t chunk = step % kScaleChunks;
          if (!warp_wait_as<kWaitAwake>(smem_addr(&s_used[chunk]), (step / kScaleChunks & 1) ^ 1,
                                        gave_up)) {
            ok = false;
            break;
          }
          const uint32_t to = scale_ring + chunk * kScaleChunk * kScaleSlotBytes + r0 * 8;
#pragma unroll
          for (int k = 0; k < kScaleChunk; ++k) {
            const float by0 = __shfl_sync(kFullMask, w, k);
            const float by1 = __shfl_sync(kFullMask, w, kScaleChunk + k);
#pragma unroll
            for (int i = 0; i < kMine; ++i)
              shared_store_f2(to + k * kScaleSlotBytes + i * 256, x[i][k] * by0, x[i][k] * by1);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&s_scaled[chunk]));
          if (s + kScaleChunk < n_slices) fetch(s + kScaleChunk);
        }
      }
    }
  } else {
    more_registers<kQuantEpilogueRegisters>();
    const int quad = warp & 3, half = warp / 4;
    uint32_t done = 0;  // slices so far
    uint32_t step = 0, scale_pass = 0;  // the chunk of scales, parity of the pass through them
    // The warp's columns: four blocks of 32, two of each 128 rows of the weight.
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * 64;
    auto block_column = [](int j) { return (j >> 1) * 128 + (j & 1) * 32; };
    // Blocks that share a tile have one tile at most: its sums may lie over the stages,
    // which are through.  A lane's 128 values: 32 steps of 512 bytes.
    const uint32_t part = smem_addr(stages + warp * 32 * 512) + lane * 16;
    const uint32_t other_part = splits > 1 ? cluster_addr(part, 1) : 0;
    const bool wide = width % 16 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
    for (Walk walk(worker, workers); walk.t < total; walk.next()) {
      const QuantTile tile = tile_at(walk.t);
      const int64_t row = tile.lo + quad * 32 + lane;
      float sums[4][32];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 32; ++i) sums[j][i] = 0.f;
      bool ok = true;
      const bool any = quad * 32 < tile.rows;
      // Frees the scales of slice s, which is through, if its chunk is.
      auto scales_used = [&](int s) {
        if (s % kScaleChunk != kScaleChunk - 1 && s != n_slices - 1) return;
        if (lane == 0) mbar_arrive(smem_addr(&s_used[step]));  // behind a __syncwarp
        if (++step == kScaleChunks) step = 0, scale_pass ^= 1;
      };
      if (!any) {  // no rows: only makes room
        for (int s = 0; ok && s < n_slices; ++s, ++done) {
          ok = warp_wait_as<kWaitHere>(smem_addr(&s_done[done & 1]), done / 2 & 1, gave_up);
          if (ok && lane == 0) mbar_arrive_relaxed(smem_addr(&s_free[done & 1]));
          scales_used(s);
        }
      } else {
        // Two blocks are on their way from tensor memory while two are added.
        // (Behind the last slice what is loaded is not used.)
        float d0[32], d1[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) d0[i] = d1[i] = 0.f;
        ok = warp_wait_as<kWaitHere>(smem_addr(&s_done[done & 1]), done / 2 & 1, gave_up);
        tc_fence_after();
        tmem_load_row32(lanes + (done & 1) * kTileFeatures, d0);
        tmem_load_row32(lanes + (done & 1) * kTileFeatures + 32, d1);
        for (int s = 0; ok && s < n_slices; ++s) {
          const uint32_t acc = lanes + (done & 1) * kTileFeatures;
          if (s % kScaleChunk == 0 &&
              !warp_wait_as<kWaitAwake>(smem_addr(&s_scaled[step]), scale_pass, gave_up)) {
            ok = false;
            break;
          }
          const float2 by = shared_load_f2(scale_ring +
                                           (step * kScaleChunk + s % kScaleChunk) * kScaleSlotBytes +
                                           (quad * 32 + lane) * 8);
          tmem_wait_load(d0);
          tmem_wait_load(d1);
#pragma unroll
          for (int i = 0; i < 32; ++i) sums[0][i] = fmaf(d0[i], by.x, sums[0][i]);
          tmem_load_row32(acc + block_column(2), d0);
#pragma unroll
          for (int i = 0; i < 32; ++i) sums[1][i] = fmaf(d1[i], by.x, sums[1][i]);
          tmem_load_row32(acc + block_column(3), d1);
          tmem_wait_load(d0);
          tmem_wait_load(d1);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_relaxed(smem_addr(&s_free[done & 1]));
          ++done;
          const uint32_t bar = smem_addr(&s_done[done & 1]), parity = done / 2 & 1;
          const bool over = s == n_slices - 1 || mbar_test_here(bar, parity);
#pragma unroll
          for (int i = 0; i < 32; ++i) sums[2][i] = fmaf(d0[i], by.y, sums[2][i]);
          if (!__all_sync(kFullMask, over) && !warp_wait_as<kWaitHere>(bar, parity, gave_up)) {
            ok = false;
            break;
          }
          tc_fence_after();
          tmem_load_row32(lanes + (done & 1) * kTileFeatures, d0);
#pragma unroll
          for (int i = 0; i < 32; ++i) sums[3][i] = fmaf(d1[i], by.y, sums[3][i]);
          tmem_load_row32(lanes + (done & 1) * kTileFeatures + 32, d1);
          scales_used(s);
        }
        tmem_wait_load(d0);
        tmem_wait_load(d1);
      }
      if (!ok) break;
      if (splits > 1) {
        if (split > 0) {
          if (any) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              shared_store16(part + j * 512,
                             make_uint4(__float_as_uint(sums[j / 8][j % 8 * 4]),
                                        __float_as_uint(sums[j / 8][j % 8 * 4 + 1]),
                                        __float_as_uint(sums[j / 8][j % 8 * 4 + 2]),
                                        __float_as_uint(sums[j / 8][j % 8 * 4 + 3])));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_addr(&s_parts), 0));
          break;
        }
        if (!warp_wait_as<kWaitCluster>(smem_addr(&s_parts), 0, gave_up,
                              cluster_addr(smem_addr(&s_issued), 1)))
          break;
        if (any) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float4 v = cluster_load4(other_part + j * 512);
            float* z = &sums[j / 8][j % 8 * 4];
            z[0] += v.x, z[1] += v.y, z[2] += v.z, z[3] += v.w;
          }
        }
      }
      if (quad * 32 + lane >= tile.rows) continue;
      T* out = static_cast<T*>(a.out) + row * width;
      if (kGatedForm) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          apply_act<32>(a.act, sums[j]);
#pragma unroll
          for (int i = 0; i < 32; ++i) sums[j][i] *= sums[2 + j][i];
#pragma unroll
          for (int i = 0; i < 2; ++i)
            store_16(out, &sums[j][16 * i], tile.f0 + half * 64 + j * 32 + i * 16, width, wide);
        }
      } else {
        const T* bias = static_cast<const T*>(a.bias);
        if (bias != nullptr) bias += static_cast<int64_t>(tile.e) * a.N;
        const T* residual = static_cast<const T*>(a.residual);
        if (residual != nullptr) residual += row * width;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // v += the 32 values from c on that exist
          auto add = [&](float* v, const T* from, int64_t c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (c + 8 * i >= width) break;
              Vec8<T> p;
              p.v = *reinterpret_cast<const uint4*>(from + c + 8 * i);
#pragma unroll
              for (int k = 0; k < 8; ++k) v[8 * i + k] += to_f(p.e[k]);
            }
          };
          const int64_t c = tile.f0 + half * 64 + block_column(j);
          if (c >= width) break;
          if (bias != nullptr) add(sums[j], bias, c);
          apply_act<32>(a.act, sums[j]);
          if (residual != nullptr) add(sums[j], residual, c);
#pragma unroll
          for (int i = 0; i < 2; ++i) store_16(out, &sums[j][16 * i], c + 16 * i, width, wide);
        }
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
  if (warp == kEpiWarps + 1) tmem_free_single(tmem, 512);
}

}  // namespace experts
}  // namespace moe
