// int8_product.cuh -- the grouped products of int8 rows and weights, on tcgen05.
//
//   z[r, n] = xs[r] ws[n] sum_k x[r, k] w[n, k]
//
// tcgen05 has no integer products on sm_103, so the codes become fp16 on their way: a
// code is a whole number of 8 bits, which fp16 holds exactly, as it does the products
// in fp32 (sums are rounded where they pass 2^24).  The tiles and the epilogue are
// those of expert_product.cuh; between the copies and the products stand eight warps
// that read 128-byte slices of codes.  The weights' go to tensor memory as fp16, the
// rows' to shared memory, whose bandwidth is what bounds the kernel: with both in shared
// memory a 128-deep slice of 256 columns moves 192 KB through it, 2000 cycles for 1024 of
// products.  Tensor memory then has two accumulators of 192 columns and four stages of 32.
// On GB300, weights in shared / in tensor memory, us: one expert, 8191 rows, 4096 -> 4096
// 235 / 226 (1.2 PFLOP/s); 8 experts, 8192 rows, 14336 -> 4096 792 / 745 (1.3); 128 experts,
// 512 rows, gated, 2048 -> 2 x 768 131 / 88; 256 experts, 32768 rows, 2048 -> 7168
// 1852 / 1361.  Twice the converting warps: 226, 89 and 1338, with registers spilled.
//   warps 0-7    epilogue: tensor memory -> registers, scaled -> shared -> rows
//   warps 8-15   codes -> fp16
//   warp 16      TMA producer: 128 codes deep, a ring of 4 x 32 KB
//   warp 17      tcgen05.mma issue (first block), tensor memory allocation
//   warps 18-19  fill up a warpgroup (setmaxnreg)
#pragma once

#include "quant_product.cuh"

namespace moe {
namespace experts {

constexpr int kRawStages = 4;
constexpr int kRawSlice = 128;     // codes of a raw stage
constexpr int kWideStages = 4;     // of fp16, 64 deep
constexpr int kInt8CapIndex = 4;   // cap_of(4) = 192 columns of an accumulator
constexpr int kInt8Columns = kMaxN - 16 * kInt8CapIndex;
constexpr int kWideColumns = kSlice / 2;  // of tensor memory
static_assert(2 * kInt8Columns + kWideStages * kWideColumns == 512, "tensor memory");
constexpr int kInt8Threads = 640;
constexpr int kInt8EpilogueRegisters = 136, kInt8ConvertRegisters = 80, kInt8OtherRegisters = 48;
static_assert(2 * kInt8EpilogueRegisters + 2 * kInt8ConvertRegisters + kInt8OtherRegisters <=
                  65536 / 640 / 8 * 8 * 5,
              "registers at launch: 96 a thread");

// Dynamic shared memory: raw and fp16 stages (1024-byte aligned), staging, then each
// expert's rows and its first tile.
inline size_t int8_product_smem(int E) {
  return 1024 + kRawStages * kStageBytes + kWideStages * kTileBBytes + kStagingBytes +
         static_cast<size_t>(E) * 12 + 4;
}
static_assert(1024 + kRawStages * kStageBytes + kWideStages * kTileBBytes + kStagingBytes +
                      MOE_MAX_LOCAL_EXPERTS * 12 + 4 + 1024 <= 227 * 1024,
              "shared memory of one block");

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

// map_a: the weight's codes as TMA tiles of 128 bytes by 128 rows (gated: make_gated_map);
// map_b: the rows' by 64 rows.
template <typename T, int kUse>
__global__ void __launch_bounds__(kInt8Threads, 1)
k_int8_product(const __grid_constant__ CUtensorMap map_a,
               const __grid_constant__ CUtensorMap map_b, const QuantArgs a) {
  constexpr bool kGatedForm = kUse == kGated;
  extern __shared__ uint8_t smem_raw[];
  // s_wide and s_free are used in a pair's first block only, s_parts in the cluster's
  // first pair.
  __shared__ __align__(8) uint64_t s_raw[kRawStages], s_read[kRawStages], s_wide[kWideStages],
      s_empty[kWideStages], s_done[2], s_free[2], s_parts;
  __shared__ uint32_t s_tmem;
  __shared__ int s_gave_up, s_cap;
  __shared__ uint32_t s_issued;  // slices that this block's producer has issued

  uint8_t* raw = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* stages = raw + kRawStages * kStageBytes;
  uint8_t* staging = stages + kWideStages * kTileBBytes;
  Segment* segments = reinterpret_cast<Segment*>(staging + kStagingBytes);
  int* first = reinterpret_cast<int*>(segments + a.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Clusters of `splits` pairs; the block's place in its pair; the rank of the
  // pair's first block.
  const uint32_t place = cluster_rank(), leader = place & ~1u;
  const int rank = static_cast<int>(place & 1u), split = static_cast<int>(place / 2);
  const int splits = static_cast<int>(cluster_size() / 2);
  const int pair = blockIdx.x / (2 * splits), pairs = gridDim.x / (2 * splits);
  constexpr int kConvert = kEpiWarps, kProducer = 2 * kEpiWarps, kIssue = kProducer + 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRawStages; ++i) {
      mbar_init(smem_addr(&s_raw[i]), 1);
      mbar_init(smem_addr(&s_read[i]), kEpiWarps);
    }
    for (int i = 0; i < kWideStages; ++i) {
      mbar_init(smem_addr(&s_wide[i]), kEpiWarps);  // half the warps of two blocks
      mbar_init(smem_addr(&s_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&s_done[i]), 1);
      mbar_init(smem_addr(&s_free[i]), 2 * kEpiWarps);
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
  if (warp == kIssue) tmem_alloc(smem_addr(&s_tmem), 512);
  pdl_wait();
  pdl_launch_dependents();

  const int width = static_cast<int>(kGatedForm ? a.N / 2 : a.N);
  const int m_blocks = (width + m_step<kUse>() - 1) / m_step<kUse>();
  const int all_slices = static_cast<int>((a.K + kRawSlice - 1) / kRawSlice);
  for (int e = threadIdx.x; e < a.E; e += kInt8Threads) {
    bool bad;
    segments[e] = segment(a.offset, e, a.num_rows, &bad);
    if (bad && a.status != nullptr && blockIdx.x == 0)
      atomicOr(a.status, MOE_FLAG_OFFSET_OUT_OF_RANGE);
  }
  __syncthreads();
  if (warp == 0) {
    // (a slice here is two of expert_product.cuh's)
    const int cap = scan_tiles<kInt8CapIndex>(a.E, segments, first, splits > 1, m_blocks,
                                              2 * all_slices, pairs);
    if (lane == 0) s_cap = cap;
  }
  tc_fence_before();
  __syncthreads();
  cluster_wait();  // the other blocks' barriers exist too
  tc_fence_after();
  const int cap = s_cap;
  int total = first[a.E];
  // (More tiles than pairs only where bad offsets make segments overlap.)
  if (splits > 1) total = min(total, pairs);
  const uint32_t tmem = s_tmem;
  volatile int* gave_up = &s_gave_up;
  const uint32_t progress = smem_addr(&s_issued);  // of the waits that span a contraction

  auto tile_at = [&](int t) {
    return find_tile<kUse>(a.E, segments, first, t, m_blocks, 0, 0, cap);
  };
  const int first_slice = all_slices * split / splits;
  const int n_slices = all_slices * (split + 1) / splits - first_slice;
  // Columns of a tile's product (each block holds half of B).
  auto mma_n = [](int cols) { return (cols + 15) / 16 * 16; };
  // First feature of the block's A tile.
  auto feature = [&](const Tile& t) { return t.m0 + rank * (m_step<kUse>() / 2); };

  if (warp >= kProducer) {
    fewer_registers<kInt8OtherRegisters>();
    if (warp == kProducer) {
      if (elect_one()) {
        uint32_t issued = 0;
        bool ok = true;
        for (Walk walk(pair, pairs); walk.t < total && ok; walk.next()) {
          const Tile tile = tile_at(walk.t);
          const int half_n = mma_n(tile.cols) / 2;
          const int b_boxes = (half_n + 63) / 64;
          const uint32_t bytes = kTileABytes + b_boxes * kBoxBytes;
          const int m = feature(tile), n = tile.lo + rank * half_n;
          for (int s = 0; s < n_slices; ++s, ++issued) {
            const uint32_t st = issued % kRawStages;
            if (withheld(issued) ||
                !mbar_wait_as<kWaitHere>(smem_addr(&s_read[st]), (issued / kRawStages & 1) ^ 1, gave_up)) {
              ok = false;
              break;
            }
            *static_cast<volatile uint32_t*>(&s_issued) = issued + 1;
            const uint32_t full = smem_addr(&s_raw[st]);
            mbar_expect(full, bytes);
            const uint32_t sa = smem_addr(raw + st * kStageBytes);
            const int k = (first_slice + s) * kRawSlice;
            if (kGatedForm) tma_load_5d(sa, &map_a, k, 0, 0, m / 8, tile.e, full);
            else tma_load_3d(sa, &map_a, k, m, tile.e, full);
            for (int i = 0; i < b_boxes; ++i)
              tma_load_2d(sa + kTileABytes + i * kBoxBytes, &map_b, k, n + i * 64, full);
          }
        }
        if (*gave_up != 0) {  // no copy may be in flight when the block ends
          const unsigned long long t0 = now_ns();
          for (uint32_t i = 1; i <= kRawStages && i <= issued; ++i)
            while (!mbar_try_here(smem_addr(&s_raw[(issued - i) % kRawStages]),
                                  (issued - i) / kRawStages & 1) &&
                   now_ns() - t0 < kWaitNs) {
            }
        }
      }
      __syncwarp();
    } else if (warp == kIssue) {
      if (rank == 0 && elect_one()) {
        uint32_t issued = 0, done = 0;  // fp16 slices, tiles
        const uint16_t both = static_cast<uint16_t>(3u << leader);
        bool ok = true;
        for (Walk walk(pair, pairs); walk.t < total && ok; walk.next(), ++done) {
          const Tile tile = tile_at(walk.t);
          const uint32_t idesc = instr_desc(false, false, false, 256, mma_n(tile.cols));
          const uint32_t buf = done & 1, acc = tmem + buf * kInt8Columns;
          if (!mbar_wait_as<kWaitHere>(smem_addr(&s_free[buf]), (done / 2 & 1) ^ 1, gave_up, progress)) break;
          for (int s = 0; s < 2 * n_slices; ++s, ++issued) {
            const uint32_t st = issued % kWideStages;
            if (!mbar_wait_as<kWaitHere>(smem_addr(&s_wide[st]), issued / kWideStages & 1, gave_up)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t pa = tmem + 2 * kInt8Columns + st * kWideColumns;
            const uint32_t pb = smem_addr(stages + st * kTileBBytes);
#pragma unroll
            for (int i = 0; i < kSlice / 16; ++i)
              tc_mma_tmem(acc, pa + i * 8, smem_desc(pb + i * 32, 16, 1024), idesc,
                          s > 0 || i > 0);
            tc_commit(smem_addr(&s_empty[st]), both);
          }
          if (ok) tc_commit(smem_addr(&s_done[buf]), both);
        }
        // The products are over before the memory they read and write is given up.
        if (*gave_up != 0) {
          const unsigned long long t0 = now_ns();
          for (uint32_t i = 1; i <= kWideStages && i <= issued; ++i)
            while (!mbar_try_here(smem_addr(&s_empty[(issued - i) % kWideStages]),
                                  (issued - i) / kWideStages & 1) &&
                   now_ns() - t0 < kWaitNs) {
            }
        }
      }
      __syncwarp();
    }
  } else if (warp >= kConvert) {
    fewer_registers<kInt8ConvertRegisters>();
    // Warps 0-3 have the first 64 codes of a slice, 4-7 the others, a lane one row of A and
    // one of B: chunk c of 16 codes lies at c ^ (row % 8), and makes 8 columns of the row's
    // lane in tensor memory, or the chunks 2 c and 2 c + 1 of 8 numbers (neither access
    // meets in a bank).  A slice is read whole, so that the next copy into its stage starts at
    // once.
    const int w = warp - kConvert, h = w >> 2, row = (w & 3) * 32 + lane, turn = lane & 7;
    const uint32_t from0 = smem_addr(raw) + row * 128;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((w & 3) * 32) << 16) + 2 * kInt8Columns;
    const uint32_t rows = smem_addr(stages) + row * 128;
    const uint32_t wide0 = cluster_addr(smem_addr(&s_wide[0]), leader);
    uint32_t step = 0;  // raw slices so far
    bool ok = true;
    for (Walk walk(pair, pairs); walk.t < total && ok; walk.next()) {
      const bool any = (w & 3) * 32 < mma_n(tile_at(walk.t).cols) / 2;  // rows of B
      for (int s = 0; s < n_slices && ok; ++s, ++step) {
        const uint32_t st = step % kRawStages;
        if (!warp_wait_as<kWaitAwake>(smem_addr(&s_raw[st]), step / kRawStages & 1, gave_up)) {
          ok = false;
          break;
        }
        const uint32_t from = from0 + st * kStageBytes;
        uint4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = shared_load16(from + (((4 * h + i) ^ turn) << 4));
        if (any) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            y[i] = shared_load16(from + kTileABytes + (((4 * h + i) ^ turn) << 4));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&s_read[st]));
        const uint32_t slice = 2 * step + h, at = slice % kWideStages;
        if (!warp_wait_as<kWaitAwake>(smem_addr(&s_empty[at]), (slice / kWideStages & 1) ^ 1,
                                      gave_up)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          tmem_store_row8(lanes + at * kWideColumns + i * 8, codes_to_fp16(x[i].x),
                          codes_to_fp16(x[i].y), codes_to_fp16(x[i].z), codes_to_fp16(x[i].w));
        if (any) {
          const uint32_t to = rows + at * kTileBBytes;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint2 a0 = codes_to_fp16(y[i].x), a1 = codes_to_fp16(y[i].y);
            const uint2 a2 = codes_to_fp16(y[i].z), a3 = codes_to_fp16(y[i].w);
            shared_store16(to + (((2 * i) ^ turn) << 4), make_uint4(a0.x, a0.y, a1.x, a1.y));
            shared_store16(to + (((2 * i + 1) ^ turn) << 4), make_uint4(a2.x, a2.y, a3.x, a3.y));
          }
          fence_async_shared();
        }
        tmem_wait_store();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_written(wide0 + at * 8);
      }
    }
    __syncwarp();
  } else {
    more_registers<kInt8EpilogueRegisters>();
    const int quad = warp & 3, g = lane >> 2, q = lane & 3;
    const uint32_t stage = smem_addr(staging + warp * kStagingWarpBytes);
    T* out = static_cast<T*>(a.out);
    T* residual = kGatedForm ? nullptr : static_cast<T*>(const_cast<void*>(a.residual));
    uint32_t done = 0;
    const uint32_t free0 = cluster_addr(smem_addr(&s_free[0]), leader);
    // Pairs that share a tile have one tile at most: its sums may lie over the raw
    // stages, which are through.  A lane's 32 values of the warp's columns c: 8 steps
    // of 512 bytes from part + 64 c on.
    const uint32_t part = smem_addr(raw + warp * 4 * 4096) + lane * 16;
    const uint32_t other_part = splits > 1 ? cluster_addr(part, 2 + rank) : 0;
    for (Walk walk(pair, pairs); walk.t < total; walk.next(), ++done) {
      const Tile tile = tile_at(walk.t);
      const int cols = tile.cols;
      // The warp's 32 features, its columns c + [0, 32); the lane's four of the former,
      // 16 h + 8 s + g (gated: 8 h + g, the gate's for s = 0 and the up's).
      const int64_t m = feature(tile) + quad * (kGatedForm ? 16 : 32);
      const int c0 = warp / 4 * 32;
      float ws[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t f = m + (kGatedForm ? j / 2 * 8 : j * 8) + g;
        ws[j] = f < width ? __ldg(a.weight_scales + static_cast<int64_t>(tile.e) * a.N + f +
                                  (kGatedForm && j % 2 == 1 ? width : 0))
                          : 0.f;
      }
      const uint32_t buf = done & 1;
      if (!warp_wait_as<kWaitNap>(smem_addr(&s_done[buf]), done / 2 & 1, gave_up, progress)) break;
      tc_fence_after();
      const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * kInt8Columns;
      if (splits > 1) {
        if (split > 0) {
          for (int c = c0; c < cols; c += 64) {
            float z[32];
            tmem_load_32x32(acc + c, z);
            tmem_wait_load(z);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              shared_store16(part + (c - c0) * 64 + j * 512,
                             make_uint4(__float_as_uint(z[4 * j]), __float_as_uint(z[4 * j + 1]),
                                        __float_as_uint(z[4 * j + 2]), __float_as_uint(z[4 * j + 3])));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_addr(&s_parts), rank));
          break;
        }
        if (!warp_wait_as<kWaitCluster>(smem_addr(&s_parts), 0, gave_up, cluster_addr(progress, 2 + rank)))
          break;
      }
      for (int c = c0; c < cols; c += 64) {
        const int64_t row = tile.lo + c;
        float xs[8];  // columns 8 i + 2 q + b
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int col = c + j / 2 * 8 + q * 2 + j % 2;
          xs[j] = col < cols ? __ldg(a.scales + tile.lo + col) : 0.f;
        }
        float z[32];
        tmem_load_32x32(acc + c, z);
        tmem_wait_load(z);
        if (splits > 1) {
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
            const T* bias = static_cast<const T*>(a.bias) + static_cast<int64_t>(tile.e) * a.N;
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // z[16 h + 4 i + 2 s + b]: feature 16 h + 8 s + g
              const int64_t f = m + j * 8 + g;
              const float x = f < a.N ? to_f(bias[f]) : 0.f;
#pragma unroll
              for (int k = 0; k < 8; ++k) z[j / 2 * 16 + k / 2 * 4 + j % 2 * 2 + k % 2] += x;
            }
          }
          apply_act<32>(a.act, z);
          if (residual != nullptr) {
            uint4 x[4];
            const Block<T> b(residual, a.N, row, cols - c, m, a.N, stage);
            load_block(x, b);
            add_block(z, x, b);
          }
          write_block(z, Block<T>(out, a.N, row, cols - c, m, a.N, stage));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed_cluster(free0 + buf * 8);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the products, loads, arrivals and reads of the cluster are over
  tc_fence_after();
  if (threadIdx.x == 0 && *gave_up != 0 && a.status != nullptr)
    atomicOr(a.status, MOE_FLAG_BARRIER_TIMEOUT);
  if (warp == kIssue) tmem_free(tmem, 512);
}

}  // namespace experts
}  // namespace moe
