// quant_product.cuh -- the grouped products of fp8 rows and weights, on tcgen05.
//
//   z[r, n] = sum over groups g of 128 columns of
//             xs[r, g] ws[n / 128, g] sum_{k in g} x[r, k] w[n, k]
//
// The tiles are those of expert_product.cuh: a pair of SMs makes 256 x (up to 256)
// outputs, weights being the A operand, and a slice is again 128 bytes deep, which here
// is one group of scales.  A group's sum is scaled by a number of its own before it
// joins the others, so each slice's products go to a tensor memory buffer of their own
// (two, of 256 columns each) and the epilogue warps add it, scaled, to sums that stay in
// their registers (128 a thread) while the next slice is multiplied.
//   warps 0-7    tensor memory -> registers, scaled; then the epilogue
//   warp 8       TMA producer: 128-deep slices into a ring of 32 KB each
//   warp 9       tcgen05.mma issue (first block), tensor memory allocation
//   warps 10-11  the rows' scales, four slices at a time, into a ring of 12 slices
// Fragments (tcgen05.ld.16x256b) give a thread 4 weight rows by 8 columns of a 32 x 32
// block, so that it needs 8 scales for 32 values, and pairs of columns go through
// fma.f32x2: a slice is about 100 instructions of a warp, 2 warps a scheduler, beside
// 512 cycles of products.
#pragma once

#include "expert_product.cuh"

namespace moe {
namespace experts {

constexpr int kGroupSlice = 128;   // contraction depth of one stage: a group of scales
constexpr int kScaleChunk = 4;     // slices whose scales are loaded at once
constexpr int kScaleChunks = 3;    // of the ring
constexpr int kScaleSlots = kScaleChunk * kScaleChunks;
constexpr int kScaleSlotBytes = kMaxN * 4;
constexpr int kQuantProductThreads = 384;
constexpr int kQuantEpilogueRegisters = 216, kQuantOtherRegisters = 72;
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
  int stages;  // of the ring
};

// Dynamic shared memory: stages (1024-byte aligned), staging, scales, then each
// expert's rows and its first tile.
inline size_t quant_product_smem(int E, int stages) {
  return 1024 + static_cast<size_t>(stages) * kStageBytes + kStagingBytes +
         kScaleSlots * kScaleSlotBytes + static_cast<size_t>(E) * 12 + 4;
}
// What a block may have beside its static shared memory.
constexpr size_t kQuantProductMost = 227 * 1024 - 1024;
static_assert(1024 + (kStages - 1) * kStageBytes + kStagingBytes + kScaleSlots * kScaleSlotBytes +
                      MOE_MAX_LOCAL_EXPERTS * 12 + 4 <=
                  kQuantProductMost,
              "shared memory of one block");

__device__ __forceinline__ float2 shared_load_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void shared_store_f(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// map_a: the weight as TMA tiles of 128 bytes by 128 rows (gated: make_gated_map);
// map_b: the rows, by 64 rows.
template <typename T, int kUse>
__global__ void __launch_bounds__(kQuantProductThreads, 1)
k_quant_product(const __grid_constant__ CUtensorMap map_a,
                const __grid_constant__ CUtensorMap map_b, const QuantArgs a) {
  constexpr bool kGatedForm = kUse == kGated;
  extern __shared__ uint8_t smem_raw[];
  // s_full and s_free are used in a pair's first block only, s_parts in the cluster's
  // first pair.
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_done[2], s_free[2],
      s_scaled[kScaleChunks], s_used[kScaleChunks], s_parts;
  __shared__ uint32_t s_tmem;
  __shared__ int s_gave_up, s_cap;
  __shared__ uint32_t s_issued;  // slices that this block's producer has issued
  __shared__ float s_block_scale[kScaleSlots][2];  // gated: the slice's gate and up blocks'

  const int n_stages = a.stages;
  uint8_t* stages = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* staging = stages + n_stages * kStageBytes;
  uint8_t* scale_ring = staging + kStagingBytes;
  Segment* segments = reinterpret_cast<Segment*>(scale_ring + kScaleSlots * kScaleSlotBytes);
  int* first = reinterpret_cast<int*>(segments + a.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Clusters of `splits` pairs; the block's place in its pair; the rank of the
  // pair's first block.
  const uint32_t place = cluster_rank(), leader = place & ~1u;
  const int rank = static_cast<int>(place & 1u), split = static_cast<int>(place / 2);
  const int splits = static_cast<int>(cluster_size() / 2);
  const int pair = blockIdx.x / (2 * splits), pairs = gridDim.x / (2 * splits);

  if (threadIdx.x == 0) {
    for (int i = 0; i < n_stages; ++i) {
      mbar_init(smem_addr(&s_full[i]), 1);
      mbar_init(smem_addr(&s_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&s_done[i]), 1);
      mbar_init(smem_addr(&s_free[i]), 2 * kEpiWarps);
    }
    for (int i = 0; i < kScaleChunks; ++i) {
      mbar_init(smem_addr(&s_scaled[i]), 2);
      mbar_init(smem_addr(&s_used[i]), kEpiWarps);
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
  if (warp == kEpiWarps + 1) tmem_alloc(smem_addr(&s_tmem), 512);
  pdl_wait();
  pdl_launch_dependents();

  const int width = static_cast<int>(kGatedForm ? a.N / 2 : a.N);
  const int m_blocks = (width + m_step<kUse>() - 1) / m_step<kUse>();
  const int groups = static_cast<int>((a.K + kGroupSlice - 1) / kGroupSlice);  // and slices
  for (int e = threadIdx.x; e < a.E; e += kQuantProductThreads) {
    bool bad;
    segments[e] = segment(a.offset, e, a.num_rows, &bad);
    if (bad && a.status != nullptr && blockIdx.x == 0)
      atomicOr(a.status, MOE_FLAG_OFFSET_OUT_OF_RANGE);
  }
  __syncthreads();
  if (warp == 0) {
    const int cap = scan_tiles(a.E, segments, first, splits > 1, m_blocks, groups, pairs);
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

  // A place in the ring of stages: stage and parity of the pass through them.
  struct Ring {
    int at = 0;
    uint32_t pass = 0;
    __device__ __forceinline__ void advance(int n) {
      if (++at == n) at = 0, pass ^= 1;
    }
  };
  // After a wait gave up: what was issued last at each stage is given the time of
  // one wait to be used up, so that nothing is in flight when the block ends.
  auto drain = [&](Ring r, uint32_t issued) {
    const unsigned long long t0 = now_ns();
    for (int i = 0; i < n_stages && static_cast<uint32_t>(i) < issued; ++i) {
      if (r.at == 0) r.at = n_stages, r.pass ^= 1;
      --r.at;
      while (!mbar_try(smem_addr(&s_empty[r.at]), r.pass) && now_ns() - t0 < kWaitNs) {
      }
    }
  };
  auto tile_at = [&](int t) {
    return find_tile<kUse>(a.E, segments, first, t, m_blocks, 0, 0, cap);
  };
  const int first_slice = groups * split / splits;
  const int n_slices = groups * (split + 1) / splits - first_slice;
  // Columns of a tile's product (each block holds half of B).
  auto mma_n = [](int cols) { return (cols + 15) / 16 * 16; };
  // First feature of the block's A tile.
  auto feature = [&](const Tile& t) { return t.m0 + rank * (m_step<kUse>() / 2); };

  if (warp >= kEpiWarps) {
    fewer_registers<kQuantOtherRegisters>();
    if (warp == kEpiWarps) {
      if (elect_one()) {
        Ring ring;
        uint32_t issued = 0;
        bool ok = true;
        const uint32_t full0 = cluster_addr(smem_addr(&s_full[0]), leader);
        for (Walk walk(pair, pairs); walk.t < total && ok; walk.next()) {
          const Tile tile = tile_at(walk.t);
          const int half_n = mma_n(tile.cols) / 2;
          const int b_boxes = (half_n + 63) / 64;
          const uint32_t bytes = kTileABytes + b_boxes * kBoxBytes;
          const int m = feature(tile), n = tile.lo + rank * half_n;
          for (int s = 0; s < n_slices; ++s, ++issued) {
            const int st = ring.at;
            if (withheld(issued) || !mbar_wait<false>(smem_addr(&s_empty[st]), ring.pass ^ 1, gave_up)) {
              ok = false;
              break;
            }
            *static_cast<volatile uint32_t*>(&s_issued) = issued + 1;
            ring.advance(n_stages);
            // Both blocks' loads report to the first block's barrier.
            const uint32_t full = full0 + st * 8;
            if (rank == 0) mbar_expect(smem_addr(&s_full[st]), 2 * bytes);
            const uint32_t sa = smem_addr(stages + st * kStageBytes);
            const int k = (first_slice + s) * kGroupSlice;
            if (kGatedForm) tma_load_5d(sa, &map_a, k, 0, 0, m / 8, tile.e, full);
            else tma_load_3d(sa, &map_a, k, m, tile.e, full);
            for (int i = 0; i < b_boxes; ++i)
              tma_load_2d(sa + kTileABytes + i * kBoxBytes, &map_b, k, n + i * 64, full);
          }
        }
        if (*gave_up != 0) drain(ring, issued);
      }
      __syncwarp();
    } else if (warp == kEpiWarps + 1) {
      if (rank == 0 && elect_one()) {
        Ring ring;
        uint32_t issued = 0;
        const uint16_t both = static_cast<uint16_t>(3u << leader);
        bool ok = true;
        for (Walk walk(pair, pairs); walk.t < total && ok; walk.next()) {
          const Tile tile = tile_at(walk.t);
          const uint32_t idesc = instr_desc(false, false, false, 256, mma_n(tile.cols));
          for (int s = 0; s < n_slices; ++s) {
            const uint32_t buf = issued & 1, acc = tmem + buf * kMaxN;
            const int st = ring.at;
            if (!mbar_wait<false>(smem_addr(&s_full[st]), ring.pass, gave_up) ||
                !mbar_wait<false>(smem_addr(&s_free[buf]), (issued / 2 & 1) ^ 1, gave_up)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t pa = smem_addr(stages + st * kStageBytes), pb = pa + kTileABytes;
#pragma unroll
            for (int i = 0; i < kGroupSlice / 32; ++i)
              tc_mma_fp8(acc, smem_desc(pa + i * 32, 16, 1024), smem_desc(pb + i * 32, 16, 1024),
                         idesc, i > 0);
            tc_commit(smem_addr(&s_done[buf]), both);
            tc_commit(smem_addr(&s_empty[st]), both);
            ++issued;
            ring.advance(n_stages);
          }
        }
        // The products are over before the memory they read and write is given up.
        if (*gave_up != 0) drain(ring, issued);
      }
      __syncwarp();
    } else {
      // Scales of the tile's columns lane + 32 i of this warp's half, kScaleChunk
      // slices of them in flight while those before are written.
      const int c0 = (warp - kEpiWarps - 2) * (kMaxN / 2);
      const int blocks = (width + kGroupSlice - 1) / kGroupSlice;
      const bool whole = groups % kScaleChunk == 0 && first_slice % kScaleChunk == 0 &&
                         (reinterpret_cast<uintptr_t>(a.scales) & 15) == 0;
      constexpr int kMine = kMaxN / 2 / 32;
      uint32_t step = 0;  // chunks so far
      bool ok = true;
      for (Walk walk(pair, pairs); walk.t < total && ok; walk.next()) {
        const Tile tile = tile_at(walk.t);
        const int64_t plane = static_cast<int64_t>(tile.e) * (kGatedForm ? 2 : 1) * blocks;
        const int block = min(feature(tile) / kGroupSlice, blocks - 1);
        const float* ws = a.weight_scales + (plane + block) * groups + first_slice;
        const float* rows = a.scales + static_cast<int64_t>(tile.lo + c0 + lane) * groups + first_slice;
        // w: lane k the block's scale of slice k of the chunk; gated, lane 4 + k the up
        // block's.
        float x[kMine][kScaleChunk], w;
        ws += lane % kScaleChunk;
        if (kGatedForm && lane / kScaleChunk == 1) ws += static_cast<int64_t>(blocks) * groups;
        auto fetch = [&](int s) {
          w = s + lane % kScaleChunk < n_slices ? __ldg(ws + s) : 0.f;
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            const float* at = rows + static_cast<int64_t>(32 * i) * groups + s;
            const bool in = c0 + lane + 32 * i < tile.cols;
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
          const int chunk = static_cast<int>(step % kScaleChunks);
          if (!warp_wait<false>(smem_addr(&s_used[chunk]), (step / kScaleChunks & 1) ^ 1, gave_up)) {
            ok = false;
            break;
          }
          const uint32_t to = smem_addr(scale_ring) + chunk * kScaleChunk * kScaleSlotBytes;
#pragma unroll
          for (int k = 0; k < kScaleChunk; ++k) {
            const float by = kGatedForm ? 1.f : __shfl_sync(kFullMask, w, k);
#pragma unroll
            for (int i = 0; i < kMine; ++i)
              shared_store_f(to + k * kScaleSlotBytes + (c0 + lane + 32 * i) * 4, x[i][k] * by);
          }
          if (kGatedForm && c0 == 0 && lane < 2 * kScaleChunk)
            s_block_scale[chunk * kScaleChunk + lane % kScaleChunk][lane / kScaleChunk] = w;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&s_scaled[chunk]));
          if (s + kScaleChunk < n_slices) fetch(s + kScaleChunk);
        }
      }
    }
  } else {
    more_registers<kQuantEpilogueRegisters>();
    const int quad = warp & 3, q = lane & 3;
    const uint32_t stage = smem_addr(staging + warp * kStagingWarpBytes);
    T* out = static_cast<T*>(a.out);
    T* residual = kGatedForm ? nullptr : static_cast<T*>(const_cast<void*>(a.residual));
    uint32_t done = 0, step = 0;  // slices and chunks of scales so far
    const uint32_t free0 = cluster_addr(smem_addr(&s_free[0]), leader);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    // The warp's 32 features, its columns c0 + 64 j + [0, 32).
    const int c0 = warp / 4 * 32;
    // Pairs that share a tile have one tile at most: its sums may lie over the
    // stages, which are through.  A lane's 32 values of block j: 8 steps of 512 bytes.
    const uint32_t part = smem_addr(stages + warp * 4 * 4096) + lane * 16;
    const uint32_t other_part = splits > 1 ? cluster_addr(part, 2 + rank) : 0;
    bool ok = true;
    for (Walk walk(pair, pairs); walk.t < total && ok; walk.next()) {
      const Tile tile = tile_at(walk.t);
      const int cols = tile.cols;
      uint64_t sums[4][16];  // z of block j: sums[j][8 h + 2 i + s], two columns each
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) sums[j][i] = 0;
      for (int s = 0; s < n_slices; ++s) {
        const int within = s % kScaleChunk, chunk = static_cast<int>(step % kScaleChunks);
        if (within == 0 && !warp_wait<false>(smem_addr(&s_scaled[chunk]), step / kScaleChunks & 1, gave_up)) {
          ok = false;
          break;
        }
        const int slot = chunk * kScaleChunk + within;
        const uint32_t scale = smem_addr(scale_ring) + slot * kScaleSlotBytes + (c0 + 2 * q) * 4;
        uint64_t by_gate = 0, by_up = 0;
        if (kGatedForm) {
          const float gate = s_block_scale[slot][0], up = s_block_scale[slot][1];
          by_gate = pack_f32x2(gate, gate), by_up = pack_f32x2(up, up);
        }
        const uint32_t buf = done & 1, acc = lanes + buf * kMaxN + c0;
        if (!warp_wait<false>(smem_addr(&s_done[buf]), done / 2 & 1, gave_up)) {
          ok = false;
          break;
        }
        ++done;
        tc_fence_after();
        // 16 lanes at a time, the next 16 being loaded meanwhile.
        float d[32];
        if (c0 < cols) tmem_load_16x32<0>(acc, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (c0 + 64 * j >= cols) break;
          uint64_t by0[4], by1[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = shared_load_f2(scale + (64 * j + 8 * i) * 4);
            const uint64_t xs = pack_f32x2(f.x, f.y);
            by0[i] = kGatedForm ? mul_f32x2(xs, by_gate) : xs;
            by1[i] = kGatedForm ? mul_f32x2(xs, by_up) : xs;
          }
          auto add = [&](int h) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float* v = d + 16 * h + 4 * i;
              uint64_t* z = &sums[j][8 * h + 2 * i];
              z[0] = fma_f32x2(pack_f32x2(v[0], v[1]), by0[i], z[0]);
              z[1] = fma_f32x2(pack_f32x2(v[2], v[3]), by1[i], z[1]);
            }
          };
          tmem_wait_load(d);
          tmem_load_16x32<16>(acc + 64 * j + (16u << 16), d);
          add(0);
          tmem_wait_load(d);
          if (j < 3 && c0 + 64 * (j + 1) < cols) tmem_load_16x32<0>(acc + 64 * (j + 1), d);
          add(1);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_relaxed_cluster(free0 + buf * 8);
          if (within == kScaleChunk - 1 || s == n_slices - 1) mbar_arrive(smem_addr(&s_used[chunk]));
        }
        if (within == kScaleChunk - 1 || s == n_slices - 1) ++step;
      }
      if (!ok) break;
      if (splits > 1) {
        if (split > 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (c0 + 64 * j >= cols) break;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 x = unpack_f32x2(sums[j][2 * i]), y = unpack_f32x2(sums[j][2 * i + 1]);
              shared_store16(part + j * 4096 + i * 512,
                             make_uint4(__float_as_uint(x.x), __float_as_uint(x.y),
                                        __float_as_uint(y.x), __float_as_uint(y.y)));
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_addr(&s_parts), rank));
          break;
        }
        if (!warp_wait<false>(smem_addr(&s_parts), 0, gave_up,
                       cluster_addr(smem_addr(&s_issued), 2 + rank)))
          break;
      }
      const int64_t m = feature(tile) + quad * (kGatedForm ? 16 : 32);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + 64 * j;
        if (c >= cols) break;
        const int64_t row = tile.lo + c;
        float z[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 x = unpack_f32x2(sums[j][i]);
          z[2 * i] = x.x, z[2 * i + 1] = x.y;
        }
        if (splits > 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 x = cluster_load4(other_part + j * 4096 + i * 512);
            z[4 * i] += x.x, z[4 * i + 1] += x.y, z[4 * i + 2] += x.z, z[4 * i + 3] += x.w;
          }
        }
        if (kGatedForm) {
          // z[16 h + 4 i + 2 s + b]: gate (s = 0) or up of feature 8 h + g, row 8 i + 2 q + b.
          float gate[16], up[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {  // k = 4 i + 2 h + b
            gate[k] = z[k / 2 % 2 * 16 + k / 4 * 4 + k % 2];
            up[k] = z[k / 2 % 2 * 16 + k / 4 * 4 + 2 + k % 2];
          }
          apply_act<16>(a.act, gate);
#pragma unroll
          for (int k = 0; k < 16; ++k) gate[k] *= up[k];
          write_half_block(gate, Block<T, 16>(out, width, row, cols - c, m, width, stage));
        } else {
          if (a.bias != nullptr) {
            const T* bias = static_cast<const T*>(a.bias) + static_cast<int64_t>(tile.e) * a.N;
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // z[16 h + 4 i + 2 s + b]: feature 16 h + 8 s + g
              const int64_t f = m + k * 8 + (lane >> 2);
              const float x = f < a.N ? to_f(bias[f]) : 0.f;
#pragma unroll
              for (int i = 0; i < 8; ++i) z[k / 2 * 16 + i / 2 * 4 + k % 2 * 2 + i % 2] += x;
            }
          }
          apply_act<32>(a.act, z);
          if (residual != nullptr) {
            uint4 r[4];
            const Block<T> b(residual, a.N, row, cols - c, m, a.N, stage);
            load_block(r, b);
            add_block(z, r, b);
          }
          write_block(z, Block<T>(out, a.N, row, cols - c, m, a.N, stage));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the products, loads, arrivals and reads of the cluster are over
  tc_fence_after();
  if (threadIdx.x == 0 && *gave_up != 0 && a.status != nullptr)
    atomicOr(a.status, MOE_FLAG_BARRIER_TIMEOUT);
  if (warp == kEpiWarps + 1) tmem_free(tmem, 512);
}

}  // namespace experts
}  // namespace moe
