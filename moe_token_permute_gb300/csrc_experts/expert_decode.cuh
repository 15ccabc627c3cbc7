// expert_decode.cuh -- the forward products of a few rows (decoding): the
// weights of the experts that have rows are streamed once, and that is the time.
//
// The tiles of expert_product.cuh are 128 or 256 features of a pair of SMs: eight
// experts' 2 x 768 features make 48 of them.  Here the work is cut into tasks of 8
// features (8 weight rows; gated: 8 gate and 8 up rows) times up to 8 rows of x, and
// each SM takes every 152nd task (768 in that example).
//
//   warps 0-15  consumers: two sets of 8 take turns with the stages, the warps
//               of a set share the stage's part of the contraction
//   warp 16     producer
//   warp 17     adds the 16 partial sums up, epilogue
// Everything comes through one ring per SM that runs on from task to task, so
// loads never pause (96 or 128 KB of weights in flight); the sums of a task are
// joined while the next is computed.  A stage's weights are one TMA tile (gated: two) of
// 64 x 8 rows x 16 values, K being read as K/64 blocks: a copy per row instead kept
// the producer at 84 cycles a copy, and the memory at 5.4 of 6.7 TB/s.  Rows of x,
// few, are bulk copies 64 bytes apart modulo 128, and the tiles are in the 128-byte
// swizzle, so that a quarter warp's reads of two rows fall into different banks.
//
// A warp multiplies with mma.sync m16n8k16, which costs nothing beside the
// loads; tcgen05's smallest tile is 64 weight rows.  The sum over k may be taken
// in any order, so the fragments are not loaded in the instruction's own k
// order: lane (g, q) loads 16 consecutive bytes (8 k-values) of weight row g and
// of row g of x, first the even and then the odd ones of a line of 128, and two
// instructions take two words of each.  Gated: rows 8-15 of the instruction's tile
// are the up rows, so that a thread has both of a feature; linear: they are zero
// (16 features per task would balance worse).
// On GB300: 2 rows of 8 x [14336 -> 4096] 38.8 us, 6.1 TB/s (90% of the measured copy
// bandwidth); 8 rows of 128 x [2048 -> 2 x 768] 14.8 us for 7.5 us of weights: 5.05
// tasks per SM are 6 rounds, and about 4 us pass before the first loads arrive.
#pragma once

#include <algorithm>

#include "expert_product.cuh"

namespace moe {
namespace experts {

constexpr int kDecodeWarps = 16;
constexpr int kDecodeThreads = (kDecodeWarps + 2) * 32;
constexpr int kDecodeFeatures = 8;               // of a task
constexpr int kDecodeGroup = 8;                  // rows of x of a task
constexpr int kDecodeSlice = 1024;               // k-values of a stage
constexpr int kDecodeBlocks = kDecodeSlice / 64;  // of 64 k-values
constexpr int kDecodeTileBytes = kDecodeFeatures * kDecodeSlice * 2;
constexpr int kDecodePitch = kDecodeSlice * 2 + 64;  // of the rows of x
constexpr int kDecodeSet = kDecodeWarps / 2;     // warps of one stage
constexpr int kDecodeStep = kDecodeSlice / 32 / kDecodeSet;  // 32-value pieces of a warp

template <bool kGatedForm>
struct DecodeShape {
  static constexpr int kTiles = kGatedForm ? 2 : 1;  // of 8 weight rows
  static constexpr int kRing = kGatedForm ? 4 : 6;
  static constexpr int kStageBytes =
      (kTiles * kDecodeTileBytes + kDecodeGroup * kDecodePitch + 1023) / 1024 * 1024;
  // Partial sums of a task: [warp][weight row][row of x].
  static constexpr int kRowPitch = kDecodeGroup + 1;
  static constexpr int kWarpPitch = kTiles * kDecodeFeatures * kRowPitch;
  static constexpr int kPartFloats = kDecodeWarps * kWarpPitch;
  // Dynamic shared memory: ring, two sets of partial sums.
  static constexpr size_t kSmem =
      1024 + static_cast<size_t>(kRing) * kStageBytes + 2 * kPartFloats * 4;
  static_assert(kSmem + 2048 <= 227 * 1024, "shared memory of one block");
};

// Rows up to which these kernels are used; a call has no more groups than rows.
constexpr int kDecodeMaxRows = 32;

// Which calls.  us from a graph, this kernel / large tiles, on GB300 (E experts, in ->
// features; the rows go to as many experts as there are; weights not in L2):
//   gated 64 x 7168 -> 2048, 8 / 16 / 32 rows    70 / 84    132 / 150   257 / 275
//   gated 8 x 4096 -> 14336, 2 / 8 / 32 rows     69 / 74    257 / 304   258 / 271
//   gated 128 x 2048 -> 768, 8 / 16 / 32 rows  14.8 / 16.9  22.6 / 25.6  39 / 37
//   gated 128 x 1984 -> 768, 8 / 16 rows       14.4 / 17.2  22.5 / 24.9
//   linear 8 x 14336 -> 4096, 2 / 8 / 32 rows    39 / 45    136 / 147   137 / 148
//   linear 8 x 4096 -> 4096, 2 / 8 rows        15.8 / 17.3  46.3 / 48.1
//   linear 8 x 4032 -> 4096, 2 / 8 rows        16.0 / 17.0  46.3 / 45.5
//   linear 1 x 4096 -> 4096, 1 / 8 / 16 rows   11.1 / 14.1  12.3 / 13.5  17.9 / 13.5
//   linear 64 x 2048 -> 7168, 8 rows             73 / 40
//   linear 128 x 768 -> 2048, 8 / 32 rows        23 / 10     78 / 25
// A task costs about 0.7 us beside its loads, so its weights have to be long; more
// than 8 rows of one expert read its weights again.  The steps are at 2048 and 4096
// inputs gated, 4096 and 8192 linear; just below the lower one (1984, 4032) the large
// tiles are taken, which costs up to 16%.
inline bool decode_pays(bool gated, int64_t rows, int64_t E, int64_t K) {
  const int64_t task_bytes = (gated ? 2 : 1) * kDecodeFeatures * K * 2;
  const int64_t most = task_bytes >= 128 * 1024  ? kDecodeMaxRows
                       : task_bytes >= 64 * 1024 ? kDecodeMaxRows / 2
                                                 : 0;
  return rows <= std::min<int64_t>(most, kDecodeGroup * E) && K % 64 == 0;
}

template <typename T>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma_16816<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1,
                                                  uint32_t a2, uint32_t a3, uint32_t b0,
                                                  uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma_16816<__half>(float (&c)[4], uint32_t a0, uint32_t a1,
                                                  uint32_t a2, uint32_t a3, uint32_t b0,
                                                  uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float act_of(int a, float z) {
  if (a == MOE_ACT_SILU) return act<MOE_ACT_SILU>(z);
  if (a == MOE_ACT_GELU) return act<MOE_ACT_GELU>(z);
  if (a == MOE_ACT_RELU) return act<MOE_ACT_RELU>(z);
  return z;
}

// Up to kDecodeGroup rows of x of one expert.
struct DecodeGroup {
  int e, lo, rows;
};

// map: the weight as [E, K/64, N, 64], tiles of kDecodeBlocks x 8 x 64.
template <typename T, bool kGatedForm>
__global__ void __launch_bounds__(kDecodeThreads, 1)
k_expert_decode(const __grid_constant__ CUtensorMap map, const T* __restrict__ x,
                const ProductArgs a) {
  using Shape = DecodeShape<kGatedForm>;
  constexpr int kRing = Shape::kRing;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_full[kRing], s_empty[kRing], s_sums[2], s_read[2];
  __shared__ int s_gave_up, s_scan[32];
  __shared__ uint32_t s_issued;  // stages that the producer has issued
  __shared__ DecodeGroup s_groups[kDecodeMaxRows];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* parts = reinterpret_cast<float*>(ring + kRing * Shape::kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    s_gave_up = 0;
    s_issued = 0;
    for (int i = 0; i < kRing; ++i) {
      mbar_init(smem_addr(&s_full[i]), 1);
      mbar_init(smem_addr(&s_empty[i]), kDecodeSet);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&s_sums[i]), kDecodeWarps);
      mbar_init(smem_addr(&s_read[i]), 1);
    }
    mbar_init_fence();
    tma_prefetch_map(&map);
  }
  pdl_wait();
  pdl_launch_dependents();
  int groups = 0;
  bool bad = false;
  for (int e0 = 0; e0 < a.E; e0 += kDecodeThreads) {
    const int e = e0 + threadIdx.x;
    Segment s = {0, 0};
    if (e < a.E) {
      bool b;
      s = segment(a.offset, e, a.num_rows, &b);
      bad |= b;
    }
    int part;
    int at = groups + block_exclusive_sum((s.hi - s.lo + kDecodeGroup - 1) / kDecodeGroup, s_scan,
                                          &part);
    // Segments that overlap (bad offsets) could make more groups than rows.
    for (int lo = s.lo; lo < s.hi && at < kDecodeMaxRows; lo += kDecodeGroup, ++at)
      s_groups[at] = {e, lo, min(kDecodeGroup, s.hi - lo)};
    groups += part;
  }
  groups = min(groups, kDecodeMaxRows);
  if (bad && a.status != nullptr && blockIdx.x == 0)
    atomicOr(a.status, MOE_FLAG_OFFSET_OUT_OF_RANGE);
  __syncthreads();

  const int F = static_cast<int>(kGatedForm ? a.N / 2 : a.N);
  const int per_group = F / kDecodeFeatures;  // F is a multiple of 8
  // The block's tasks: t = blockIdx.x, blockIdx.x + gridDim.x, ... as (group,
  // features), without a division.
  struct Task {
    int group, part;
  };
  const Task start = {static_cast<int>(blockIdx.x) / per_group,
                      static_cast<int>(blockIdx.x) % per_group};
  auto advance = [&](Task& t) {
    t.part += gridDim.x;
    while (t.part >= per_group) t.part -= per_group, ++t.group;
  };
  const int K = static_cast<int>(a.K);
  const int n_slices = (K + kDecodeSlice - 1) / kDecodeSlice;
  volatile int* gave_up = &s_gave_up;
  if (warp == kDecodeWarps) {
    if (elect_one()) {
      int step = 0;
      bool ok = true;
      for (Task t = start; t.group < groups && ok; advance(t)) {
        const DecodeGroup task = s_groups[t.group];
        const int f0 = t.part * kDecodeFeatures;
        const T* rows = x + static_cast<int64_t>(task.lo) * a.K;
        for (int s = 0; s < n_slices; ++s, ++step) {
          const int st = step % kRing;
          const uint32_t full = smem_addr(&s_full[st]);
          if (withheld(step) ||
              !mbar_wait(smem_addr(&s_empty[st]), (step / kRing & 1) ^ 1, gave_up)) {
            ok = false;
            break;
          }
          *static_cast<volatile uint32_t*>(&s_issued) = step + 1;
          const int k = s * kDecodeSlice;
          const uint32_t bytes = min(kDecodeSlice, K - k) * 2;
          mbar_expect(full, Shape::kTiles * kDecodeTileBytes + task.rows * bytes);
          uint32_t dst = smem_addr(ring + st * Shape::kStageBytes);
          tma_load_4d_single(dst, &map, 0, f0, s * kDecodeBlocks, task.e, full);
          dst += kDecodeTileBytes;
          if (kGatedForm) {
            tma_load_4d_single(dst, &map, 0, F + f0, s * kDecodeBlocks, task.e, full);
            dst += kDecodeTileBytes;
          }
          for (int i = 0; i < task.rows; ++i, dst += kDecodePitch)
            bulk_load(dst, rows + i * a.K + k, bytes, full);
        }
      }
      if (*gave_up != 0) {  // no copy may be in flight when the block ends
        const unsigned long long t0 = now_ns();
        for (int i = 1; i <= kRing && i <= step; ++i)
          while (!mbar_try(smem_addr(&s_full[(step - i) % kRing]),
                           (step - i) / kRing & 1) &&
                 now_ns() - t0 < kWaitNs) {
          }
      }
    }
    __syncwarp();
  } else if (warp < kDecodeWarps) {
    const int g = lane >> 2, q = lane & 3;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    int step = 0, turn = 0;
    bool ok = true;
    for (Task t = start; t.group < groups && ok; advance(t), ++turn) {
      const int rows = s_groups[t.group].rows;
      float acc[kDecodeStep][4] = {};  // chains of their own: an instruction takes 100 cycles
      for (int s = 0; s < n_slices; ++s, ++step) {
        if ((step & 1) != warp / kDecodeSet) continue;
        const int st = step % kRing;
        if (!warp_wait(smem_addr(&s_full[st]), step / kRing & 1, gave_up)) {
          ok = false;
          break;
        }
        const uint8_t* stage = ring + st * Shape::kStageBytes;
        uint4 v[kDecodeStep], w[kDecodeStep], u[kDecodeStep];
#pragma unroll
        for (int i = 0; i < kDecodeStep; ++i) {
          // Piece i: block b, 16-byte chunk c of its 128 bytes.
          const int b = i / 2 * kDecodeSet + warp % kDecodeSet, c = 2 * q + (i & 1);
          const uint8_t* at = stage + (b * 8 + g) * 128 + ((c ^ g) << 4);
          v[i] = *reinterpret_cast<const uint4*>(at);
          w[i] = kGatedForm ? *reinterpret_cast<const uint4*>(at + kDecodeTileBytes) : zero;
          // Behind K the weights' tile is zero; the rows of x, there and behind
          // the last row, are older values.
          u[i] = g < rows && s * kDecodeSlice + b * 64 + c * 8 < K
                     ? *reinterpret_cast<const uint4*>(stage + Shape::kTiles * kDecodeTileBytes +
                                                       g * kDecodePitch + b * 128 + c * 16)
                     : zero;
        }
#pragma unroll
        for (int i = 0; i < kDecodeStep; ++i) {
          mma_16816<T>(acc[i], v[i].x, w[i].x, v[i].y, w[i].y, u[i].x, u[i].y);
          mma_16816<T>(acc[i], v[i].z, w[i].z, v[i].w, w[i].w, u[i].z, u[i].w);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&s_empty[st]));
      }
      if (!ok) break;
      const int buf = turn & 1;
      if (!warp_wait(smem_addr(&s_read[buf]), (turn / 2 & 1) ^ 1, gave_up)) break;
      float* part = parts + buf * Shape::kPartFloats + warp * Shape::kWarpPitch +
                    g * Shape::kRowPitch + q * 2;
      static_assert(kDecodeStep == 4, "the sum below");
#pragma unroll
      for (int i = 0; i < 2 * Shape::kTiles; ++i)
        part[i / 2 * kDecodeFeatures * Shape::kRowPitch + i % 2] =
            (acc[0][i] + acc[1][i]) + (acc[2][i] + acc[3][i]);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&s_sums[buf]));
    }
  } else {
    T* out = static_cast<T*>(a.out);
    T* preact = static_cast<T*>(a.preact);
    int turn = 0;
    for (Task t = start; t.group < groups; advance(t), ++turn) {
      const DecodeGroup task = s_groups[t.group];
      const int buf = turn & 1;
      // (spans a task's contraction)
      if (!warp_wait(smem_addr(&s_sums[buf]), turn / 2 & 1, gave_up, smem_addr(&s_issued))) break;
      // Value j of the lane: feature and row (j * 32 + lane) of the task.
      constexpr int kValues = kDecodeFeatures * kDecodeGroup / 32;
      const int f = lane % kDecodeFeatures, r0 = lane / kDecodeFeatures;
      float z[kValues], up[kValues];
#pragma unroll
      for (int j = 0; j < kValues; ++j) {
        const float* part = parts + buf * Shape::kPartFloats + f * Shape::kRowPitch + r0 +
                            j * (32 / kDecodeFeatures);
        z[j] = up[j] = 0.f;
#pragma unroll
        for (int k = 0; k < kDecodeWarps; ++k) {
          z[j] += part[k * Shape::kWarpPitch];
          if (kGatedForm) up[j] += part[k * Shape::kWarpPitch + kDecodeFeatures * Shape::kRowPitch];
        }
      }
      // Before the results are stored: an arrival waits until the stores before
      // it are performed, 1500 cycles.
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&s_read[buf]));
      const int c = t.part * kDecodeFeatures + f;
#pragma unroll
      for (int j = 0; j < kValues; ++j) {
        const int r = r0 + j * (32 / kDecodeFeatures);
        if (r >= task.rows) break;
        const int64_t row = task.lo + r;
        float v = z[j];
        if (kGatedForm) {
          if (preact != nullptr) {
            preact[row * a.N + c] = from_f<T>(v);
            preact[row * a.N + F + c] = from_f<T>(up[j]);
          }
          out[row * F + c] = from_f<T>(act_of(a.act, v) * up[j]);
        } else {
          if (a.bias != nullptr)
            v += to_f(static_cast<const T*>(a.bias)[static_cast<int64_t>(task.e) * a.N + c]);
          if (preact != nullptr) preact[row * a.N + c] = from_f<T>(v);
          v = act_of(a.act, v);
          if (a.residual != nullptr)
            v += to_f(static_cast<const T*>(a.residual)[row * a.N + c]);
          out[row * a.N + c] = from_f<T>(v);
        }
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && *gave_up != 0 && a.status != nullptr)
    atomicOr(a.status, MOE_FLAG_BARRIER_TIMEOUT);
}

}  // namespace experts
}  // namespace moe
