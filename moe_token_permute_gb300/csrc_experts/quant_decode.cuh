// quant_decode.cuh -- the products of a few 8-bit rows (decoding): the weights of the
// experts that have rows are streamed once, and that is the time.
//
// The kernel is expert_decode.cuh's with 128 codes in the place of 64 values of 16 bits:
// the same ring, copies and reads, byte for byte.  A 128-byte line is a group of
// scales, and falls to one warp: four instructions of mma.sync m16n8k32 in sums of their
// own, which then join the task's, scaled.  int8 sums are whole numbers until the end.
// The 8-bit forms of mma.sync are slow on GB300, so all 16 rows of their A tile are used:
// a task of the linear product has two tiles of 8 features where it can, and an SM an
// even share of the tiles, one after another.  (2 rows of 8 x [14336 -> 4096], int8: with 8
// features a task 34 us, with the codes made fp16 for m16n8k16 32, here 27; 4.3 TB/s, and 6.1
// of 16384 features.  4-way dot products in the place of mma.sync: 26, but 12.4 instead of 11.4 from
// 4096.)  What bounds short contractions is the way of a task's sums to their results, so
// the warp that adds them up loads the next task's scales meanwhile and never sleeps (8 rows
// of 128 x [2048 -> 2 x 768] 14.4 -> 11.4 us, of 64 x [2048 -> 7168] 55 -> 35; with two such
// warps no better).
#pragma once

#include <type_traits>

#include "expert_decode.cuh"
#include "quant_product.cuh"

namespace moe {
namespace experts {

constexpr int kDecodeCodes = kDecodeBlocks * 128;  // of a stage
constexpr int kQuantDecodeGroups = 256;            // of rows; a call has no more than rows

// Which calls.  us from a graph, this kernel / tiles, on GB300 (experts x in -> features; the
// rows go to as many experts as there are, evenly, or z: by a Zipf law; weights not in L2):
//                                                  fp8                  int8
//   gated  128 x 1024 -> 768, 8, 32 rows           11.1 / 12.5          10.8 / 13.4, 27 / 26
//            256 rows, z                                                85 / 60, 55 / 35
//          128 x 2048 -> 768, 8, 16 rows           12.1 / 14.7, 19 / 16 11.9 / 19.1, 17 / 24
//            10, 12, 13 rows               14.2 / 15.3, 15.5 / 16.1, 16.3 / 15.1
//            32, 256 rows, z              32 / 30, 105 / 76, 69 / 43    28 / 41, 86 / 102, 57 / 57
//          128 x 2048 -> 1024, 1280, 8 rows        14.3 / 15.4, 16.5 / 15.2
//          64 x 7168 -> 2048, 8, 32 rows           44 / 44, 146 / 156   45 / 60, 151 / 212
//            256 rows, z                           287 / 279, 301 / 232 295 / 364, 306 / 312
//          8 x 4096 -> 14336, 2, 8, 64 rows   44 / 53, 149 / 147, 152 / 146   42 / 68, 143 / 186, 147 / 187
//          1 x 4096 -> 14336, 8, 16, 17 rows  26 / 26, 43 / 26, 62 / 27       25 / 38, 38 / 38, 59 / 38
//          1 x 2048 -> 6144, 8, 16, 24 rows   12.5 / 15.4, 18 / 15            11.6 / 17.6, 16 / 18, 21 / 18
//   linear 8 x 14336 -> 4096, 2, 8, 64 rows   26 / 36, 77 / 77, 79 / 77       27 / 52, 78 / 107, 79 / 108
//          8 x 4096 -> 4096, 2, 8, 64 rows    12.6 / 17, 30 / 28, 30 / 29     11.9 / 20, 28 / 38, 29 / 38
//          1 x 4096 -> 4096, 1, 16 rows       8.9 / 15.8, 11.5 / 16.7         8.8 / 18.8, 10.8 / 18.8
//            32, 64 rows                      16.4 / 16.8, 28 / 18            14.8 / 18.9, 24 / 20
//          1 x 4096 -> 14336, 8, 16, 24 rows  17 / 20, 26 / 20, 36 / 20       16 / 29, 22 / 29, 32 / 29
//          1 x 14336 -> 4096, 16, 32 rows     24 / 35, 37 / 35                23 / 50, 34 / 50
//          2 x 4096 -> 14336, 16, 24 rows     27 / 26, 46 / 26                26 / 38, 39 / 38
//          3 x 4096 -> 14336, 24, 32 rows     37 / 48, 66 / 48                35 / 67, 60 / 67
//          64 x 2048 -> 7168, 8, 16, 256 rows 35 / 30, 234 / 147              34 / 40, 61 / 56, 212 / 192
//          64 x 2048 -> 2048, 8, 10 rows      14.2 / 15.1, 16.8 / 14.7
//          128 x 2048 -> 2048, 32, 128 rows                                   38 / 41, 127 / 116
//          64 x 2816 -> 2048, 64 rows, 256 z                                  81 / 91, 83 / 71
//          128 x 768 -> 2048, 8, 256 rows     13.0 / 9.8, 127 / 44            12.1 / 12.6, 123 / 56
// A group of rows is one reading of its expert's weights, and a task costs about 0.7 us beside
// its loads.  int8 tiles spend their time on the codes, whatever the rows, so that int8 streams
// while rows are one reading of the weights on average, and contractions long; fp8 tiles
// stream as fast where there are enough of them for the SMs.
inline bool quant_decode_pays(bool fp8, bool gated, int64_t rows, int64_t E, int64_t K,
                              int64_t features) {
  if (K % 128 != 0 || rows > kQuantDecodeGroups) return false;
  const int64_t used = std::min(E, rows);
  const int64_t groups = used + (rows - used) / kDecodeGroup;  // about
  // Of the tiled kernel, if every group had its own.
  const int64_t tiles = groups * ((features + (gated ? 127 : 255)) / (gated ? 128 : 256));
  if (fp8)
    return rows <= kDecodeMaxRows && ((K >= 4096 && rows <= std::max<int64_t>(8, 4 * E)) ||
                                      (K >= 1024 && tiles <= 64));
  const int64_t contraction = (gated ? 2 : 1) * K;  // of a task
  if (contraction < 2048) return false;
  if (rows > kDecodeGroup * E)
    return rows <= kDecodeMaxRows && (tiles <= 96 || (K >= 4096 && rows <= 2 * kDecodeGroup));
  return contraction >= 2816 || tiles <= 256;
}

__device__ __forceinline__ void mma_16832(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16832(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// map: the weight as [E, K/128, N, 128], tiles of kDecodeBlocks x 8 x 128.
template <typename T, bool kFp8, bool kGatedForm>
__global__ void __launch_bounds__(kDecodeThreads, 1)
k_quant_decode(const __grid_constant__ CUtensorMap map, const QuantArgs a) {
  using Sum = typename std::conditional<kFp8, float, int>::type;
  const uint8_t* x = static_cast<const uint8_t*>(a.codes);
  using Shape = DecodeShape<true>;
  constexpr int kRing = Shape::kRing;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_full[kRing], s_empty[kRing], s_sums[2], s_read[2];
  __shared__ int s_gave_up, s_scan[32];
  __shared__ uint32_t s_issued;  // stages that the producer has issued
  __shared__ DecodeGroup s_groups[kQuantDecodeGroups];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Sum* parts = reinterpret_cast<Sum*>(ring + kRing * Shape::kStageBytes);
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
    for (int lo = s.lo; lo < s.hi && at < kQuantDecodeGroups; lo += kDecodeGroup, ++at)
      s_groups[at] = {e, lo, min(kDecodeGroup, s.hi - lo)};
    groups += part;
  }
  groups = min(groups, kQuantDecodeGroups);
  if (bad && a.status != nullptr && blockIdx.x == 0)
    atomicOr(a.status, MOE_FLAG_OFFSET_OUT_OF_RANGE);
  __syncthreads();

  const int F = static_cast<int>(kGatedForm ? a.N / 2 : a.N);
  const int per_group = F / kDecodeFeatures;  // F is a multiple of 8
  // The block's tasks: its share of the tiles of 8 features, group by group; two at a time
  // in the linear product.
  struct Task {
    int group, part, tiles, left;  // `left` ahead of the task's own
  };
  const int64_t all = static_cast<int64_t>(groups) * per_group;
  const int64_t begin = all * blockIdx.x / gridDim.x, end = all * (blockIdx.x + 1) / gridDim.x;
  auto take = [&](Task& t) {
    t.tiles = kGatedForm ? min(1, t.left) : min(min(2, per_group - t.part), t.left);
  };
  Task start = {static_cast<int>(begin / per_group), static_cast<int>(begin % per_group), 0,
                static_cast<int>(end - begin)};
  take(start);
  auto advance = [&](Task& t) {
    t.left -= t.tiles;
    t.part += t.tiles;
    if (t.part == per_group) t.part = 0, ++t.group;
    take(t);
  };
  const int K = static_cast<int>(a.K);
  const int n_slices = (K + kDecodeCodes - 1) / kDecodeCodes;
  const int scale_groups = K / kGroupSlice;  // K is a multiple of 128
  const int blocks = (F + kGroupSlice - 1) / kGroupSlice;
  volatile int* gave_up = &s_gave_up;
  if (warp == kDecodeWarps) {
    if (elect_one()) {
      int step = 0;
      bool ok = true;
      for (Task t = start; t.left > 0 && ok; advance(t)) {
        const DecodeGroup task = s_groups[t.group];
        const int f0 = t.part * kDecodeFeatures;
        const uint8_t* rows = x + static_cast<int64_t>(task.lo) * a.K;
        for (int s = 0; s < n_slices; ++s, ++step) {
          const int st = step % kRing;
          const uint32_t full = smem_addr(&s_full[st]);
          if (withheld(step) ||
              !mbar_wait_as<kWaitAwake>(smem_addr(&s_empty[st]), (step / kRing & 1) ^ 1, gave_up)) {
            ok = false;
            break;
          }
          *static_cast<volatile uint32_t*>(&s_issued) = step + 1;
          const int k = s * kDecodeCodes;
          const uint32_t bytes = min(kDecodeCodes, K - k);
          mbar_expect(full, (kGatedForm ? 2 : t.tiles) * kDecodeTileBytes + task.rows * bytes);
          uint32_t dst = smem_addr(ring + st * Shape::kStageBytes);
          tma_load_4d_single(dst, &map, 0, f0, s * kDecodeBlocks, task.e, full);
          dst += kDecodeTileBytes;
          if (kGatedForm || t.tiles > 1)
            tma_load_4d_single(dst, &map, 0, (kGatedForm ? F : kDecodeFeatures) + f0,
                               s * kDecodeBlocks, task.e, full);
          dst += kDecodeTileBytes;
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
    for (Task t = start; t.left > 0 && ok; advance(t), ++turn) {
      const DecodeGroup task = s_groups[t.group];
      const int rows = task.rows;
      const bool second = kGatedForm || t.tiles > 1;
      // fp8: scales of rows 2 q and 2 q + 1 of x, and of the blocks of the tiles' features.
      const float* xs[2];
      const float *ws = nullptr, *us = nullptr;
      if (kFp8) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          xs[i] = a.scales + static_cast<int64_t>(task.lo + min(2 * q + i, rows - 1)) * scale_groups;
        ws = a.weight_scales +
             (static_cast<int64_t>(task.e) * (kGatedForm ? 2 : 1) * blocks +
              t.part * kDecodeFeatures / kGroupSlice) * scale_groups;
        const int next = kGatedForm ? blocks
                                    : (t.part + t.tiles - 1) * kDecodeFeatures / kGroupSlice -
                                          t.part * kDecodeFeatures / kGroupSlice;
        us = ws + static_cast<int64_t>(next) * scale_groups;
      }
      Sum acc[kDecodeStep][4] = {};  // int8: chains of their own; fp8: blocks i and i + 1 in turn
      for (int s = 0; s < n_slices; ++s, ++step) {
        if ((step & 1) != warp / kDecodeSet) continue;
        const int st = step % kRing;
        float by[kDecodeStep / 2][4];  // of block i, for the sums' four numbers
        if (kFp8) {
#pragma unroll
          for (int i = 0; i < kDecodeStep / 2; ++i) {
            const int b = s * kDecodeBlocks + i * kDecodeSet + warp % kDecodeSet;
            const int k = min(b, scale_groups - 1);
            const bool in = b < scale_groups;  // (no scale but 0 behind: it may be infinite)
            const float w = in ? __ldg(ws + k) : 0.f, u = in ? __ldg(us + k) : 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float v = in ? __ldg(xs[j] + k) : 0.f;
              by[i][j] = v * w, by[i][2 + j] = v * u;
            }
          }
        }
        if (!warp_wait_as<kWaitAwake>(smem_addr(&s_full[st]), step / kRing & 1, gave_up)) {
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
          w[i] = second ? *reinterpret_cast<const uint4*>(at + kDecodeTileBytes) : zero;
          // Behind K the weights' tile is zero; the rows of x, there and behind
          // the last row, are older values.
          u[i] = g < rows && s * kDecodeCodes + b * 128 + c * 16 < K
                     ? *reinterpret_cast<const uint4*>(stage + Shape::kTiles * kDecodeTileBytes +
                                                       g * kDecodePitch + b * 128 + c * 16)
                     : zero;
        }
        if (kFp8) {
#pragma unroll
          for (int i = 0; i < kDecodeStep; i += 2) {
            Sum part[2][4] = {};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              mma_16832(part[j], v[i + j].x, w[i + j].x, v[i + j].y, w[i + j].y, u[i + j].x, u[i + j].y);
              mma_16832(part[j], v[i + j].z, w[i + j].z, v[i + j].w, w[i + j].w, u[i + j].z, u[i + j].w);
            }
            // (a block behind K has zeros)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] += (part[0][j] + part[1][j]) * by[i / 2][j];
          }
        } else {
#pragma unroll
          for (int i = 0; i < kDecodeStep; ++i) {
            mma_16832(acc[i], v[i].x, w[i].x, v[i].y, w[i].y, u[i].x, u[i].y);
            mma_16832(acc[i], v[i].z, w[i].z, v[i].w, w[i].w, u[i].z, u[i].w);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&s_empty[st]));
      }
      if (!ok) break;
      const int buf = turn & 1;
      if (!warp_wait_as<kWaitAwake>(smem_addr(&s_read[buf]), (turn / 2 & 1) ^ 1, gave_up)) break;
      Sum* part = parts + buf * Shape::kPartFloats + warp * Shape::kWarpPitch +
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
    int turn = 0;
    // Value j of the lane: feature and row (j * 32 + lane) of the task.
    constexpr int kValues = kDecodeFeatures * kDecodeGroup / 32;
    const int f = lane % kDecodeFeatures, r0 = lane / kDecodeFeatures;
    // int8: scales of a task's two channels and of its rows; a task's are loaded while the
    // one before is summed.
    float w = 0.f, u = 0.f, xs[kValues] = {};
    auto fetch = [&](const Task& t) {
      if (kFp8 || t.left <= 0) return;
      const DecodeGroup task = s_groups[t.group];
      const float* ws = a.weight_scales + static_cast<int64_t>(task.e) * a.N +
                        t.part * kDecodeFeatures + f;
      w = __ldg(ws);
      u = kGatedForm ? __ldg(ws + F) : t.tiles > 1 ? __ldg(ws + kDecodeFeatures) : 0.f;
#pragma unroll
      for (int j = 0; j < kValues; ++j)
        xs[j] = __ldg(a.scales + task.lo + min(r0 + j * (32 / kDecodeFeatures), task.rows - 1));
    };
    fetch(start);
    for (Task t = start, next; t.left > 0; t = next, ++turn) {
      next = t;
      advance(next);
      const DecodeGroup task = s_groups[t.group];
      const int buf = turn & 1;
      const int c = t.part * kDecodeFeatures + f;
      // (spans a task's contraction)
      if (!warp_wait_as<kWaitAwake>(smem_addr(&s_sums[buf]), turn / 2 & 1, gave_up,
                                    smem_addr(&s_issued)))
        break;
      float by[kValues], by_up[kValues];
#pragma unroll
      for (int j = 0; j < kValues; ++j) by[j] = xs[j] * w, by_up[j] = xs[j] * u;
      fetch(next);
      Sum z[kValues], up[kValues];
#pragma unroll
      for (int j = 0; j < kValues; ++j) {
        const Sum* part = parts + buf * Shape::kPartFloats + f * Shape::kRowPitch + r0 +
                          j * (32 / kDecodeFeatures);
        z[j] = up[j] = 0;
#pragma unroll
        for (int k = 0; k < kDecodeWarps; ++k) {
          z[j] += part[k * Shape::kWarpPitch];
          up[j] += part[k * Shape::kWarpPitch + kDecodeFeatures * Shape::kRowPitch];
        }
      }
      // Before the results are stored: an arrival waits until the stores before
      // it are performed, 1500 cycles.
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&s_read[buf]));
#pragma unroll
      for (int j = 0; j < kValues; ++j) {
        const int r = r0 + j * (32 / kDecodeFeatures);
        if (r >= task.rows) break;
        const int64_t row = task.lo + r;
        const float v = kFp8 ? z[j] : static_cast<float>(z[j]) * by[j];
        const float y = kFp8 ? up[j] : static_cast<float>(up[j]) * by_up[j];
        if (kGatedForm) {
          out[row * F + c] = from_f<T>(act_of(a.act, v) * y);
        } else {
          auto store = [&](float z, int64_t f) {
            if (a.bias != nullptr)
              z += to_f(static_cast<const T*>(a.bias)[static_cast<int64_t>(task.e) * a.N + f]);
            z = act_of(a.act, z);
            if (a.residual != nullptr)
              z += to_f(static_cast<const T*>(a.residual)[row * a.N + f]);
            out[row * a.N + f] = from_f<T>(z);
          };
          store(v, c);
          if (t.tiles > 1) store(y, c + kDecodeFeatures);
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
