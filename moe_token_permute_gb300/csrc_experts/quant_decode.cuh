// quant_decode.cuh -- the products of a few 8-bit rows (decoding): the weights of the
// experts that have rows are streamed once, and that is the time.
//
// The kernel is expert_decode.cuh's with 128 codes in the place of 64 values of 16 bits:
// the same tasks, ring, copies and reads, byte for byte.  Both kinds of codes become fp16,
// which holds them exactly, and go through mma.sync m16n8k16: the 8-bit forms of mma.sync
// are too slow on GB300 to keep up with the loads (2 rows of 8 x [14336 -> 4096]: int8
// 34 us at 81% of that pipe, fp8 31).  A 128-byte line is a group of scales, and falls to
// one warp: its products go to sums of their own, which then join the task's, scaled.
#pragma once

#include "expert_decode.cuh"
#include "int8_product.cuh"

namespace moe {
namespace experts {

constexpr int kDecodeCodes = kDecodeBlocks * 128;  // of a stage

// Which calls: see decode_pays.
inline bool quant_decode_pays(bool gated, int64_t rows, int64_t E, int64_t K) {
  const int64_t task_bytes = (gated ? 2 : 1) * kDecodeFeatures * K;
  const int64_t most = task_bytes >= 64 * 1024   ? kDecodeMaxRows
                       : task_bytes >= 32 * 1024 ? kDecodeMaxRows / 2
                                                 : 0;
  return rows <= std::min<int64_t>(most, kDecodeGroup * E) && K % 128 == 0;
}

// 4 codes as fp16, two in each register.
template <bool kFp8>
__device__ __forceinline__ uint2 widen(uint32_t c) {
  if (!kFp8) return codes_to_fp16(c);
  uint2 r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(c));
  return r;
}
// 4 codes of 8 (gated: 16) weight rows and of 8 rows of x.
template <bool kFp8, bool kGatedForm>
__device__ __forceinline__ void multiply_codes(float (&c)[4], uint32_t v, uint32_t w, uint32_t u) {
  const uint2 a = widen<kFp8>(v), x = widen<kFp8>(u);
  const uint2 b = kGatedForm ? widen<kFp8>(w) : make_uint2(0, 0);
  mma_16816<__half>(c, a.x, b.x, a.y, b.y, x.x, x.y);
}

// map: the weight as [E, K/128, N, 128], tiles of kDecodeBlocks x 8 x 128.
template <typename T, bool kFp8, bool kGatedForm>
__global__ void __launch_bounds__(kDecodeThreads, 1)
k_quant_decode(const __grid_constant__ CUtensorMap map, const QuantArgs a) {
  const uint8_t* x = static_cast<const uint8_t*>(a.codes);
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
  const int n_slices = (K + kDecodeCodes - 1) / kDecodeCodes;
  const int scale_groups = K / kGroupSlice;  // K is a multiple of 128
  const int blocks = (F + kGroupSlice - 1) / kGroupSlice;
  volatile int* gave_up = &s_gave_up;
  if (warp == kDecodeWarps) {
    if (elect_one()) {
      int step = 0;
      bool ok = true;
      for (Task t = start; t.group < groups && ok; advance(t)) {
        const DecodeGroup task = s_groups[t.group];
        const int f0 = t.part * kDecodeFeatures;
        const uint8_t* rows = x + static_cast<int64_t>(task.lo) * a.K;
        for (int s = 0; s < n_slices; ++s, ++step) {
          const int st = step % kRing;
          const uint32_t full = smem_addr(&s_full[st]);
          if (withheld(step) ||
              !mbar_wait(smem_addr(&s_empty[st]), (step / kRing & 1) ^ 1, gave_up)) {
            ok = false;
            break;
          }
          *static_cast<volatile uint32_t*>(&s_issued) = step + 1;
          const int k = s * kDecodeCodes;
          const uint32_t bytes = min(kDecodeCodes, K - k);
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
      const DecodeGroup task = s_groups[t.group];
      const int rows = task.rows;
      // fp8: scales of rows 2 q and 2 q + 1 of x, and of the task's block of features.
      const float* xs[2];
      const float* ws = nullptr;
      if (kFp8) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          xs[i] = a.scales + static_cast<int64_t>(task.lo + min(2 * q + i, rows - 1)) * scale_groups;
        ws = a.weight_scales +
             (static_cast<int64_t>(task.e) * (kGatedForm ? 2 : 1) * blocks +
              t.part * kDecodeFeatures / kGroupSlice) * scale_groups;
      }
      float acc[kDecodeStep][4] = {};  // int8: chains of their own; fp8: blocks i and i + 1 in turn
      for (int s = 0; s < n_slices; ++s, ++step) {
        if ((step & 1) != warp / kDecodeSet) continue;
        const int st = step % kRing;
        float by[kDecodeStep / 2][4];  // of block i, for the sums' four numbers
        if (kFp8) {
#pragma unroll
          for (int i = 0; i < kDecodeStep / 2; ++i) {
            const int k = min(s * kDecodeBlocks + i * kDecodeSet + warp % kDecodeSet, scale_groups - 1);
            const float w = __ldg(ws + k);
            const float u = kGatedForm ? __ldg(ws + static_cast<int64_t>(blocks) * scale_groups + k) : 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float v = __ldg(xs[j] + k);
              by[i][j] = v * w, by[i][2 + j] = v * u;
            }
          }
        }
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
          u[i] = g < rows && s * kDecodeCodes + b * 128 + c * 16 < K
                     ? *reinterpret_cast<const uint4*>(stage + Shape::kTiles * kDecodeTileBytes +
                                                       g * kDecodePitch + b * 128 + c * 16)
                     : zero;
        }
        if (kFp8) {
#pragma unroll
          for (int i = 0; i < kDecodeStep; i += 2) {
            float part[2][4] = {};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              multiply_codes<kFp8, kGatedForm>(part[j], v[i + j].x, w[i + j].x, u[i + j].x);
              multiply_codes<kFp8, kGatedForm>(part[j], v[i + j].y, w[i + j].y, u[i + j].y);
              multiply_codes<kFp8, kGatedForm>(part[j], v[i + j].z, w[i + j].z, u[i + j].z);
              multiply_codes<kFp8, kGatedForm>(part[j], v[i + j].w, w[i + j].w, u[i + j].w);
            }
            // (a block behind K has zeros and the last block's scales)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] += (part[0][j] + part[1][j]) * by[i / 2][j];
          }
        } else {
#pragma unroll
          for (int i = 0; i < kDecodeStep; ++i) {
            multiply_codes<kFp8, kGatedForm>(acc[i], v[i].x, w[i].x, u[i].x);
            multiply_codes<kFp8, kGatedForm>(acc[i], v[i].y, w[i].y, u[i].y);
            multiply_codes<kFp8, kGatedForm>(acc[i], v[i].z, w[i].z, u[i].z);
            multiply_codes<kFp8, kGatedForm>(acc[i], v[i].w, w[i].w, u[i].w);
          }
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
    int turn = 0;
    for (Task t = start; t.group < groups; advance(t), ++turn) {
      const DecodeGroup task = s_groups[t.group];
      const int buf = turn & 1;
      // Value j of the lane: feature and row (j * 32 + lane) of the task.
      constexpr int kValues = kDecodeFeatures * kDecodeGroup / 32;
      const int f = lane % kDecodeFeatures, r0 = lane / kDecodeFeatures;
      const int c = t.part * kDecodeFeatures + f;
      float by[kValues], by_up[kValues];
      if (!kFp8) {
        const float* ws = a.weight_scales + static_cast<int64_t>(task.e) * a.N + c;
        const float w = __ldg(ws), u = kGatedForm ? __ldg(ws + F) : 0.f;
#pragma unroll
        for (int j = 0; j < kValues; ++j) {
          const int r = min(r0 + j * (32 / kDecodeFeatures), task.rows - 1);
          const float v = __ldg(a.scales + task.lo + r);
          by[j] = v * w, by_up[j] = v * u;
        }
      }
      // (spans a task's contraction)
      if (!warp_wait(smem_addr(&s_sums[buf]), turn / 2 & 1, gave_up, smem_addr(&s_issued))) break;
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
#pragma unroll
      for (int j = 0; j < kValues; ++j) {
        const int r = r0 + j * (32 / kDecodeFeatures);
        if (r >= task.rows) break;
        const int64_t row = task.lo + r;
        float v = kFp8 ? z[j] : z[j] * by[j];
        if (kGatedForm) {
          const float y = kFp8 ? up[j] : up[j] * by_up[j];
          out[row * F + c] = from_f<T>(act_of(a.act, v) * y);
        } else {
          if (a.bias != nullptr)
            v += to_f(static_cast<const T*>(a.bias)[static_cast<int64_t>(task.e) * a.N + c]);
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
