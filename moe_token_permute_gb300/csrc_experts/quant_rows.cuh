// quant_rows.cuh -- rows of 16-bit values to 8-bit codes and fp32 scales.
//
//   fp8   scale = amax / 448 over each 128 columns, code = e4m3(x / scale)
//   int8  scale = amax / 127 over the row,          code = rint(x / scale)
// Both divisions are those of fp32.  A thread has pieces of 16 columns: 32 bytes in,
// 16 out; 8 threads a group of 128 columns.
#pragma once

#include <cuda_fp8.h>

#include "../csrc/quant.cuh"
#include "expert_math.cuh"

namespace moe {
namespace experts {

constexpr int kQuantThreads = 256;
constexpr float kInt8Max = 127.0f;

struct QuantRowsArgs {
  const void* rows;
  const int64_t* offset;  // null: all rows
  int64_t num_rows;
  int64_t H;
  int E;
  void* codes;
  float* scales;
  unsigned* status;
};

// One block per row at a time.
template <typename T, bool kFp8>
__global__ void __launch_bounds__(kQuantThreads) k_quant_rows(const QuantRowsArgs a) {
  __shared__ float s_max[kQuantThreads / 32];
  __shared__ int s_nan;
  pdl_wait();
  pdl_launch_dependents();
  RowRange range = {0, static_cast<int>(a.num_rows), false};
  if (a.offset != nullptr) {
    range = rows_in_use<kQuantThreads>(a.offset, a.E, a.num_rows);
    if (range.bad && a.status != nullptr && blockIdx.x == 0 && threadIdx.x == 0)
      atomicOr(a.status, MOE_FLAG_OFFSET_OUT_OF_RANGE);
  }
  const int pieces = static_cast<int>(a.H / 16);
  const int groups = static_cast<int>((a.H + kQuantGroup - 1) / kQuantGroup);
  for (int64_t r = range.lo + blockIdx.x; r < range.hi; r += gridDim.x) {
    if (range.bad && !in_segment(a.offset, a.E, a.num_rows, r)) continue;
    const T* row = static_cast<const T*>(a.rows) + r * a.H;
    uint8_t* codes = static_cast<uint8_t*>(a.codes) + r * a.H;
    if (kFp8) {
      for (int g = threadIdx.x; g < groups; g += kQuantThreads) {
        const int64_t c0 = static_cast<int64_t>(g) * kQuantGroup;
        const int64_t c1 = min(c0 + kQuantGroup, a.H);
        float amax = 0.f;
        for (int64_t c = c0; c < c1; ++c) amax = fmaxf(amax, fabsf(to_f(row[c])));
        const float scale = amax > 0.f ? __fdiv_rn(amax, kE4m3Max) : 1.f;
        a.scales[r * groups + g] = scale;
        for (int64_t c = c0; c < c1; ++c)
          codes[c] = __nv_cvt_float_to_fp8(__fdiv_rn(to_f(row[c]), scale), __NV_SATFINITE,
                                           __NV_E4M3);
      }
      continue;
    }
    float amax = 0.f;
    bool nan = false;
    for (int c = threadIdx.x; c < a.H; c += kQuantThreads) {
      const float x = to_f(row[c]);
      nan |= x != x;
      amax = fmaxf(amax, fabsf(x));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, d));
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
    s_nan = __syncthreads_or(nan);
    for (int i = 0; i < kQuantThreads / 32; ++i) amax = fmaxf(amax, s_max[i]);
    float scale = amax > 0.f ? __fdiv_rn(amax, kInt8Max) : 1.f;
    if (s_nan) scale = __int_as_float(0x7fffffff);
    if (threadIdx.x == 0) a.scales[r] = scale;
    for (int c = threadIdx.x; c < pieces * 16; c += kQuantThreads) {
      const float q = __fdiv_rn(to_f(row[c]), scale);
      codes[c] = static_cast<uint8_t>(
          isfinite(scale) ? static_cast<int>(rintf(fminf(fmaxf(q, -kInt8Max), kInt8Max))) : 0);
    }
    __syncthreads();
  }
}

}  // namespace experts
}  // namespace moe
