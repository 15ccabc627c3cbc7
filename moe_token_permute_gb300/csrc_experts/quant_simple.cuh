// quant_simple.cuh -- the grouped products of 8-bit rows and weights.
//
//   fp8   z[r, n] = sum over groups g of 128 columns of
//                   xs[r, g] ws[n / 128, g] sum_{k in g} x[r, k] w[n, k]
//   int8  z[r, n] = xs[r] ws[n] sum_k x[r, k] w[n, k]
#pragma once

#include <cuda_fp8.h>

#include "quant_product.cuh"

namespace moe {
namespace experts {

__device__ __forceinline__ float activate(int a, float z) {
  if (a == MOE_ACT_SILU) return act<MOE_ACT_SILU>(z);
  if (a == MOE_ACT_GELU) return act<MOE_ACT_GELU>(z);
  if (a == MOE_ACT_RELU) return act<MOE_ACT_RELU>(z);
  return z;
}

template <bool kFp8>
__device__ __forceinline__ float code_value(uint8_t c) {
  if (!kFp8) return static_cast<float>(static_cast<int8_t>(c));
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(h);
}

// A block: 64 features of an expert, its rows 16 at a time.  Thread (i, j) has row i
// and features j + 16 f.
template <typename T, bool kFp8, bool kGatedForm>
__global__ void __launch_bounds__(256) k_quant_simple(const QuantArgs a) {
  constexpr int kRows = 16, kFeatures = 64, kDepth = 32, kParts = kGatedForm ? 2 : 1;
  __shared__ float s_x[kRows][kDepth + 1], s_w[kParts][kFeatures][kDepth + 1];
  pdl_wait();
  pdl_launch_dependents();
  const int e = blockIdx.y;
  bool bad;
  const Segment s = segment(a.offset, e, a.num_rows, &bad);
  if (bad && a.status != nullptr && blockIdx.x == 0 && threadIdx.x == 0)
    atomicOr(a.status, MOE_FLAG_OFFSET_OUT_OF_RANGE);
  const int i = threadIdx.x / 16, j = threadIdx.x % 16;
  const int width = static_cast<int>(kGatedForm ? a.N / 2 : a.N), K = static_cast<int>(a.K);
  const int f0 = blockIdx.x * kFeatures;
  const int groups = (K + kGroupSlice - 1) / kGroupSlice;
  const int blocks = (width + kGroupSlice - 1) / kGroupSlice;
  const uint8_t* x = static_cast<const uint8_t*>(a.codes);
  const uint8_t* w = static_cast<const uint8_t*>(a.weight) + static_cast<int64_t>(e) * a.N * K;
  for (int r0 = s.lo; r0 < s.hi; r0 += kRows) {
    float z[kParts][4] = {};
    int zi[kParts][4] = {};
    for (int k0 = 0; k0 < K; k0 += kDepth) {
      __syncthreads();
      for (int t = threadIdx.x; t < kRows * kDepth; t += 256) {
        const int r = r0 + t / kDepth, k = k0 + t % kDepth;
        s_x[t / kDepth][t % kDepth] =
            r < s.hi && k < K ? code_value<kFp8>(x[static_cast<int64_t>(r) * K + k]) : 0.f;
      }
      for (int t = threadIdx.x; t < kParts * kFeatures * kDepth; t += 256) {
        const int p = t / (kFeatures * kDepth), f = t / kDepth % kFeatures, k = k0 + t % kDepth;
        s_w[p][f][t % kDepth] =
            f0 + f < width && k < K
                ? code_value<kFp8>(w[(static_cast<int64_t>(p) * width + f0 + f) * K + k])
                : 0.f;
      }
      __syncthreads();
      const int g = k0 / kGroupSlice, r = r0 + i;
      const float xs = kFp8 && r < s.hi ? a.scales[static_cast<int64_t>(r) * groups + g] : 1.f;
#pragma unroll
      for (int p = 0; p < kParts; ++p)
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          if (kFp8) {
            float sum = 0.f;
            for (int k = 0; k < kDepth; ++k) sum += s_x[i][k] * s_w[p][j + 16 * f][k];
            const int n = min(f0 + j + 16 * f, width - 1);
            const float ws =
                a.weight_scales[((static_cast<int64_t>(e) * kParts + p) * blocks +
                                 n / kGroupSlice) * groups + g];
            z[p][f] += sum * (xs * ws);
          } else {
            for (int k = 0; k < kDepth; ++k)
              zi[p][f] += static_cast<int>(s_x[i][k]) * static_cast<int>(s_w[p][j + 16 * f][k]);
          }
        }
    }
    const int r = r0 + i;
    if (r >= s.hi) continue;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int n = f0 + j + 16 * f;
      if (n >= width) continue;
      if (!kFp8)
        for (int p = 0; p < kParts; ++p)
          z[p][f] = static_cast<float>(zi[p][f]) *
                    (a.scales[r] * a.weight_scales[static_cast<int64_t>(e) * a.N + p * width + n]);
      float v = z[0][f];
      if (kGatedForm) {
        v = activate(a.act, v) * z[kParts - 1][f];
      } else {
        if (a.bias != nullptr)
          v += to_f(static_cast<const T*>(a.bias)[static_cast<int64_t>(e) * a.N + n]);
        v = activate(a.act, v);
        if (a.residual != nullptr)
          v += to_f(static_cast<const T*>(a.residual)[static_cast<int64_t>(r) * width + n]);
      }
      static_cast<T*>(a.out)[static_cast<int64_t>(r) * width + n] = from_f<T>(v);
    }
  }
}

}  // namespace experts
}  // namespace moe
