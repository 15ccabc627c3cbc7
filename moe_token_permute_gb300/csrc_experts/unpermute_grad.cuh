// unpermute_grad.cuh -- the gradients of moe_unpermute.
//
// Pure memory traffic: d_out is read once, every kept row read and written
// once.  A block owns a token: its threads hold a slice of d_out in registers
// and pass over the token's K rows, writing w * d_out and summing
// d_out * row; the K sums are joined across the block once at the end.
#pragma once

#include "expert_math.cuh"

namespace moe {
namespace experts {

constexpr int kCombineMaxWarps = 8;

template <typename VecT>
union BfVec {
  static constexpr int kElems = sizeof(VecT) / 2;
  VecT v;
  __nv_bfloat16 e[sizeof(VecT) / 2];
};

template <typename VecT, int V>
__global__ void __launch_bounds__(kCombineMaxWarps * 32)
k_unpermute_backward(const VecT* __restrict__ d_out, const VecT* rows, int64_t num_rows,
                     int64_t row_vecs, const float* __restrict__ topk_weights,
                     const int32_t* __restrict__ inv_permuted_idx, int K, VecT* d_rows,
                     float* __restrict__ d_weights, unsigned* __restrict__ status) {
  constexpr int kE = BfVec<VecT>::kElems;
  pdl_wait();
  __shared__ float part[MOE_MAX_TOPK][kCombineMaxWarps];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int p_lane = -1;
  float w_lane = 0.f;
  bool bad = false;
  if (lane < K) {
    p_lane = __ldg(inv_permuted_idx + t * K + lane);
    w_lane = __ldg(topk_weights + t * K + lane);
    bad = p_lane < -1 || p_lane >= num_rows;
    if (bad) p_lane = -1;
    part[lane][warp] = 0.f;
  }
  if (status != nullptr && warp == 0 && __any_sync(kFullMask, bad) && lane == 0)
    atomicOr(status, MOE_FLAG_INV_OUT_OF_RANGE);
  __syncwarp();
  const unsigned kept = __ballot_sync(kFullMask, p_lane >= 0);
  for (int64_t c0 = threadIdx.x; c0 - lane < row_vecs; c0 += static_cast<int64_t>(V) * blockDim.x) {
    BfVec<VecT> d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t c = c0 + static_cast<int64_t>(i) * blockDim.x;
      if (c < row_vecs) d[i].v = ld_stream(d_out + t * row_vecs + c);
    }
    for (unsigned m = kept; m != 0u; m &= m - 1u) {
      const int k = __ffs(m) - 1;
      const int64_t p = __shfl_sync(kFullMask, p_lane, k);
      const float w = __shfl_sync(kFullMask, w_lane, k);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int64_t c = c0 + static_cast<int64_t>(i) * blockDim.x;
        if (c >= row_vecs) continue;
        if (rows != nullptr) {
          BfVec<VecT> x;
          x.v = rows[p * row_vecs + c];
#pragma unroll
          for (int e = 0; e < kE; ++e) dot = fmaf(to_f(d[i].e[e]), to_f(x.e[e]), dot);
        }
        if (d_rows != nullptr) {
          BfVec<VecT> y;
#pragma unroll
          for (int e = 0; e < kE; ++e) y.e[e] = __float2bfloat16_rn(w * to_f(d[i].e[e]));
          d_rows[p * row_vecs + c] = y.v;
        }
      }
      if (rows != nullptr) {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(kFullMask, dot, s);
        if (lane == 0) part[k][warp] += dot;
      }
    }
  }
  if (d_weights == nullptr) return;
  __syncthreads();
  if (threadIdx.x < K) {
    float sum = 0.f;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) sum += part[threadIdx.x][i];
    d_weights[t * K + threadIdx.x] = sum;
  }
}

}  // namespace experts
}  // namespace moe
