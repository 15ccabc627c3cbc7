// unpermute_grad.cuh -- the gradients of moe_unpermute.
//
// Pure memory traffic: d_out is read once from memory, every kept row read and
// written once.  A warp takes a few consecutive (t, k), drops those without a row
// at once, and passes over the others' rows one by one: a row's dot product stays
// in one warp, and the rows of a token read its d_out from L1.
// T = 4096, K = 8, H = 7168 on GB300: 150 us, the measured copy bandwidth.
// (With a block's threads across the columns of one row after another, each row's
// sum was a round of shuffles through the block that held the loads back: 203 us.
// With a warp for every (t, k) the warps without a row left most of the SM idle
// where an expert map drops three rows in four: 35 us at T = 8192, K = 6, H = 2048.)
#pragma once

#include "expert_math.cuh"

namespace moe {
namespace experts {

constexpr int kCombineWarps = 8;
constexpr int kCombineAhead = 4;  // vectors of a lane in flight, of the row and of d_out each

template <typename VecT>
union BfVec {
  static constexpr int kElems = sizeof(VecT) / 2;
  VecT v;
  __nv_bfloat16 e[sizeof(VecT) / 2];
};

// rows may be d_rows: a lane reads a vector before it writes it.
template <typename VecT>
__global__ void __launch_bounds__(kCombineWarps * 32)
k_unpermute_backward(const VecT* __restrict__ d_out, const VecT* rows, int64_t num_rows,
                     int64_t row_vecs, const float* __restrict__ topk_weights,
                     const int32_t* __restrict__ inv_permuted_idx, int64_t items, int K,
                     int per_warp, VecT* d_rows,
                     float* __restrict__ d_weights, unsigned* __restrict__ status) {
  constexpr int kE = BfVec<VecT>::kElems;
  constexpr int V = kCombineAhead;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * kCombineWarps + (threadIdx.x >> 5)) * per_warp;
  // Lane l: item i0 + l, whose row is p_lane.
  int p_lane = -1;
  float w_lane = 0.f;
  if (lane < per_warp && i0 + lane < items) {
    p_lane = __ldg(inv_permuted_idx + i0 + lane);
    w_lane = __ldg(topk_weights + i0 + lane);
    if (p_lane < 0 || p_lane >= num_rows) {
      if (p_lane != -1 && status != nullptr) atomicOr(status, MOE_FLAG_INV_OUT_OF_RANGE);
      if (d_weights != nullptr) d_weights[i0 + lane] = 0.f;
      p_lane = -1;
    }
  }
  for (unsigned kept = __ballot_sync(kFullMask, p_lane >= 0); kept != 0u; kept &= kept - 1u) {
    const int l = __ffs(kept) - 1;
    const int64_t p = __shfl_sync(kFullMask, p_lane, l);
    const float w = __shfl_sync(kFullMask, w_lane, l);
    const VecT* d = d_out + (i0 + l) / K * row_vecs;
    const VecT* row = rows + p * row_vecs;
    VecT* to = d_rows + p * row_vecs;
    float dot = 0.f;
    for (int64_t c0 = lane; c0 - lane < row_vecs; c0 += V * 32) {
      BfVec<VecT> x[V], g[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int64_t c = c0 + i * 32;
        if (rows != nullptr && c < row_vecs) x[i].v = row[c];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int64_t c = c0 + i * 32;
        if (c < row_vecs) g[i].v = __ldg(d + c);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int64_t c = c0 + i * 32;
        if (c >= row_vecs) continue;
        if (rows != nullptr) {
#pragma unroll
          for (int e = 0; e < kE; ++e) dot = fmaf(to_f(g[i].e[e]), to_f(x[i].e[e]), dot);
        }
        if (d_rows != nullptr) {
          BfVec<VecT> y;
#pragma unroll
          for (int e = 0; e < kE; ++e) y.e[e] = __float2bfloat16_rn(w * to_f(g[i].e[e]));
          to[c] = y.v;
        }
      }
    }
    if (d_weights != nullptr) {
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(kFullMask, dot, s);
      if (lane == 0) d_weights[i0 + l] = dot;
    }
  }
}

}  // namespace experts
}  // namespace moe
