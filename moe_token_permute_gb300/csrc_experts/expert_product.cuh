// expert_product.cuh -- the grouped matrix products.
//
// One kernel, three uses, all D = sum over k of A[i,k] B[j,k] per expert e:
//   forward   rows r of e:  z[r, n]   = sum_k x[r,k] W[e][n,k]
//   d_rows    rows r of e:  dx[r, k]  = sum_n dz[r,n] W[e][n,k]
//   d_weight  per expert:   dW[e][n,k] = sum_r dz[r,n] x[r,k]
// The simplest form: a block computes a 64 x 64 tile from 64 x 16 slices in
// shared memory, a thread 4 x 4 values in fp32.
#pragma once

#include "expert_math.cuh"

namespace moe {
namespace experts {

enum Use { kForward, kGated, kRowsGrad, kWeightGrad };

struct ProductArgs {
  const void* x;        // forward: rows; d_rows: dz; d_weight: rows
  const void* w;        // forward, d_rows: weight; d_weight: dz
  const int64_t* offset;
  int64_t num_rows;
  int64_t K, N;         // in_size and out_size of the weight [E, N, K]
  int E;
  const void* bias;
  const void* residual;
  void* out;
  void* preact;
  unsigned* status;
};

constexpr int kTile = 64, kSlice = 16;

template <typename T, int kUse, int kAct>
__global__ void __launch_bounds__(256) k_expert_product(ProductArgs a) {
  pdl_wait();
  __shared__ float sa[kSlice][kTile + 4], sb[2][kSlice][kTile + 4];
  __shared__ int s_e, s_lo, s_hi;
  // Row tiles of all experts are numbered one after the other.
  const int64_t i_tile = blockIdx.x;
  int e = 0;
  int64_t i0 = 0;
  if (kUse == kWeightGrad) {
    const int64_t per = (a.N + kTile - 1) / kTile;
    e = static_cast<int>(i_tile / per);
    i0 = (i_tile - e * per) * kTile;
  }
  if (threadIdx.x == 0) {
    if (kUse == kWeightGrad) {
      bool bad;
      const Segment s = segment(a.offset, e, a.num_rows, &bad);
      if (bad && a.status != nullptr) atomicOr(a.status, MOE_FLAG_OFFSET_OUT_OF_RANGE);
      s_e = e, s_lo = s.lo, s_hi = s.hi;
    } else {
      int64_t left = i_tile;
      s_e = -1;
      bool any_bad = false;
      for (int g = 0; g < a.E; ++g) {
        bool bad;
        const Segment s = segment(a.offset, g, a.num_rows, &bad);
        any_bad |= bad;
        const int64_t n = (s.hi - s.lo + kTile - 1) / kTile;
        if (left < n) {
          s_e = g, s_lo = s.lo + static_cast<int>(left) * kTile, s_hi = s.hi;
          break;
        }
        left -= n;
      }
      if (any_bad && a.status != nullptr) atomicOr(a.status, MOE_FLAG_OFFSET_OUT_OF_RANGE);
    }
  }
  __syncthreads();
  e = s_e;
  if (e < 0) return;
  const int lo = s_lo, hi = s_hi;
  const int64_t j0 = static_cast<int64_t>(blockIdx.y) * kTile;
  const T* x = static_cast<const T*>(a.x);
  const T* w = static_cast<const T*>(a.w);
  const int64_t F = a.N / 2;
  const int64_t jn = kUse == kForward ? a.N : kUse == kGated ? F : a.K;
  const int64_t in = kUse == kWeightGrad ? a.N : hi - lo;
  const int64_t kn = kUse == kForward || kUse == kGated ? a.K : kUse == kRowsGrad ? a.N : hi - lo;
  const int64_t we = static_cast<int64_t>(e) * a.N * a.K;
  float acc[2][4][4] = {};
  const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
  for (int64_t k0 = 0; k0 < kn; k0 += kSlice) {
    for (int s = threadIdx.x; s < kTile * kSlice; s += 256) {
      const int r = s / kSlice, k = s % kSlice;
      const int64_t i = i0 + r, j = j0 + r, kk = k0 + k;
      float va = 0.f, vb = 0.f, vc = 0.f;
      if (kk < kn) {
        if (kUse == kForward || kUse == kGated) {
          if (r < in) va = to_f(x[(lo + r) * a.K + kk]);
          if (j < jn) vb = to_f(w[we + j * a.K + kk]);
          if (kUse == kGated && j < jn) vc = to_f(w[we + (F + j) * a.K + kk]);
        } else if (kUse == kRowsGrad) {
          if (r < in) va = to_f(x[(lo + r) * a.N + kk]);
          if (j < jn) vb = to_f(w[we + kk * a.K + j]);
        } else {
          if (i < in) va = to_f(w[(lo + kk) * a.N + i]);
          if (j < jn) vb = to_f(x[(lo + kk) * a.K + j]);
        }
      }
      sa[k][r] = va;
      sb[0][k][r] = vb;
      if (kUse == kGated) sb[1][k][r] = vc;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSlice; ++k)
#pragma unroll
      for (int p = 0; p < (kUse == kGated ? 2 : 1); ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[p][i][j] = fmaf(sa[k][ti * 4 + i], sb[p][k][tj * 4 + j], acc[p][i][j]);
    __syncthreads();
  }
  T* out = static_cast<T*>(a.out);
  T* preact = static_cast<T*>(a.preact);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t ii = i0 + ti * 4 + i, jj = j0 + tj * 4 + j;
      if (ii >= in || jj >= jn) continue;
      float z = acc[0][i][j];
      if (kUse == kWeightGrad) {
        out[we + ii * a.K + jj] = from_f<T>(z);
        continue;
      }
      const int64_t r = lo + ii;
      if (kUse == kRowsGrad) {
        out[r * a.K + jj] = from_f<T>(z);
      } else if (kUse == kGated) {
        if (preact != nullptr) {
          preact[r * a.N + jj] = from_f<T>(z);
          preact[r * a.N + F + jj] = from_f<T>(acc[1][i][j]);
        }
        out[r * F + jj] = from_f<T>(act<kAct>(z) * acc[1][i][j]);
      } else {
        if (a.bias != nullptr)
          z += to_f(static_cast<const T*>(a.bias)[static_cast<int64_t>(e) * a.N + jj]);
        if (preact != nullptr) preact[r * a.N + jj] = from_f<T>(z);
        z = act<kAct>(z);
        if (a.residual != nullptr) z += to_f(static_cast<const T*>(a.residual)[r * a.N + jj]);
        out[r * a.N + jj] = from_f<T>(z);
      }
    }
}

}  // namespace experts
}  // namespace moe
