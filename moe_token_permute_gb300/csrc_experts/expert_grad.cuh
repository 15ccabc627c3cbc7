// expert_grad.cuh -- the elementwise and column-sum parts of the expert
// operators' backward passes.  All are memory traffic only.
#pragma once

#include "expert_math.cuh"

namespace moe {
namespace experts {

constexpr int kGradThreads = 256;
constexpr int kGradWarps = kGradThreads / 32;

// dz from d_out and the saved z, one warp per (row, 32 vectors of 8 columns).
//   gated:  z = [gate, up] [rows, 2W]; dz = [d * up * act'(gate), d * act(gate)]
//   linear: z [rows, W]; dz = d * act'(z)
// W is d_out's width.  Computed in fp32 from 16-bit z and rounded once: dz is
// the operand of two 16-bit matrix products.
template <typename T, bool kGatedForm, int kAct>
__global__ void __launch_bounds__(kGradThreads)
k_act_grad(const T* __restrict__ d_out, const T* __restrict__ z, T* __restrict__ dz,
           const int64_t* __restrict__ offset, int E, int64_t num_rows, int64_t W) {
  pdl_wait();
  const int64_t n = rows_in_use(offset, E, num_rows);
  const int64_t vecs = W / 8;
  const int64_t chunks = (vecs + 31) / 32;
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = static_cast<int64_t>(blockIdx.x) * kGradWarps + (threadIdx.x >> 5);
  const int64_t n_warps = static_cast<int64_t>(gridDim.x) * kGradWarps;
  for (int64_t item = warp0; item < n * chunks; item += n_warps) {
    const int64_t r = item / chunks;
    const int64_t c = (item - r * chunks) * 32 + lane;
    if (c >= vecs) continue;
    Vec8<T> d, g, u;
    d.v = ld_stream(reinterpret_cast<const uint4*>(d_out + r * W) + c);
    if (kGatedForm) {
      g.v = ld_stream(reinterpret_cast<const uint4*>(z + r * 2 * W) + c);
      u.v = ld_stream(reinterpret_cast<const uint4*>(z + r * 2 * W + W) + c);
    } else {
      g.v = ld_stream(reinterpret_cast<const uint4*>(z + r * W) + c);
    }
    Vec8<T> dg, du;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a;
      const float da = act_grad<kAct>(to_f(g.e[i]), a);
      const float di = to_f(d.e[i]);
      if (kGatedForm) {
        dg.e[i] = from_f<T>(di * to_f(u.e[i]) * da);
        du.e[i] = from_f<T>(di * a);
      } else {
        dg.e[i] = from_f<T>(di * da);
      }
    }
    if (kGatedForm) {
      reinterpret_cast<uint4*>(dz + r * 2 * W)[c] = dg.v;
      reinterpret_cast<uint4*>(dz + r * 2 * W + W)[c] = du.v;
    } else {
      reinterpret_cast<uint4*>(dz + r * W)[c] = dg.v;
    }
  }
}

// d_bias[e] = column sums of dz over e's rows, in fp32 and in a fixed order: a
// block takes 64 columns of one expert, 8 threads a row and 32 rows at a time.
template <typename T>
__global__ void __launch_bounds__(kGradThreads)
k_bias_grad(const T* __restrict__ dz, const int64_t* __restrict__ offset, int64_t num_rows,
            int64_t N, T* __restrict__ d_bias) {
  pdl_wait();
  __shared__ float part[32][64 + 1];
  const int e = blockIdx.y;
  const Segment s = segment(offset, e, num_rows);
  const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 8 + tx;
  float acc[8] = {};
  if (c < N / 8) {
#pragma unroll 4
    for (int r = s.lo + ty; r < s.hi; r += 32) {
      Vec8<T> v;
      v.v = ld_stream(reinterpret_cast<const uint4*>(dz + static_cast<int64_t>(r) * N) + c);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += to_f(v.e[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[ty][tx * 8 + i] = acc[i];
  __syncthreads();
  if (threadIdx.x < 64) {
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += part[i][threadIdx.x];
    if (col < N) d_bias[static_cast<int64_t>(e) * N + col] = from_f<T>(sum);
  }
}

}  // namespace experts
}  // namespace moe
