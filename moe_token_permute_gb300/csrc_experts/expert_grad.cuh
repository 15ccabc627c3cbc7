// expert_grad.cuh -- the elementwise and column-sum parts of the expert
// operators' backward passes.  All are memory traffic only.
#pragma once

#include <type_traits>

#include "expert_math.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace experts {

constexpr int kGradThreads = 256;
constexpr int kGradWarps = kGradThreads / 32;

// dz from d_out and the saved z.
//   gated:  z = [gate, up] [rows, 2W]; dz = [d * up * act'(gate), d * act(gate)]
//   linear: z [rows, W]; dz = d * act'(z)
// W is d_out's width.  Computed in fp32 from 16-bit z and rounded once: dz is
// the operand of two 16-bit matrix products.  A warp has 32 vectors of 8 columns
// (blockIdx.y) and takes rows of them, two in flight.  dz is written for the rows of
// the experts' segments, which are what the products read, and for no others.
// Gated, 65536 rows of 768 over 128 experts: 81 us, 93% of the measured copy bandwidth.
template <typename T, bool kGatedForm, int kAct>
__global__ void __launch_bounds__(kGradThreads)
k_act_grad(const T* __restrict__ d_out, const T* __restrict__ z, T* __restrict__ dz,
           const int64_t* __restrict__ offset, int E, int64_t num_rows, int64_t W,
           unsigned* __restrict__ status) {
  constexpr int kRows = 2;
  pdl_wait();
  pdl_launch_dependents();
  const RowRange range = rows_in_use<kGradThreads>(offset, E, num_rows);
  if (range.bad && status != nullptr && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    atomicOr(status, MOE_FLAG_OFFSET_OUT_OF_RANGE);
  const int64_t c = static_cast<int64_t>(blockIdx.y) * 32 + (threadIdx.x & 31);
  const bool in_width = c < W / 8;  // (the whole warp stays for in_segment)
  const int64_t zw = kGatedForm ? 2 * W : W;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGradWarps;
  const int64_t first = range.lo + static_cast<int64_t>(blockIdx.x) * kGradWarps + (threadIdx.x >> 5);
  // Malformed offsets have a loop of their own, which asks for every row.
  auto run = [&](auto gaps) {
    for (int64_t r0 = first; r0 < range.hi; r0 += kRows * step) {
      Vec8<T> d[kRows], g[kRows], u[kRows];
      bool use[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int64_t r = r0 + j * step;
        use[j] = r < range.hi && in_width;
        if (decltype(gaps)::value && r < range.hi && !in_segment(offset, E, num_rows, r))
          use[j] = false;
        if (!use[j]) continue;
        d[j].v = ld_stream(reinterpret_cast<const uint4*>(d_out + r * W) + c);
        g[j].v = ld_stream(reinterpret_cast<const uint4*>(z + r * zw) + c);
        if (kGatedForm) u[j].v = ld_stream(reinterpret_cast<const uint4*>(z + r * zw + W) + c);
      }
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int64_t r = r0 + j * step;
        if (!use[j]) continue;
        Vec8<T> dg, du;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float a;
          const float da = act_grad<kAct>(to_f(g[j].e[i]), a);
          const float di = to_f(d[j].e[i]);
          if (kGatedForm) {
            dg.e[i] = from_f<T>(di * to_f(u[j].e[i]) * da);
            du.e[i] = from_f<T>(di * a);
          } else {
            dg.e[i] = from_f<T>(di * da);
          }
        }
        reinterpret_cast<uint4*>(dz + r * zw)[c] = dg.v;
        if (kGatedForm) reinterpret_cast<uint4*>(dz + r * zw + W)[c] = du.v;
      }
    }
  };
  if (range.bad) run(std::true_type());
  else run(std::false_type());
}

// d_bias[e] = column sums of dz over e's rows, in fp32 and in a fixed order: a
// block takes kVecs vectors of 8 columns of one expert and 256 / kVecs rows at a
// time: 64 columns and 32 rows, or, for experts of few rows, 512 and 4 (256 experts
// of 8 rows, 7168 columns: 43 us in narrow blocks).  With few experts and columns a
// cluster of blocks shares the rows and the first adds the others' sums up.
// 8 experts of 1024 rows, 4096 columns: 10.9 us, 92% of the measured copy bandwidth.
constexpr int kBiasSplit = 8;
constexpr int kBiasNarrow = 8, kBiasWide = 64;

template <typename T, int kVecs>
__global__ void __launch_bounds__(kGradThreads)
k_bias_grad(const T* __restrict__ dz, const int64_t* __restrict__ offset, int64_t num_rows,
            int64_t N, T* __restrict__ d_bias, unsigned* __restrict__ status) {
  constexpr int kAhead = kVecs == kBiasNarrow ? 8 : 4;
  constexpr int kLanes = kGradThreads / kVecs;  // rows at a time
  constexpr int kCols = 8 * kVecs;
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float part[kLanes][kCols + 1];
  __shared__ float sums[kCols];
  const int e = blockIdx.y;
  bool bad;
  const Segment s = segment(offset, e, num_rows, &bad);
  if (bad && status != nullptr && blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0)
    atomicOr(status, MOE_FLAG_OFFSET_OUT_OF_RANGE);
  const int splits = gridDim.z, split = blockIdx.z;
  const int share = (s.hi - s.lo + splits - 1) / splits;
  const int lo = min(s.hi, s.lo + split * share), hi = min(s.hi, lo + share);
  const int tx = threadIdx.x % kVecs, ty = threadIdx.x / kVecs;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kVecs + tx;
  float acc[8] = {};
  if (c < N / 8) {
    const uint4* at = reinterpret_cast<const uint4*>(dz) + c;
    for (int r = lo + ty; r < hi; r += kLanes * kAhead) {
      Vec8<T> v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        v[j].v = r + kLanes * j < hi
                     ? ld_stream(at + static_cast<int64_t>(r + kLanes * j) * (N / 8))
                     : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += to_f(v[j].e[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[ty][tx * 8 + i] = acc[i];
  __syncthreads();
  for (int i = threadIdx.x; i < kCols; i += kGradThreads) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < kLanes; ++j) sum += part[j][i];
    sums[i] = sum;
  }
  if (splits > 1) cluster_sync();
  if (split == 0) {
    for (int i = threadIdx.x; i < kCols; i += kGradThreads) {
      float sum = sums[i];
      for (int j = 1; j < splits; ++j) sum += cluster_load(cluster_addr(smem_addr(&sums[i]), j));
      const int64_t col = static_cast<int64_t>(blockIdx.x) * kCols + i;
      if (col < N) d_bias[static_cast<int64_t>(e) * N + col] = from_f<T>(sum);
    }
  }
  if (splits > 1) cluster_sync();  // the others' sums stay until they are read
}

}  // namespace experts
}  // namespace moe
