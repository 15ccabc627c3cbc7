// expert_math.cuh -- element types, activations and expert segments shared by
// the expert operators' kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../csrc/common.cuh"
#include "moe_experts.h"

namespace moe {
namespace experts {

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f<__half>(float x) {
  return __float2half_rn(x);
}

// Two values in one register, and back; the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t x);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t x) {
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

// 16 bytes of a row: 8 elements.
template <typename T>
union Vec8 {
  uint4 v;
  T e[8];
};

// 1 / (1 + exp(-z)); 0 and 1 at the infinities.  The fast exponential is good to
// 2 + 1.173 |z| ulp and the fast division to 2, so the relative error is at most
// (4.5 + 1.173 |z|) 2^-23: 2^-19 at |z| = 10, 2^-16 at 88, far below the 16-bit
// results (the correctly rounded reciprocal took a third of the gated product's
// epilogue).  The division gives 0 for denominators beyond 2^126, before the
// exponential overflows: 0 for z < -87.3, where the value is below 2^-126.
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

constexpr float kGeluA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// 0.5 (1 + tanh(a)) = sigmoid(2a), so both smooth activations are z times one
// sigmoid: an exponential and a reciprocal each.  Beyond |z| = 16 gelu's
// sigmoid is 0 or 1 in fp32, so its polynomials take z cut to that range:
// squares of larger z would overflow against the zero.
constexpr float kGeluCut = 16.0f;
__device__ __forceinline__ float gelu_cut(float z) {
  return fminf(fmaxf(z, -kGeluCut), kGeluCut);
}

__device__ __forceinline__ float gelu_sigmoid(float zc) {
  return sigmoid(2.0f * kGeluA * zc * (1.0f + kGeluB * zc * zc));
}

template <int kAct>
__device__ __forceinline__ float act(float z) {
  if (kAct == MOE_ACT_SILU) return z * sigmoid(z);
  if (kAct == MOE_ACT_GELU) return z * gelu_sigmoid(gelu_cut(z));
  if (kAct == MOE_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
  return z;
}

// a = act(z), and its derivative.  z was rounded to 16 bits: an fp16 z beyond 65504 is
// infinite here though it was not in the forward pass, and takes the limits (act -> 0
// and act' -> 0 below, act' -> 1 above) instead of infinity times zero.  The cuts lie
// where the sigmoid is 0 or 1 already, so they change no other value; NaN stays NaN (fmaxf would
// lose it).
constexpr float kSiluCut = 128.0f;
template <int kAct>
__device__ __forceinline__ float act_grad(float z, float& a) {
  if (kAct == MOE_ACT_SILU) {
    const float p = sigmoid(z);
    a = (z < -kSiluCut ? -kSiluCut : z) * p;
    return p + (a > kSiluCut ? kSiluCut : a) * (1.0f - p);
  }
  if (kAct == MOE_ACT_GELU) {
    const float zc = gelu_cut(z);
    const float p = gelu_sigmoid(zc);
    a = (z < -kGeluCut ? -kGeluCut : z) * p;
    return p + (a > kGeluCut ? kGeluCut : a) * (1.0f - p) *
                   (2.0f * kGeluA * (1.0f + 3.0f * kGeluB * zc * zc));
  }
  if (kAct == MOE_ACT_RELU) {
    a = z > 0.0f ? z : (z != z ? z : 0.0f);
    return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  }
  a = z;
  return 1.0f;
}

// Rows of expert e, cut to [0, num_rows] whatever the offsets hold.
struct Segment {
  int lo, hi;
};

__device__ __forceinline__ Segment segment(const int64_t* offset, int e, int64_t num_rows,
                                           bool* bad = nullptr) {
  const int64_t a = __ldg(offset + e), b = __ldg(offset + e + 1);
  const int64_t lo = a < 0 ? 0 : (a > num_rows ? num_rows : a);
  const int64_t hi = b < lo ? lo : (b > num_rows ? num_rows : b);
  if (bad != nullptr) *bad = lo != a || hi != b;
  return {static_cast<int>(lo), static_cast<int>(hi)};
}

// The rows that belong to an expert at all, found by a whole block of kThreads: a range
// that holds every segment.  Valid offsets leave no gaps in it (a thread looks at one
// expert in kThreads, and the range is the offsets' ends); decreasing ones may, and then
// in_segment says which of its rows count.
struct RowRange {
  int lo, hi;
  bool bad;
};

template <int kThreads>
__device__ __forceinline__ RowRange rows_in_use(const int64_t* offset, int num_experts,
                                                int64_t num_rows) {
  const int64_t first = __ldg(offset), last = __ldg(offset + num_experts);
  bool bad = false;
  for (int e = threadIdx.x; e < num_experts; e += kThreads) {
    bool b;
    segment(offset, e, num_rows, &b);
    bad |= b;
  }
  if (!__syncthreads_or(bad)) return {static_cast<int>(first), static_cast<int>(last), false};
  int lo = INT32_MAX, hi = 0;
  for (int e = threadIdx.x & 31; e < num_experts; e += 32) {
    const Segment s = segment(offset, e, num_rows);
    if (s.lo < s.hi) lo = min(lo, s.lo), hi = max(hi, s.hi);
  }
  return {__reduce_min_sync(kFullMask, lo), __reduce_max_sync(kFullMask, hi), true};
}

// Whether row r, the same in the whole warp, lies in any expert's segment.
__device__ __forceinline__ bool in_segment(const int64_t* offset, int num_experts,
                                           int64_t num_rows, int64_t r) {
  bool in = false;
  for (int e = threadIdx.x & 31; e < num_experts; e += 32) {
    const Segment s = segment(offset, e, num_rows);
    in |= s.lo <= r && r < s.hi;
  }
  return __any_sync(kFullMask, in) != 0;
}

}  // namespace experts
}  // namespace moe
