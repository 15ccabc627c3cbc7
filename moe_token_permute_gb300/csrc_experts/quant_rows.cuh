// quant_rows.cuh -- rows of 16-bit values to 8-bit codes and fp32 scales.
//
//   fp8   scale = amax / 448 over each 128 columns, code = e4m3(x / scale)
//   int8  scale = amax / 127 over the row,          code = rint(x / scale)
// Both divisions are those of fp32.  Memory traffic only: 3 bytes a value, and about 9
// instructions for each, which is half of what an SM issues in that time.  A thread has
// pieces of 16 columns, 32 bytes in and 16 out, several of them in flight.
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "../csrc/quant.cuh"
#include "expert_math.cuh"

namespace moe {
namespace experts {

constexpr int kQuantThreads = 256;
// Blocks of an SM, which run all at the same time.  8192 x 14336 bf16 to fp8, with 1 piece in
// flight and 8 blocks 69 us, 2 and 5 59 (one register spilled), 2 and 6 68 (more), 3 and 4 61, 4 and
// 4 62; to int8, with 3 blocks 61, 4 59 (12 spilled), 5 66 (more).  At the copy bandwidth it
// would be 52.
constexpr int kFp8Blocks = 5, kInt8Blocks = 4;
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

// 16 values; kWide: in one access, where rows are 32-byte aligned.
struct Piece {
  uint32_t v[8];
};
template <bool kWide>
__device__ __forceinline__ Piece load_piece(const void* at) {
  Piece p;
  if (kWide) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(p.v[0]), "=r"(p.v[1]), "=r"(p.v[2]), "=r"(p.v[3]), "=r"(p.v[4]),
                   "=r"(p.v[5]), "=r"(p.v[6]), "=r"(p.v[7])
                 : "l"(at));
  } else {
    const uint4 a = ld_stream(static_cast<const uint4*>(at));
    const uint4 b = ld_stream(static_cast<const uint4*>(at) + 1);
    p = {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  }
  return p;
}

// The largest |x| of the 16 as two 16-bit patterns: magnitudes are ordered as whole
// numbers are, NaN above infinity.
__device__ __forceinline__ uint32_t piece_max(const Piece& p) {
  uint32_t m = p.v[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __vmaxu2(m, p.v[i] & 0x7fff7fffu);
  return m;
}
// The larger of the two, as its pattern.
__device__ __forceinline__ uint32_t halves_max(uint32_t m) {
  return max(m & 0xffffu, m >> 16);
}
// The same of the numbers alone: a maximum with NaN is the other operand.
template <typename T>
__device__ __forceinline__ uint32_t max_numbers(uint32_t x, uint32_t y) {
  using Two = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
  const Two m = __hmax2(*reinterpret_cast<const Two*>(&x), *reinterpret_cast<const Two*>(&y));
  return *reinterpret_cast<const uint32_t*>(&m);
}
template <typename T>
__device__ __forceinline__ uint32_t piece_max_numbers(const Piece& p) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_numbers<T>(m, p.v[i] & 0x7fff7fffu);
  return m;
}
template <typename T>
__device__ __forceinline__ float magnitude(uint32_t pattern) {
  return unpack2<T>(pattern).x;
}

// x / scale for the 16, in the order they lie.
template <typename T, typename Put>
__device__ __forceinline__ void divide_piece(const Piece& p, float scale, Put put) {
  if (scale_in_range(scale)) {
    const float y = __frcp_rn(scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = unpack2<T>(p.v[i]);
      put(2 * i, div_by_scale(f.x, scale, y));
      put(2 * i + 1, div_by_scale(f.y, scale, y));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = unpack2<T>(p.v[i]);
      put(2 * i, __fdiv_rn(f.x, scale));
      put(2 * i + 1, __fdiv_rn(f.y, scale));
    }
  }
}

template <typename T>
__device__ __forceinline__ uint4 fp8_codes(const Piece& p, float scale) {
  float q[16];
  divide_piece<T>(p, scale, [&](int i, float v) { q[i] = v; });
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * i], q[4 * i + 1]),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * i + 2], q[4 * i + 3]),
                                                 __NV_SATFINITE, __NV_E4M3);
    c[i] = lo | hi << 16;
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// Added to a number below 2^22, 1.5 * 2^23 leaves it rounded to a whole one, ties to even,
// in the low bits.
template <typename T>
__device__ __forceinline__ uint4 int8_codes(const Piece& p, float scale) {
  if (!isfinite(scale)) return make_uint4(0, 0, 0, 0);
  uint32_t q[16];
  divide_piece<T>(p, scale, [&](int i, float v) {
    // (a subnormal scale is so much rounded that quotients pass 127)
    if (!scale_in_range(scale)) v = fminf(fmaxf(v, -kInt8Max), kInt8Max);
    q[i] = __float_as_uint(__fadd_rn(v, 12582912.0f));
  });
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = __byte_perm(__byte_perm(q[4 * i], q[4 * i + 1], 0x0040),
                       __byte_perm(q[4 * i + 2], q[4 * i + 3], 0x0040), 0x5410);
  return make_uint4(c[0], c[1], c[2], c[3]);
}

__device__ __forceinline__ RowRange quant_rows_range(const QuantRowsArgs& a) {
  if (a.offset == nullptr) return {0, static_cast<int>(a.num_rows), false};
  const RowRange range = rows_in_use<kQuantThreads>(a.offset, a.E, a.num_rows);
  if (range.bad && a.status != nullptr && blockIdx.x == 0 && threadIdx.x == 0)
    atomicOr(a.status, MOE_FLAG_OFFSET_OUT_OF_RANGE);
  return range;
}
// Whether row r belongs to an expert where malformed offsets leave gaps; r may differ
// from lane to lane.
__device__ __forceinline__ bool row_in_use(const QuantRowsArgs& a, const RowRange& range,
                                           int64_t r) {
  if (!range.bad) return true;
  bool in = false;
  for (int e = 0; e < a.E; ++e) {
    const Segment s = segment(a.offset, e, a.num_rows);
    in |= s.lo <= r && r < s.hi;
  }
  return in;
}

// fp8: eight threads a group of scales.  The rows' pieces, each row's rounded up to whole
// groups, are one list that all threads walk through in steps of the grid, kPieces in
// flight.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kQuantThreads, kFp8Blocks) k_quant_rows_fp8(const QuantRowsArgs a) {
  constexpr int kPieces = 2;
  pdl_wait();
  pdl_launch_dependents();
  const RowRange range = quant_rows_range(a);
  const int pieces = static_cast<int>(a.H / 16);
  const int groups = static_cast<int>((a.H + kQuantGroup - 1) / kQuantGroup), slots = groups * 8;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kQuantThreads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kQuantThreads + threadIdx.x;
  const int64_t step_rows = step / slots;
  const int step_slots = static_cast<int>(step % slots);
  int64_t row = range.lo + first / slots;
  int slot = static_cast<int>(first % slots);
  const T* rows = static_cast<const T*>(a.rows);
  // (the lanes of a warp end in different rounds, but it stays together)
  while (__any_sync(kFullMask, row < range.hi)) {
    Piece p[kPieces];
    int64_t at_row[kPieces];
    int at[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      at_row[i] = row, at[i] = slot;
      if (row < range.hi && slot < pieces) {
        p[i] = load_piece<kWide>(rows + row * a.H + slot * 16);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[i].v[j] = 0;
      }
      row += step_rows, slot += step_slots;
      if (slot >= slots) slot -= slots, ++row;
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      uint32_t m = piece_max_numbers<T>(p[i]);
#pragma unroll
      for (int d = 1; d < 8; d *= 2) m = __vmaxu2(m, __shfl_xor_sync(kFullMask, m, d));
      const float amax = magnitude<T>(halves_max(m));
      const float scale = amax > 0.f ? __fdiv_rn(amax, kE4m3Max) : 1.f;
      if (at_row[i] >= range.hi || at[i] >= pieces || !row_in_use(a, range, at_row[i])) continue;
      if (at[i] % 8 == 0) a.scales[at_row[i] * groups + at[i] / 8] = scale;
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.codes) + at_row[i] * a.H + at[i] * 16) =
          fp8_codes<T>(p[i], scale);
    }
  }
}

// int8: `kRowThreads` threads a row, which stays in their registers between its maximum
// and its codes (kHeld pieces each; what a wider row has beyond is read twice).
template <typename T, bool kWide, int kRowThreads, int kHeld>
__global__ void __launch_bounds__(kQuantThreads, kInt8Blocks) k_quant_rows_int8(const QuantRowsArgs a) {
  constexpr int kRows = kQuantThreads / kRowThreads;  // of a block at a time
  __shared__ uint32_t s_max[2][kQuantThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const RowRange range = quant_rows_range(a);
  const int pieces = static_cast<int>(a.H / 16);
  const int lane = threadIdx.x % kRowThreads;  // of the row's
  int turn = 0;
  for (int64_t r0 = range.lo + static_cast<int64_t>(blockIdx.x) * kRows; r0 < range.hi;
       r0 += static_cast<int64_t>(gridDim.x) * kRows, turn ^= 1) {
    const int64_t r = r0 + threadIdx.x / kRowThreads;
    const bool in = r < range.hi && row_in_use(a, range, r);
    const T* row = static_cast<const T*>(a.rows) + r * a.H;
    Piece p[kHeld];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int at = lane + i * kRowThreads;
      if (in && at < pieces) {
        p[i] = load_piece<kWide>(row + at * 16);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[i].v[j] = 0;
      }
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) m = __vmaxu2(m, piece_max(p[i]));
    if (in)
      for (int at = lane + kHeld * kRowThreads; at < pieces; at += kRowThreads)
        m = __vmaxu2(m, piece_max(load_piece<kWide>(row + at * 16)));
    m = halves_max(m);
    m = __reduce_max_sync(kFullMask, m);
    if (kRowThreads > 32) {
      if (threadIdx.x % 32 == 0) s_max[turn][threadIdx.x / 32] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kRowThreads / 32; ++i)
        m = max(m, s_max[turn][threadIdx.x / kRowThreads * (kRowThreads / 32) + i]);
    }
    if (!in) continue;
    const float amax = magnitude<T>(m);  // NaN if the row has one
    const float scale = m > 0 ? __fdiv_rn(amax, kInt8Max) : 1.f;
    if (lane == 0) a.scales[r] = scale;
    uint8_t* codes = static_cast<uint8_t*>(a.codes) + r * a.H;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int at = lane + i * kRowThreads;
      if (at < pieces) *reinterpret_cast<uint4*>(codes + at * 16) = int8_codes<T>(p[i], scale);
    }
    for (int at = lane + kHeld * kRowThreads; at < pieces; at += kRowThreads)
      *reinterpret_cast<uint4*>(codes + at * 16) =
          int8_codes<T>(load_piece<kWide>(row + at * 16), scale);
  }
}

}  // namespace experts
}  // namespace moe
