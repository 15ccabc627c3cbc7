// product_host.cuh -- host side of the tiled products: TMA maps of their operands and
// the number of their tiles.
#pragma once

#include <algorithm>
#include <type_traits>

#include "expert_decode.cuh"
#include "expert_product.cuh"
#include "host_util.cuh"

namespace moe {
namespace experts {
namespace {

// cuTensorMapEncodeTiled, looked up once: the library is not linked against
// the driver.
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// Values of 128 bytes.
template <typename T>
constexpr int kLineValues = 128 / static_cast<int>(sizeof(T));

// A TMA map: sizes and boxes in elements, fastest dimension first, the pitches of
// the others; a tile's rows are 128 bytes, in the 128-byte swizzle.  What a
// tile reaches outside reads as zero.  L2 fetches 256 bytes at a time, the next slice
// of a row with this one, where rows are whole 128-byte lines (Qwen3-shaped gated
// T = 64 97 us, 99 with 128); elsewhere 128 (training step of 792 -> 2 x 11784 495
// us, 532 with 256).
template <typename T, int kDims>
bool make_map_nd(CUtensorMap* map, const void* base, const int64_t (&size)[kDims],
                 const int64_t (&pitch)[kDims - 1], const int (&box_size)[kDims]) {
  const EncodeFn encode = encode_fn();
  if (encode == nullptr) return false;
  cuuint64_t dims[kDims], strides[kDims - 1];
  cuuint32_t box[kDims], steps[kDims];
  for (int i = 0; i < kDims; ++i) {
    dims[i] = static_cast<cuuint64_t>(size[i]);
    box[i] = static_cast<cuuint32_t>(box_size[i]);
    steps[i] = 1;
    if (i + 1 < kDims) strides[i] = static_cast<cuuint64_t>(pitch[i]) * sizeof(T);
  }
  constexpr CUtensorMapDataType kType =
      sizeof(T) == 1                            ? CU_TENSOR_MAP_DATA_TYPE_UINT8
      : std::is_same<T, __nv_bfloat16>::value ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return encode(map, kType, kDims, const_cast<void*>(base), dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                pitch[0] % kLineValues<T> == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                   : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [planes, rows, cols] (two dimensions with planes = 0), tiles of box_rows rows.
template <typename T>
bool make_map(CUtensorMap* map, const void* base, int64_t planes, int64_t rows, int64_t cols,
              int box_rows) {
  if (planes == 0) return make_map_nd<T, 2>(map, base, {cols, rows}, {cols}, {kLineValues<T>, box_rows});
  return make_map_nd<T, 3>(map, base, {cols, rows, planes}, {cols, cols * rows},
                            {kLineValues<T>, box_rows, 1});
}

// The weight [E, N, K] as [E, K/64, N, 64] (8 bits: 128 for 64), tiles of blocks x rows
// x 64.
template <typename T>
bool make_decode_map(CUtensorMap* map, const void* base, int64_t E, int64_t N, int64_t K) {
  constexpr int kLine = kLineValues<T>;
  return make_map_nd<T, 4>(map, base, {kLine, N, K / kLine, E}, {K, kLine, N * K},
                           {kLine, kDecodeFeatures, kDecodeBlocks, 1});
}

// The gated weight [E, 2, F, K] as [E, F/8, 2, 8, K], tiles of 8 x 2 x 8 rows by 64: in
// an A tile 8 gate rows and the 8 up rows of the same features take turns, so that
// they meet in the tensor memory lanes that one thread reads.  One load takes the
// whole tile (as four, the products of 2048 -> 2 x 768 ran 11% slower).
template <typename T>
bool make_gated_map(CUtensorMap* map, const void* base, int64_t E, int64_t F, int64_t K) {
  return make_map_nd<T, 5>(map, base, {K, 8, 2, F / 8, E}, {K, F * K, 8 * K, 2 * F * K},
                           {kLineValues<T>, 8, 2, 8, 1});
}

// The most tiles a product may have, of `step` features and at most `columns` columns
// each.
template <int kUse, typename Args>
int64_t most_tiles(const Args& a, int columns, int step = m_step<kUse>()) {
  const int64_t m = kUse == kForward || kUse == kWeightGrad ? a.N : kUse == kGated ? a.N / 2 : a.K;
  const int64_t blocks = kUse == kWeightGrad ? a.E * ceil_div(a.K, kMaxN)
                         : a.E == 1          ? ceil_div(a.num_rows, columns)
                                    : a.num_rows / columns + std::min<int64_t>(a.E, a.num_rows);
  return ceil_div(m, step) * blocks;
}

// Pairs that share a tile, each with 4 slices at least.
int tile_splits(int64_t tiles, int64_t slices, int64_t pairs) {
  return tiles * kMaxSplits <= pairs && slices >= 4 * kMaxSplits ? kMaxSplits : 1;
}

}  // namespace
}  // namespace experts
}  // namespace moe
