// expert_product.cuh -- the grouped matrix products, on tcgen05.
//
// Three uses of one kernel, per expert e with its rows r in [lo, hi):
//   forward   Z[n, r] = sum_k W[e][n,k] x[r,k]     A = W  (k contiguous)   B = x  (k contiguous)
//   d_rows    X[k, r] = sum_n W[e][n,k] dz[r,n]    A = W  (m contiguous)   B = dz (k contiguous)
//   d_weight  G[n, k] = sum_r dz[r,n] x[r,k]       A = dz (m contiguous)   B = x  (n contiguous)
// Weights are the A operand, so that the ragged number of rows is the MMA's N,
// which goes in steps of 16: a segment costs its own rows rounded up to 16,
// not to 128, and a single row costs one 16-column product.
//
// A block computes 256 x (up to 256) outputs: two A tiles of 128 rows (forward
// gated: the gate rows and the up rows of the same 128 features, so that the
// activation and the product happen in registers; else 256 consecutive ones)
// against one B tile, accumulated in all 512 columns of tensor memory.
//   warps 0-7  epilogue: tensor memory -> registers -> shared -> rows
//   warp 8     TMA producer: 64-deep slices into kStages stages of 64 KB
//   warp 9     tcgen05.mma issue, and tensor memory allocation
// The grid is persistent; tiles are numbered expert by expert, the row blocks
// of one weight tile next to each other so that they share it in L2.
#pragma once

#include "expert_math.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace experts {

enum Use { kForward, kGated, kRowsGrad, kWeightGrad };

constexpr int kMaxN = 256;     // columns of one accumulator
constexpr int kSlice = 64;     // contraction depth of one stage: 128 bytes
constexpr int kStages = 3;
constexpr int kTileABytes = 128 * kSlice * 2;
constexpr int kTileBBytes = kMaxN * kSlice * 2;
constexpr int kStageBytes = 2 * kTileABytes + kTileBBytes;
constexpr int kBoxRows = 32;   // rows of one TMA box of a k-contiguous B
constexpr int kEpiWarps = 8;
constexpr int kProductThreads = (kEpiWarps + 2) * 32;
// Staging of 16 columns of a warp's block: 16 rows of 32 values transposed, or
// 32 rows of 16, each padded by 4 against bank conflicts.
constexpr int kStageFloats = 32 * (16 + 4);
constexpr int kStagingBytes = kEpiWarps * kStageFloats * 4;

struct ProductArgs {
  const int64_t* offset;
  int64_t num_rows;
  int64_t K, N;  // in_size and out_size of the weight [E, N, K]
  int E;
  int act;
  const void* bias;
  const void* residual;
  void* out;
  void* preact;
  unsigned* status;
};

// Dynamic shared memory: stages (1024-byte aligned), staging, tile numbers.
inline size_t product_smem(int E) {
  return 1024 + kStages * kStageBytes + kStagingBytes + static_cast<size_t>(E + 1) * 4;
}

struct Tile {
  int e, lo, rows;  // expert; first row and row count (d_weight: all of e's rows)
  int m0, n0;       // first output feature; d_weight: first column
};

// Row blocks of a segment: as few as fit, of even size (a multiple of 16).
__device__ __forceinline__ int row_blocks(int rows) { return (rows + kMaxN - 1) / kMaxN; }
__device__ __forceinline__ int block_rows(int rows, int blocks) {
  return ((rows + blocks - 1) / blocks + 15) / 16 * 16;
}

// Output features of one tile.
template <int kUse>
__device__ __forceinline__ int m_step() { return kUse == kGated ? 128 : 256; }

template <int kUse>
__device__ __forceinline__ Tile find_tile(const ProductArgs& a, const int* first, int t,
                                          int m_blocks, int n_blocks) {
  Tile r;
  if (kUse == kWeightGrad) {
    const int per = m_blocks * n_blocks;
    r.e = t / per;
    const int local = t - r.e * per;
    const Segment s = segment(a.offset, r.e, a.num_rows);
    r.lo = s.lo;
    r.rows = s.hi - s.lo;
    r.m0 = local / n_blocks * m_step<kUse>();
    r.n0 = local % n_blocks * kMaxN;
    return r;
  }
  int lo = 0, hi = a.E;  // first[lo] <= t < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first[mid] <= t) lo = mid;
    else hi = mid;
  }
  r.e = lo;
  const Segment s = segment(a.offset, lo, a.num_rows);
  const int rows = s.hi - s.lo;
  const int blocks = row_blocks(rows), step = block_rows(rows, blocks);
  const int local = t - first[lo];
  const int b = local % blocks;
  r.lo = s.lo + b * step;
  r.rows = min(step, rows - b * step);
  r.m0 = local / blocks * m_step<kUse>();
  r.n0 = 0;
  return r;
}

// Eight consecutive outputs of a row, rounded and stored as 16 bytes.
template <typename T>
__device__ __forceinline__ void store8(T* dst, const float* v) {
  Vec8<T> o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o.e[i] = from_f<T>(v[i]);
  *reinterpret_cast<uint4*>(dst) = o.v;
}

template <int kAct>
__device__ __forceinline__ void apply_act(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = act<kAct>(v[i]);
}
__device__ __forceinline__ void apply_act(int a, float (&v)[32]) {
  if (a == MOE_ACT_SILU) apply_act<MOE_ACT_SILU>(v);
  else if (a == MOE_ACT_GELU) apply_act<MOE_ACT_GELU>(v);
  else if (a == MOE_ACT_RELU) apply_act<MOE_ACT_RELU>(v);
}

// A warp's 32 x 32 values, lane l holding v[j] = value (l, j), to the matrix
// `out` of row pitch `pitch`: transposed, value (l, j) goes to row r0 + j,
// column c0 + l; else to row r0 + l, column c0 + j.  Rows and columns from
// `rows` and `cols` on are left out (cols is a multiple of 8).  Through shared
// memory, so that neighbouring lanes write consecutive bytes of a row (64
// transposed, 32 not: whole sectors).
template <typename T, bool kTranspose>
__device__ __forceinline__ void write_block(const float (&v)[32], float* stage, T* out,
                                            const T* residual, int64_t pitch, int64_t r0, int rows,
                                            int64_t c0, int64_t cols) {
  constexpr int kPitch = kTranspose ? 36 : 20;
  constexpr int kLanesPerRow = kTranspose ? 4 : 2;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 0; h < 32; h += 16) {
    __syncwarp();
    if (kTranspose) {
#pragma unroll
      for (int j = 0; j < 16; ++j) stage[j * kPitch + lane] = v[h + j];
    } else {
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<float4*>(stage + lane * kPitch + j) =
            make_float4(v[h + j], v[h + j + 1], v[h + j + 2], v[h + j + 3]);
    }
    __syncwarp();
    const int seg = lane % kLanesPerRow * 8;
    const int64_t col = c0 + seg + (kTranspose ? 0 : h);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = i * (32 / kLanesPerRow) + lane / kLanesPerRow;
      const int row = r + (kTranspose ? h : 0);
      if (row >= rows || col >= cols) continue;
      const float4* src = reinterpret_cast<const float4*>(stage + r * kPitch + seg);
      const float4 p = src[0], q = src[1];
      float w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
      const int64_t at = (r0 + row) * pitch + col;
      if (residual != nullptr) {
        Vec8<T> x;
        x.v = *reinterpret_cast<const uint4*>(residual + at);
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] += to_f(x.e[k]);
      }
      store8(out + at, w);
    }
  }
}

// map_a, map_b: the operands as TMA tiles of 64 contiguous values (128 bytes,
// 128-byte swizzle) by 128 (forward A), 64 (MN-major) or kBoxRows rows.
template <typename T, int kUse>
__global__ void __launch_bounds__(kProductThreads, 1)
k_expert_product(const __grid_constant__ CUtensorMap map_a,
                 const __grid_constant__ CUtensorMap map_b, const ProductArgs a) {
  constexpr bool kBf16 = sizeof(T) == 2 && !__is_same(T, __half);
  constexpr bool kAMn = kUse == kRowsGrad || kUse == kWeightGrad;
  constexpr bool kBMn = kUse == kWeightGrad;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_done, s_free;
  __shared__ uint32_t s_tmem;
  __shared__ int s_gave_up, s_scan[32];

  uint8_t* stages = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* staging = reinterpret_cast<float*>(stages + kStages * kStageBytes);
  int* first = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(staging) + kStagingBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&s_full[i]), 1);
      mbar_init(smem_addr(&s_empty[i]), 1);
    }
    mbar_init(smem_addr(&s_done), 1);
    mbar_init(smem_addr(&s_free), kEpiWarps);
    mbar_init_fence();
    s_gave_up = 0;
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
  }
  if (warp == kEpiWarps + 1) tmem_alloc(smem_addr(&s_tmem), 512);
  pdl_wait();

  // Tiles of each expert, and the sum before it.
  const int F = static_cast<int>(a.N / 2);
  const int m_size = static_cast<int>(kUse == kForward ? a.N : kUse == kGated ? F
                                      : kUse == kRowsGrad ? a.K : a.N);
  const int m_blocks = (m_size + m_step<kUse>() - 1) / m_step<kUse>();
  const int n_blocks = static_cast<int>((a.K + kMaxN - 1) / kMaxN);  // d_weight
  int total = 0;
  bool bad = false;
  for (int e0 = 0; e0 < a.E; e0 += kProductThreads) {
    const int e = e0 + threadIdx.x;
    int n = 0;
    if (e < a.E) {
      bool b;
      const Segment s = segment(a.offset, e, a.num_rows, &b);
      bad |= b;
      n = row_blocks(s.hi - s.lo) * m_blocks;
    }
    int part;
    const int before = block_exclusive_sum(n, s_scan, &part);
    if (e < a.E) first[e] = total + before;
    total += part;
  }
  if (threadIdx.x == 0) first[a.E] = total;
  if (kUse == kWeightGrad) total = a.E * m_blocks * n_blocks;
  if (a.status != nullptr && blockIdx.x == 0 && bad)
    atomicOr(a.status, MOE_FLAG_OFFSET_OUT_OF_RANGE);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* gave_up = &s_gave_up;

  // Slices of the contraction (d_weight: of the expert's rows).
  const int k_size = static_cast<int>(kUse == kRowsGrad ? a.N : a.K);
  auto slices = [&](const Tile& t) {
    return ((kUse == kWeightGrad ? t.rows : k_size) + kSlice - 1) / kSlice;
  };
  // Columns of the tile, and whether its second A tile holds anything.
  auto columns = [&](const Tile& t) {
    return kUse == kWeightGrad ? min(kMaxN, static_cast<int>(a.K) - t.n0) : t.rows;
  };
  auto two = [&](const Tile& t) { return kUse == kGated || t.m0 + 128 < m_size; };

  if (warp == kEpiWarps) {
    if (lane == 0) {
      uint32_t step = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const Tile tile = find_tile<kUse>(a, first, t, m_blocks, n_blocks);
        const int n_slices = slices(tile), cols = columns(tile);
        const int a_tiles = two(tile) ? 2 : 1;
        const int b_boxes = kBMn ? (cols + 63) / 64 : (cols + kBoxRows - 1) / kBoxRows;
        const uint32_t bytes = a_tiles * kTileABytes +
                               b_boxes * (kBMn ? 64 * kSlice * 2 : kBoxRows * kSlice * 2);
        for (int s = 0; s < n_slices; ++s, ++step) {
          const int st = step % kStages;
          const uint32_t full = smem_addr(&s_full[st]);
          if (!mbar_wait(smem_addr(&s_empty[st]), (step / kStages & 1) ^ 1, gave_up)) {
            ok = false;
            break;
          }
          mbar_expect(full, bytes);
          const uint32_t sa = smem_addr(stages + st * kStageBytes);
          const uint32_t sb = sa + 2 * kTileABytes;
          const int k = s * kSlice;
          for (int i = 0; i < a_tiles; ++i) {
            const int m = tile.m0 + (kUse == kGated ? i * F : i * 128);
            const uint32_t dst = sa + i * kTileABytes;
            if (kUse == kForward || kUse == kGated) {
              tma_load_3d(dst, &map_a, k, m, tile.e, full);
            } else if (kUse == kRowsGrad) {
              tma_load_3d(dst, &map_a, m, k, tile.e, full);
              tma_load_3d(dst + kTileABytes / 2, &map_a, m + 64, k, tile.e, full);
            } else {
              tma_load_2d(dst, &map_a, m, tile.lo + k, full);
              tma_load_2d(dst + kTileABytes / 2, &map_a, m + 64, tile.lo + k, full);
            }
          }
          for (int i = 0; i < b_boxes; ++i) {
            if (kBMn)
              tma_load_2d(sb + i * 64 * kSlice * 2, &map_b, tile.n0 + i * 64, tile.lo + k, full);
            else
              tma_load_2d(sb + i * kBoxRows * kSlice * 2, &map_b, k, tile.lo + i * kBoxRows, full);
          }
        }
      }
      // Nothing of this block may still be in flight when it ends.  After an
      // ordinary run the MMA warp has seen every load; after a wait gave up,
      // the loads are given the time of one wait to land.
      if (*gave_up != 0) {
        const unsigned long long t0 = now_ns();
        for (int i = 0; i < kStages && step > 0; ++i) {
          const uint32_t last = step - 1 - i;  // the newest load of its stage
          if (static_cast<int>(last) < 0) break;
          while (!mbar_try(smem_addr(&s_full[last % kStages]), last / kStages & 1) &&
                 now_ns() - t0 < kWaitNs) {
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == kEpiWarps + 1) {
    uint32_t step = 0, done = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const Tile tile = find_tile<kUse>(a, first, t, m_blocks, n_blocks);
      const int n_slices = slices(tile);
      if (n_slices == 0) continue;
      const int n = (columns(tile) + 15) / 16 * 16;
      const bool both = two(tile);
      const uint32_t idesc = instr_desc(kBf16, kAMn, kBMn, 128, n);
      if (!warp_wait(smem_addr(&s_free), (done & 1) ^ 1, gave_up)) break;
      tc_fence_after();
      for (int s = 0; s < n_slices; ++s, ++step) {
        const int st = step % kStages;
        if (!warp_wait(smem_addr(&s_full[st]), step / kStages & 1, gave_up)) {
          ok = false;
          break;
        }
        uint8_t* sa = stages + st * kStageBytes;
        uint8_t* sb = sa + 2 * kTileABytes;
        int depth = 4;  // products of 16 k-values each
        if (kUse == kWeightGrad) {
          const int left = tile.rows - s * kSlice;
          if (left < kSlice) {
            // The slice runs past the expert's rows.  What follows belongs to
            // another expert or to none and may be infinite or NaN, so it is
            // overwritten in both operands rather than multiplied by zeros.
            depth = (left + 15) / 16;
            const int rows = depth * 16 - left;
            for (int i = lane; i < rows * 64; i += 32) {
              const int box = i / 8 & 7, r = left + i / 64;
              uint8_t* at = box < 4 ? sa + box * (kTileABytes / 2)
                                    : sb + (box - 4) * (kTileBBytes / 4);
              *reinterpret_cast<uint4*>(at + r * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_async_shared();
            __syncwarp();
          }
        }
        tc_fence_after();
        if (lane == 0) {
          constexpr uint32_t kStepA = kAMn ? 2048 : 32, kStepB = kBMn ? 2048 : 32;
          const uint32_t pa = smem_addr(sa), pb = smem_addr(sb);
          for (int i = 0; i < depth; ++i) {
            const uint64_t db = smem_desc(pb + i * kStepB, kBMn ? 8192 : 16, 1024);
            const bool acc = s > 0 || i > 0;
            tc_mma(tmem, smem_desc(pa + i * kStepA, kAMn ? 8192 : 16, 1024), db, idesc, acc);
            if (both)
              tc_mma(tmem + kMaxN,
                     smem_desc(pa + kTileABytes + i * kStepA, kAMn ? 8192 : 16, 1024), db, idesc,
                     acc);
          }
          tc_commit(smem_addr(&s_empty[st]));
          if (s == n_slices - 1) tc_commit(smem_addr(&s_done));
        }
        __syncwarp();
      }
      ++done;
    }
    // The products are over before the memory they read and write is given up.
    if (*gave_up != 0 && lane == 0) {
      const unsigned long long t0 = now_ns();
      for (int i = 0; i < kStages; ++i) {
        const uint32_t last = step - 1 - i;
        if (static_cast<int>(last) < 0) break;
        while (!mbar_try(smem_addr(&s_empty[last % kStages]), last / kStages & 1) &&
               now_ns() - t0 < kWaitNs) {
        }
      }
    }
    __syncwarp();
  } else {
    const int quad = warp & 3, half = warp >> 2;
    float* stage = staging + warp * kStageFloats;
    T* out = static_cast<T*>(a.out);
    T* preact = static_cast<T*>(a.preact);
    const T* residual = static_cast<const T*>(a.residual);
    uint32_t done = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
      const Tile tile = find_tile<kUse>(a, first, t, m_blocks, n_blocks);
      const int cols = columns(tile);
      const bool any = slices(tile) > 0;
      if (any) {
        if (!warp_wait(smem_addr(&s_done), done & 1, gave_up)) break;
        tc_fence_after();
      }
      const uint32_t base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
      for (int c = half * 32; c < cols; c += 64) {
        const int64_t m = tile.m0 + quad * 32;  // the warp's first feature
        if (kUse == kGated) {
          float g[32], u[32];
          tmem_load32(base + c, g);
          tmem_load32(base + kMaxN + c, u);
          tmem_wait_load(g);
          tmem_wait_load(u);
          if (preact != nullptr) {
            write_block<T, true>(g, stage, preact, nullptr, a.N, tile.lo + c, cols - c, m, F);
            write_block<T, true>(u, stage, preact + F, nullptr, a.N, tile.lo + c, cols - c, m, F);
          }
          apply_act(a.act, g);
#pragma unroll
          for (int i = 0; i < 32; ++i) g[i] *= u[i];
          write_block<T, true>(g, stage, out, nullptr, F, tile.lo + c, cols - c, m, F);
        } else {
          const int parts = two(tile) ? 2 : 1;
          for (int i = 0; i < parts; ++i) {
            const int64_t mi = m + i * 128;
            float z[32];
            if (any) {
              tmem_load32(base + i * kMaxN + c, z);
              tmem_wait_load(z);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) z[j] = 0.f;
            }
            if (kUse == kForward) {
              if (a.bias != nullptr && mi + lane < a.N) {
                const float bias = to_f(static_cast<const T*>(
                    a.bias)[static_cast<int64_t>(tile.e) * a.N + mi + lane]);
#pragma unroll
                for (int j = 0; j < 32; ++j) z[j] += bias;
              }
              if (preact != nullptr)
                write_block<T, true>(z, stage, preact, nullptr, a.N, tile.lo + c, cols - c, mi,
                                     a.N);
              apply_act(a.act, z);
              write_block<T, true>(z, stage, out, residual, a.N, tile.lo + c, cols - c, mi, a.N);
            } else if (kUse == kRowsGrad) {
              write_block<T, true>(z, stage, out, nullptr, a.K, tile.lo + c, cols - c, mi, a.K);
            } else {
              const int64_t left = a.N - mi;
              write_block<T, false>(z, stage, out, nullptr, a.K,
                                    static_cast<int64_t>(tile.e) * a.N + mi,
                                    static_cast<int>(left < 32 ? (left < 0 ? 0 : left) : 32),
                                    tile.n0 + c, a.K);
            }
          }
        }
      }
      if (any) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&s_free));
        ++done;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && *gave_up != 0 && a.status != nullptr)
    atomicOr(a.status, MOE_FLAG_BARRIER_TIMEOUT);
  if (warp == kEpiWarps + 1) tmem_free(tmem, 512);
}

}  // namespace experts
}  // namespace moe
