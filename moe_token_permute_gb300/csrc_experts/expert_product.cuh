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
// A pair of blocks (two SMs, cta_group::2) computes 256 x (up to 256) outputs: an
// A tile of 128 rows in each block against one B tile of which each block holds
// half the columns.  Gated: an A tile holds 8 gate rows and the 8 up rows of the same
// features in turns, so that both of an output meet in one thread's registers.  Tensor
// memory (512 columns) holds two accumulators: the epilogue of one tile overlaps the
// products of the next.
//   warps 0-7  epilogue: tensor memory -> registers -> shared -> rows
//   warp 8     TMA producer: 64-deep slices into a ring of 6 x 32 KB
//   warp 9     tcgen05.mma issue (first block), tensor memory allocation
//   warp 10    d_weight: clears what a slice holds beyond the expert's rows
// What bounds it: a slice of 256 columns is 512 cycles of products, for which a
// block loads 32 KB into shared memory and tcgen05 reads 32 KB of it: 128 bytes a
// cycle, all there is.  (A block on its own, without the pair, would need 160.
// Two A tiles per block need 112, but fill tensor memory, and then every tile's
// epilogue holds the products up: Qwen3-shaped training 5% slower, many experts of
// 128 rows 1% faster.)  Large products run at the power limit: Mixtral-shaped
// gated T = 4096 at 1.83-1.90 PFLOP/s in a burst and 1.53-1.60 over seconds.  With few rows
// per expert the weights' way from memory bounds it: Qwen3-shaped gated T = 64 at
// 6.2 TB/s.  Rows that are not whole 128-byte lines make every load touch two lines
// for one (a contraction of 792 takes 1.65 times as long as one of 768).
// The grid is persistent; tiles are numbered expert by expert, in panels.
// Where the tiles of a forward product or d_rows are at most half as many as the pairs
// (a dense layer and few rows; counted as if every expert had rows), two pairs make a
// cluster and share a tile's contraction: each takes half of its slices, the second leaves its sums in its own shared memory, and the
// first adds them to its own through the cluster.  Dense 4096 -> 4096, 64 rows: 16
// us instead of 22; four pairs, whose clusters do not all run at once, 26.  d_weight
// is not shared: one expert of 512 x 256 is two tiles, and its rows go through two of
// the 76 pairs.
#pragma once

#include "expert_math.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace experts {

enum Use { kForward, kGated, kRowsGrad, kWeightGrad };

constexpr int kMaxN = 256;     // columns of one accumulator
constexpr int kSlice = 64;     // contraction depth of one stage: 128 bytes
constexpr int kTileABytes = 128 * kSlice * 2;
constexpr int kTileBBytes = kMaxN / 2 * kSlice * 2;
constexpr int kStageBytes = kTileABytes + kTileBBytes;
constexpr int kStages = 6;
constexpr int kMaxSplits = 2;  // pairs of a cluster
// Slices of a d_weight tile multiplied before its tail slice, which was loaded first
// (Mixtral-shaped linear training step, 1024 rows per expert: 1702 us; 1767 without
// the delay, 1835 with the tail loaded last).
constexpr int kTailDelay = 3;
constexpr int kBoxBytes = 64 * kSlice * 2;  // a TMA load of B: 64 rows or columns of a slice
constexpr int kEpiWarps = 8;
constexpr int kProductThreads = (kEpiWarps + 3) * 32;
constexpr int kStagingWarpBytes = 32 * 64;  // 32 x 32 outputs of 16 bits
constexpr int kStagingBytes = kEpiWarps * kStagingWarpBytes;

struct ProductArgs {
  const int64_t* offset;
  int64_t num_rows;
  int64_t K, N;  // in_size and out_size of the weight [E, N, K]
  int E;
  int act;
  // The launch before is another of the same call and reads what this one reads:
  // nothing is waited for at the start, and that launch at the end.  What both read was
  // written before that launch: it must wait (pdl_wait) ahead of letting this one start
  // (pdl_launch_dependents) in every block, so that all earlier launches are over and
  // their writes performed when this one begins.  k_bias_grad and the products do;
  // so must whatever else is ever put in front of such a launch.
  bool beside_previous;
  const void* bias;
  const void* residual;
  void* out;
  void* preact;
  unsigned* status;
};

// Dynamic shared memory: stages (1024-byte aligned), staging, then each
// expert's rows and its first tile.
inline size_t product_smem(int E) {
  return 1024 + kStages * kStageBytes + kStagingBytes + static_cast<size_t>(E) * 12 + 4;
}

static_assert(1024 + kStages * kStageBytes + kStagingBytes + MOE_MAX_LOCAL_EXPERTS * 12 + 4 + 1024 <=
                  227 * 1024,
              "shared memory of one block");

struct Tile {
  int e, lo, rows;  // expert; first row and row count (d_weight: all of e's rows)
  int m0, n0, cols;  // first output feature; d_weight: first column and their number
};

// Row blocks of a segment, and column blocks of a d_weight: as few as fit, of even
// size (a multiple of 16).
__device__ __forceinline__ int row_blocks(int rows, int most) { return (rows + most - 1) / most; }
__device__ __forceinline__ int even_step(int size, int blocks) {
  return ((size + blocks - 1) / blocks + 15) / 16 * 16;
}

// Output features of one tile.
template <int kUse>
__host__ __device__ constexpr int m_step() { return kUse == kGated ? 128 : 256; }

// The most columns of a tile, chosen for the rows there are.  Six waves of tiles
// and more are cut into 256.  Below, fewer columns can fill the waves better, but a
// slice costs 256 + columns cycles (its traffic in shared memory) whether or not the
// products need them, and a tile about 700 to its first product.  Dense 4096 ->
// 4096: 500 rows 25 us in blocks of 128 and 31 of 256, 8191 rows 238 and 166.
constexpr int kCaps = 13;  // 256, 240, ..., 64
constexpr int kLeastCap = kMaxN - 16 * (kCaps - 1);
__device__ __forceinline__ int cap_of(int i) { return kMaxN - 16 * i; }
__device__ __forceinline__ float cap_cost(int blocks, int rows, int m_blocks, int slices, int pairs) {
  const int64_t waves = (static_cast<int64_t>(blocks) * m_blocks + pairs - 1) / pairs;
  const float columns = static_cast<float>(rows) / static_cast<float>(max(blocks, 1));
  return static_cast<float>(waves) * (static_cast<float>(slices) * (256.f + columns) + 700.f);
}

// Tile `local` of an expert's m_blocks x n_blocks, in panels of kPanel column
// blocks, all of a panel's row blocks after one another: the tiles that run at the
// same time make a square of about kPanel x 76 / kPanel, whose operands together
// are small enough to be shared through L2 (dense 4096 -> 4096, 16384 rows: 333 us
// instead of 389 with all column blocks in one panel).
constexpr int kPanel = 8;
__device__ __forceinline__ void place_in_panels(int local, int m_blocks, int n_blocks, int& m,
                                                int& n) {
  const int panel = local / (kPanel * m_blocks);
  const int width = min(kPanel, n_blocks - panel * kPanel);
  local -= panel * kPanel * m_blocks;
  m = local / width;
  n = panel * kPanel + local - m * width;
}

template <int kUse>
__device__ __forceinline__ Tile find_tile(int E, const Segment* segments, const int* first, int t,
                                          int m_blocks, int n_blocks, int n_size, int cap) {
  Tile r;
  if (kUse == kWeightGrad) {
    const int per = m_blocks * n_blocks;
    const int place = t / per;
    r.e = first[place];  // experts by falling number of rows
    const Segment s = segments[r.e];
    r.lo = s.lo;
    r.rows = s.hi - s.lo;
    int m, n;
    place_in_panels(t - place * per, m_blocks, n_blocks, m, n);
    r.m0 = m * m_step<kUse>();
    const int step = even_step(n_size, n_blocks);
    r.n0 = n * step;
    r.cols = min(step, n_size - r.n0);
    return r;
  }
  int lo = 0, hi = E;  // first[lo] <= t < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first[mid] <= t) lo = mid;
    else hi = mid;
  }
  r.e = lo;
  const Segment s = segments[lo];
  const int rows = s.hi - s.lo;
  const int blocks = row_blocks(rows, cap), step = even_step(rows, blocks);
  int m, n;
  place_in_panels(t - first[lo], m_blocks, blocks, m, n);
  r.lo = s.lo + n * step;
  r.rows = min(step, rows - n * step);
  r.m0 = m * m_step<kUse>();
  r.n0 = 0;
  r.cols = r.rows;
  return r;
}

template <int kCount, int kAct>
__device__ __forceinline__ void apply_act(float* v) {
#pragma unroll
  for (int i = 0; i < kCount; ++i) v[i] = act<kAct>(v[i]);
}
template <int kCount>
__device__ __forceinline__ void apply_act(int a, float* v) {
  if (a == MOE_ACT_SILU) apply_act<kCount, MOE_ACT_SILU>(v);
  else if (a == MOE_ACT_GELU) apply_act<kCount, MOE_ACT_GELU>(v);
  else if (a == MOE_ACT_RELU) apply_act<kCount, MOE_ACT_RELU>(v);
}

// A warp's block of a matrix in memory: rows r0 + [0, rows), at most 32 (16 with 64
// columns), and columns c0 + [0, kCols) below `cols` (a multiple of 8).  Its shared
// memory copy has rows of kCols values, the 16-byte chunks of some rows exchanged
// so that neither the fragments' accesses (8 rows of a chunk) nor the rows' (128
// bytes) meet in a bank.
template <typename T, int kCols = 32>
struct Block {
  static constexpr int kChunks = kCols / 8;          // 16 bytes each, of a row
  static constexpr int kLaneRows = 32 / kChunks;     // rows the warp reads at once
  T* at;            // the lane's first 8 values: row lane / kChunks, chunk lane % kChunks
  int64_t step;     // kLaneRows rows
  int rows;         // of the lane's rows lane / kChunks + kLaneRows i, those below `rows` exist
  uint32_t line;    // shared memory address of those 8 values
  uint32_t matrix;  // and of the row the lane gives for fragments

  static __device__ __forceinline__ uint32_t place(int row, int chunk) {
    const int turn = kCols == 64 ? row & 7 : kCols == 32 ? row >> 1 & 3 : row >> 2 & 1;
    return row * (kCols * 2) + ((chunk ^ turn) << 4);
  }
  __device__ __forceinline__ Block(T* base, int64_t pitch, int64_t r0, int n_rows, int64_t c0,
                                   int64_t cols, uint32_t stage) {
    const int lane = threadIdx.x & 31, r = lane / kChunks, c = lane % kChunks;
    at = base + (r0 + r) * pitch + c0 + c * 8;
    step = kLaneRows * pitch;
    rows = c0 + c * 8 < cols ? n_rows - r : 0;
    line = stage + place(r, c);
    // 64 and 32 columns: lane l row l % 8 of chunk l / 8; 16: chunk l / 8 % 2 of row
    // l % 8, the upper lanes of row 8 + l % 8.
    const int k = lane >> 3;
    matrix = stage + (kCols == 16 ? place((k >> 1) * 8 + (lane & 7), k & 1) : place(lane & 7, k));
  }
};

__device__ __forceinline__ uint4 shared_load16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void shared_store16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

// v, as tmem_load_32x32 gives it, rounded and written to the block: tensor memory
// lanes are the block's columns.
template <typename T>
__device__ __forceinline__ void write_block(const float (&v)[32], const Block<T>& b) {
  uint32_t p[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) p[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
  __syncwarp();  // the block before this one is read
#pragma unroll
  for (int j = 0; j < 4; ++j)  // p[8 h + 2 i + s]: lanes 16 h + 8 s + [0, 8), columns 8 i + [0, 8)
    store_matrices<true>(b.matrix + j * 512, p[2 * j], p[2 * j + 1], p[8 + 2 * j],
                         p[8 + 2 * j + 1]);
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 x = shared_load16(b.line + j * 512);
    if (8 * j < b.rows) *reinterpret_cast<uint4*>(b.at + j * b.step) = x;
  }
}

// v, as tmem_load_16x64 gives it: tensor memory lanes are the block's rows.  128
// bytes of a row at a time: where rows are not whole sectors, pieces of 64 bytes
// touch three sectors for two.
template <typename T>
__device__ __forceinline__ void write_row_block(const float (&v)[32], const Block<T, 64>& b) {
  uint32_t p[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) p[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
  __syncwarp();  // the block before this one is read
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // p[2 i + s]: lanes 8 s + [0, 8), columns 8 i + [0, 8)
    const int s = j / 2, i = j % 2 * 4;
    store_matrices<false>((b.matrix + s * 1024) ^ (i << 4), p[2 * i + s], p[2 * i + 2 + s],
                          p[2 * i + 4 + s], p[2 * i + 6 + s]);
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 x = shared_load16((b.line + j * 512) ^ (j % 2 * 64));
    if (4 * j < b.rows) *reinterpret_cast<uint4*>(b.at + j * b.step) = x;
  }
}

// The transposed block of 16 columns, v[4 i + 2 s + b] being column 8 s + g and row
// 8 i + 2 q + b.
template <typename T>
__device__ __forceinline__ void write_half_block(const float* v, const Block<T, 16>& b) {
  uint32_t p[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) p[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
  __syncwarp();  // the block before this one is read
#pragma unroll
  for (int j = 0; j < 2; ++j)
    store_matrices<true>(b.matrix + j * 512, p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint4 x = shared_load16(b.line + j * 512);
    if (16 * j < b.rows) *reinterpret_cast<uint4*>(b.at + j * b.step) = x;
  }
}

// v += the block (transposed), in two steps, as its loads take long; what lies
// outside the matrix counts as zero.
template <typename T>
__device__ __forceinline__ void load_block(uint4 (&x)[4], const Block<T>& b) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    x[j] = 8 * j < b.rows ? *reinterpret_cast<const uint4*>(b.at + j * b.step)
                          : make_uint4(0, 0, 0, 0);
}
template <typename T>
__device__ __forceinline__ void add_block(float (&v)[32], const uint4 (&x)[4], const Block<T>& b) {
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) shared_store16(b.line + j * 512, x[j]);
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t r[4];
    load_matrices_transposed(b.matrix + j * 512, r[0], r[1], r[2], r[3]);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float2 f = unpack2<T>(r[m]);
      v[m / 2 * 16 + 4 * j + m % 2 * 2] += f.x;
      v[m / 2 * 16 + 4 * j + m % 2 * 2 + 1] += f.y;
    }
  }
}

// map_a, map_b: the operands as TMA tiles of 64 contiguous values (128 bytes,
// 128-byte swizzle) by 64 rows, A of the forward product by 128.  map_a of the gated
// product: make_gated_map.
template <typename T, int kUse>
__global__ void __launch_bounds__(kProductThreads, 1)
k_expert_product(const __grid_constant__ CUtensorMap map_a,
                 const __grid_constant__ CUtensorMap map_b, const ProductArgs a) {
  constexpr bool kBf16 = sizeof(T) == 2 && !__is_same(T, __half);
  constexpr bool kAMn = kUse == kRowsGrad || kUse == kWeightGrad;
  constexpr bool kBMn = kUse == kWeightGrad;
  extern __shared__ uint8_t smem_raw[];
  // s_full, s_free and s_clear are used in a pair's first block only, s_parts in
  // the cluster's first pair.
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_done[2], s_free[2],
      s_clear[kStages], s_tail[kStages], s_parts;
  __shared__ uint32_t s_tmem;
  __shared__ int s_gave_up, s_cap;
  __shared__ uint32_t s_issued;  // slices that this block's producer has issued

  uint8_t* stages = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* staging = stages + kStages * kStageBytes;
  Segment* segments = reinterpret_cast<Segment*>(staging + kStagingBytes);
  int* first = reinterpret_cast<int*>(segments + a.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Clusters of `splits` pairs; the block's place in its pair; the rank of the
  // pair's first block.
  const uint32_t place = cluster_rank(), leader = place & ~1u;
  const int rank = static_cast<int>(place & 1u), split = static_cast<int>(place / 2);
  const int splits = static_cast<int>(cluster_size() / 2);
  const int pair = blockIdx.x / (2 * splits), pairs = gridDim.x / (2 * splits);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&s_full[i]), 1);
      mbar_init(smem_addr(&s_empty[i]), 1);
      mbar_init(smem_addr(&s_clear[i]), 2);
      mbar_init(smem_addr(&s_tail[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&s_done[i]), 1);
      mbar_init(smem_addr(&s_free[i]), 2 * kEpiWarps);
    }
    mbar_init(smem_addr(&s_parts), kEpiWarps);
    mbar_init_fence();
    s_gave_up = 0;
    s_issued = 0;
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
  }
  __syncthreads();
  cluster_arrive();  // this block's barriers exist
  if (warp == kEpiWarps + 1) tmem_alloc(smem_addr(&s_tmem), 512);
  if (!a.beside_previous) pdl_wait();
  pdl_launch_dependents();

  const int F = static_cast<int>(a.N / 2);
  const int m_size = static_cast<int>(kUse == kForward ? a.N : kUse == kGated ? F
                                      : kUse == kRowsGrad ? a.K : a.N);
  const int m_blocks = (m_size + m_step<kUse>() - 1) / m_step<kUse>();
  const int n_blocks = static_cast<int>((a.K + kMaxN - 1) / kMaxN);  // d_weight
  const int k_size = static_cast<int>(kUse == kRowsGrad ? a.N : a.K);
  const int all_slices = (k_size + kSlice - 1) / kSlice;

  for (int e = threadIdx.x; e < a.E; e += kProductThreads) {
    bool bad;
    segments[e] = segment(a.offset, e, a.num_rows, &bad);
    if (bad && a.status != nullptr && blockIdx.x == 0)
      atomicOr(a.status, MOE_FLAG_OFFSET_OUT_OF_RANGE);
  }
  __syncthreads();
  if (kUse == kWeightGrad) {
    // A tile costs its expert's rows: the experts go by falling rows, and the
    // pairs take the tiles to and fro (Walk), so that each gets its share of the
    // long ones (Zipf 1.2 over 128 experts: the longest pair 1.4% over the average
    // instead of 14%).
    for (int e = threadIdx.x; e < a.E; e += kProductThreads) {
      const int rows = segments[e].hi - segments[e].lo;
      int before = 0;
      for (int f = 0; f < a.E; ++f) {
        const int other = segments[f].hi - segments[f].lo;
        before += other > rows || (other == rows && f < e);
      }
      first[before] = e;
    }
  } else if (warp == 0) {
    // In how many blocks of each size the experts' rows are cut; the choice; and
    // each expert's first tile.
    int cap = kMaxN;
    if (splits == 1) {
      int blocks[kCaps] = {}, all = 0;
      for (int e = lane; e < a.E; e += 32) {
        const int rows = segments[e].hi - segments[e].lo;
        all += rows;
#pragma unroll
        for (int i = 0; i < kCaps; ++i) blocks[i] += row_blocks(rows, cap_of(i));
      }
      all = __reduce_add_sync(kFullMask, all);
      int mine = 0, most = 0;  // lane i: with cap_of(i)
#pragma unroll
      for (int i = 0; i < kCaps; ++i) {
        const int n = __reduce_add_sync(kFullMask, blocks[i]);
        if (i == 0) most = n;
        if (lane == i) mine = n;
      }
      float cost = INFINITY;
      if (lane == 0 || (lane < kCaps && most < (6 * pairs + m_blocks - 1) / m_blocks))
        cost = cap_cost(mine, all, m_blocks, all_slices, pairs);
      float best = cost;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) best = fminf(best, __shfl_xor_sync(kFullMask, best, d));
      cap = cap_of(__ffs(__ballot_sync(kFullMask, cost == best)) - 1);
    }
    // The host has made sure that the tiles of num_rows rows can be counted; where
    // bad offsets make segments overlap, those beyond kMostTiles are left out.
    constexpr int64_t kMostTiles = INT32_MAX / 2;
    int64_t before = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int64_t n = e < a.E ? static_cast<int64_t>(
                                      row_blocks(segments[e].hi - segments[e].lo, cap)) * m_blocks
                                : 0;
      int64_t sum = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(kFullMask, sum, d);
        if (lane >= d) sum += x;
      }
      if (e < a.E) first[e] = static_cast<int>(min(kMostTiles, before + sum - n));
      before += __shfl_sync(kFullMask, sum, 31);
    }
    if (lane == 0) {
      first[a.E] = static_cast<int>(min(kMostTiles, before));
      s_cap = cap;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_wait();  // the other blocks' barriers exist too
  tc_fence_after();
  const int cap = s_cap;
  int total = kUse == kWeightGrad ? a.E * m_blocks * n_blocks : first[a.E];
  // (More tiles than pairs only where bad offsets make segments overlap.)
  if (splits > 1) total = min(total, pairs);
  const uint32_t tmem = s_tmem;
  volatile int* gave_up = &s_gave_up;
  const uint32_t progress = smem_addr(&s_issued);  // of the waits that span a contraction

  // A place in the ring of stages: stage and parity of the pass through them.
  struct Ring {
    int at = 0;
    uint32_t pass = 0;
    __device__ __forceinline__ void advance() {
      if (++at == kStages) at = 0, pass ^= 1;
    }
  };
  // After a wait gave up: what was issued last at each stage is given the time of
  // one wait to be used up, so that nothing is in flight when the block ends.
  auto drain = [&](Ring r, uint32_t issued) {
    const unsigned long long t0 = now_ns();
    for (int i = 0; i < kStages && static_cast<uint32_t>(i) < issued; ++i) {
      if (r.at == 0) r.at = kStages, r.pass ^= 1;
      --r.at;
      while (!mbar_try(smem_addr(&s_empty[r.at]), r.pass) && now_ns() - t0 < kWaitNs) {
      }
    }
  };
  // The pair's tiles: one of every `pairs`, in turn from the front and the back.
  struct Walk {
    int t, up, down;
    __device__ __forceinline__ Walk(int pair, int pairs)
        : t(pair), up(2 * (pairs - pair) - 1), down(2 * pair + 1) {}
    __device__ __forceinline__ void next() {
      t += up;
      const int s = up;
      up = down;
      down = s;
    }
  };
  auto tile_at = [&](int t) {
    return find_tile<kUse>(a.E, segments, first, t, m_blocks, n_blocks, static_cast<int>(a.K), cap);
  };
  // Slices of the contraction (d_weight: of the expert's rows), from first_slice on
  // in pairs that share it.
  const int first_slice = all_slices * split / splits;
  auto slices = [&](const Tile& t) {
    return kUse == kWeightGrad ? (t.rows + kSlice - 1) / kSlice
                               : all_slices * (split + 1) / splits - first_slice;
  };
  // Columns of a tile's product (each block holds half of B).
  auto mma_n = [](int cols) { return (cols + 15) / 16 * 16; };
  // First feature of the block's A tile.
  auto feature = [&](const Tile& t) { return t.m0 + rank * (m_step<kUse>() / 2); };
  // Whether a d_weight tile has a slice that runs past the expert's rows.  It is
  // loaded first and multiplied a little later, as clearing it takes time.
  auto has_tail = [&](const Tile& t) { return kUse == kWeightGrad && t.rows % kSlice != 0; };
  // A slice that runs past the expert's rows: what follows belongs to another
  // expert or to none and may be infinite or NaN, so it is overwritten in both
  // operands rather than multiplied by zeros.
  auto clear_tail = [&](int st, int left) {
    const int chunks = ((left + 15) / 16 * 16 - left) * 8;  // of 16 bytes, in each box
    uint8_t* at = stages + st * kStageBytes + left * 128 + lane * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i * 32 + lane < chunks) {
#pragma unroll
        for (int box = 0; box < 4; ++box)  // 64 values x 64 rows: two of A, two of B
          *reinterpret_cast<uint4*>(at + i * 512 + box * (kTileABytes / 2)) = make_uint4(0, 0, 0, 0);
      }
    fence_async_shared();
    __syncwarp();
  };
  if (warp == kEpiWarps) {
    if (elect_one()) {  // one lane alone: a warp-wide wait per slice costs a quarter of the rate
      Ring ring;
      uint32_t issued = 0;
      bool ok = true;
      const uint32_t full0 = cluster_addr(smem_addr(&s_full[0]), leader);
      for (Walk walk(pair, pairs); walk.t < total && ok; walk.next()) {
        const Tile tile = tile_at(walk.t);
        const int n_slices = slices(tile), half_n = mma_n(tile.cols) / 2;
        const int b_boxes = (half_n + 63) / 64;
        const uint32_t bytes = kTileABytes + b_boxes * kBoxBytes;
        for (int s = 0; s < n_slices; ++s, ++issued) {
          const int st = ring.at;
          if (withheld(issued) || !mbar_wait(smem_addr(&s_empty[st]), ring.pass ^ 1, gave_up)) {
            ok = false;
            break;
          }
          *static_cast<volatile uint32_t*>(&s_issued) = issued + 1;
          ring.advance();
          // Both blocks' loads report to the first block's barrier; those of a
          // tail slice to their own block's, where it is cleared first (s_clear).
          uint32_t full = full0 + st * 8;
          if (s == 0 && has_tail(tile)) {
            if (rank == 0) mbar_arrive(smem_addr(&s_full[st]));
            full = smem_addr(&s_tail[st]);
            mbar_expect(full, bytes);
          } else if (rank == 0) {
            mbar_expect(smem_addr(&s_full[st]), 2 * bytes);
          }
          const uint32_t sa = smem_addr(stages + st * kStageBytes);
          const uint32_t sb = sa + kTileABytes;
          const int slice = kUse != kWeightGrad ? first_slice + s
                            : !has_tail(tile)   ? s
                            : s == 0            ? n_slices - 1
                                                : s - 1;
          const int k = slice * kSlice, m = feature(tile);
          if (kUse == kGated) {
            tma_load_5d(sa, &map_a, k, 0, 0, m / 8, tile.e, full);
          } else if (kUse == kForward) {
            tma_load_3d(sa, &map_a, k, m, tile.e, full);
          } else if (kUse == kRowsGrad) {
            tma_load_3d(sa, &map_a, m, k, tile.e, full);
            tma_load_3d(sa + kTileABytes / 2, &map_a, m + 64, k, tile.e, full);
          } else {
            tma_load_2d(sa, &map_a, m, tile.lo + k, full);
            tma_load_2d(sa + kTileABytes / 2, &map_a, m + 64, tile.lo + k, full);
          }
          for (int i = 0; i < b_boxes; ++i) {
            const int n = rank * half_n + i * 64;
            if (kBMn) tma_load_2d(sb + i * kBoxBytes, &map_b, tile.n0 + n, tile.lo + k, full);
            else tma_load_2d(sb + i * kBoxBytes, &map_b, k, tile.lo + n, full);
          }
        }
      }
      if (*gave_up != 0) drain(ring, issued);
    }
    __syncwarp();
  } else if (warp == kEpiWarps + 1) {
    if (rank == 0 && elect_one()) {
      Ring ring;
      uint32_t issued = 0, done = 0;
      uint32_t tails = 0;  // bit st: parity of the stage's tail slices so far
      const uint16_t both = static_cast<uint16_t>(3u << leader);
      bool ok = true;
      for (Walk walk(pair, pairs); walk.t < total && ok; walk.next()) {
        const Tile tile = tile_at(walk.t);
        const int n_slices = slices(tile);
        if (n_slices == 0) continue;
        const uint32_t idesc = instr_desc(kBf16, kAMn, kBMn, 256, mma_n(tile.cols));
        const uint32_t buf = done & 1, acc = tmem + buf * kMaxN;
        if (!mbar_wait(smem_addr(&s_free[buf]), (done / 2 & 1) ^ 1, gave_up)) break;
        ++done;
        tc_fence_after();
        // The products of the slice at `place`; false if it never came.
        bool accumulate = false;
        auto multiply = [&](const Ring& place, int depth, bool cleared) {
          const int st = place.at;
          if (!mbar_wait(smem_addr(&s_full[st]), place.pass, gave_up)) return false;
          if (cleared) {
            if (!mbar_wait(smem_addr(&s_clear[st]), tails >> st & 1, gave_up)) return false;
            tails ^= 1u << st;
          }
          tc_fence_after();
          const uint32_t pa = smem_addr(stages + st * kStageBytes);
          const uint32_t pb = pa + kTileABytes;
          constexpr uint32_t kStepA = kAMn ? 2048 : 32, kStepB = kBMn ? 2048 : 32;
          for (int i = 0; i < depth; ++i) {
            tc_mma(acc, smem_desc(pa + i * kStepA, kAMn ? 8192 : 16, 1024),
                   smem_desc(pb + i * kStepB, kBMn ? 8192 : 16, 1024), idesc, accumulate);
            accumulate = true;
          }
          tc_commit(smem_addr(&s_empty[st]), both);
          ++issued;
          return true;
        };
        const bool tail = has_tail(tile);
        const Ring tail_place = ring;
        const int tail_after = min(kTailDelay, n_slices - 1);  // slices before the tail's products
        if (tail) ring.advance();
        for (int s = tail ? 1 : 0; ok && s <= n_slices; ++s) {
          if (tail && s == tail_after + 1)
            ok = multiply(tail_place, (tile.rows % kSlice + 15) / 16, true);
          if (!ok || s == n_slices) break;
          ok = multiply(ring, kSlice / 16, false);
          ring.advance();
        }
        if (ok) tc_commit(smem_addr(&s_done[buf]), both);
      }
      // The products are over before the memory they read and write is given up.
      if (*gave_up != 0) drain(ring, issued);
    }
    __syncwarp();
  } else if (warp == kEpiWarps + 2) {
    if (kUse == kWeightGrad) {
      // Tail slices: each block clears its own and tells the first block.
      const uint32_t clear0 = cluster_addr(smem_addr(&s_clear[0]), leader);
      uint32_t step = 0;
      uint32_t tails = 0;  // bit st: parity of the stage's tail slices so far
      for (Walk walk(pair, pairs); walk.t < total; walk.next()) {
        const Tile tile = tile_at(walk.t);
        const int n_slices = slices(tile);
        if (has_tail(tile)) {
          const int st = static_cast<int>(step % kStages);
          const uint32_t parity = tails >> st & 1;
          tails ^= 1u << st;
          if (!warp_wait(smem_addr(&s_tail[st]), parity, gave_up, progress)) break;
          clear_tail(st, tile.rows % kSlice);
          if (lane == 0) mbar_arrive_cluster(clear0 + st * 8);
        }
        step += n_slices;
      }
      __syncwarp();
    }
  } else {
    const int quad = warp & 3;
    const uint32_t stage = smem_addr(staging + warp * kStagingWarpBytes);
    T* out = static_cast<T*>(a.out);
    T* preact = static_cast<T*>(a.preact);
    T* residual = kUse == kForward ? static_cast<T*>(const_cast<void*>(a.residual)) : nullptr;
    uint32_t done = 0;
    const uint32_t free0 = cluster_addr(smem_addr(&s_free[0]), leader);
    // Pairs that share a tile have one tile at most: its sums may lie over the
    // stages, which are through.  A lane's 32 values of the warp's columns c: 8
    // steps of 512 bytes from part + 64 c on.
    const uint32_t part = smem_addr(stages + warp * 4 * 4096) + lane * 16;
    const uint32_t other_part = splits > 1 ? cluster_addr(part, 2 + rank) : 0;
    for (Walk walk(pair, pairs); walk.t < total; walk.next()) {
      const Tile tile = tile_at(walk.t);
      const int cols = tile.cols;
      const bool any = slices(tile) > 0;
      // The warp's 32 features, its columns c + [0, 32).
      const int64_t m = feature(tile) + quad * (kUse == kGated ? 16 : 32);
      const int c0 = warp / 4 * 32;
      uint4 ahead[4];  // the next columns' residual
      auto residual_block = [&](int c) {
        return Block<T>(residual, a.N, tile.lo + c, cols - c, m, a.N, stage);
      };
      if (residual != nullptr && c0 < cols) load_block(ahead, residual_block(c0));
      const uint32_t buf = done & 1;
      if (any) {
        if (!warp_wait(smem_addr(&s_done[buf]), done / 2 & 1, gave_up, progress)) break;
        ++done;
        tc_fence_after();
      }
      const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * kMaxN;
      if (kUse != kWeightGrad && splits > 1) {
        if (split > 0) {
          for (int c = c0; c < cols; c += 64) {
            float z[32];
            tmem_load_32x32(acc + c, z);
            tmem_wait_load(z);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              shared_store16(part + (c - c0) * 64 + j * 512,
                             make_uint4(__float_as_uint(z[4 * j]), __float_as_uint(z[4 * j + 1]),
                                        __float_as_uint(z[4 * j + 2]), __float_as_uint(z[4 * j + 3])));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_addr(&s_parts), rank));
          break;
        }
        if (!warp_wait(smem_addr(&s_parts), 0, gave_up, cluster_addr(progress, 2 + rank))) break;
      }
      if (kUse == kWeightGrad) {
        for (int c = warp / 4 * 64; c < cols; c += 128) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // lanes 16 h + [0, 16)
            float z[32];
            if (any) {
              tmem_load_16x64(acc + (static_cast<uint32_t>(16 * h) << 16) + c, z);
              tmem_wait_load(z);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) z[j] = 0.f;
            }
            const int64_t left = a.N - m - 16 * h;
            write_row_block(z, Block<T, 64>(out, a.K, static_cast<int64_t>(tile.e) * a.N + m + 16 * h,
                                            static_cast<int>(left < 0 ? 0 : left < 16 ? left : 16),
                                            tile.n0 + c, tile.n0 + cols, stage));
          }
        }
      } else
      for (int c = c0; c < cols; c += 64) {
        const int64_t row = tile.lo + c;
        float z[32];
        tmem_load_32x32(acc + c, z);
        tmem_wait_load(z);
        if (splits > 1) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 x = cluster_load4(other_part + (c - c0) * 64 + j * 512);
            z[4 * j] += x.x, z[4 * j + 1] += x.y, z[4 * j + 2] += x.z, z[4 * j + 3] += x.w;
          }
        }
        if (kUse == kGated) {
          // The warp's 32 lanes: 8 gate rows and the up rows of the same features,
          // and again; a thread holds both of a value, z[16 h + 4 i + 2 s + b]
          // being gate (s = 0) or up of feature 8 h + g, row 8 i + 2 q + b.
          float gate[16], up[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {  // j = 4 i + 2 h + b
            gate[j] = z[j / 2 % 2 * 16 + j / 4 * 4 + j % 2];
            up[j] = z[j / 2 % 2 * 16 + j / 4 * 4 + 2 + j % 2];
          }
          if (preact != nullptr) {
            write_half_block(gate, Block<T, 16>(preact, a.N, row, cols - c, m, F, stage));
            write_half_block(up, Block<T, 16>(preact + F, a.N, row, cols - c, m, F, stage));
          }
          apply_act<16>(a.act, gate);
#pragma unroll
          for (int j = 0; j < 16; ++j) gate[j] *= up[j];
          write_half_block(gate, Block<T, 16>(out, F, row, cols - c, m, F, stage));
        } else if (kUse == kForward) {
          if (a.bias != nullptr) {
            const T* bias = static_cast<const T*>(a.bias) + static_cast<int64_t>(tile.e) * a.N;
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // z[16 h + 4 i + 2 s + b]: feature 16 h + 8 s + g
              const int64_t f = m + j * 8 + (lane >> 2);
              const float x = f < a.N ? to_f(bias[f]) : 0.f;
#pragma unroll
              for (int k = 0; k < 8; ++k) z[j / 2 * 16 + k / 2 * 4 + j % 2 * 2 + k % 2] += x;
            }
          }
          if (preact != nullptr)
            write_block(z, Block<T>(preact, a.N, row, cols - c, m, a.N, stage));
          apply_act<32>(a.act, z);
          if (residual != nullptr) {
            add_block(z, ahead, residual_block(c));
            if (c + 64 < cols) load_block(ahead, residual_block(c + 64));
          }
          write_block(z, Block<T>(out, a.N, row, cols - c, m, a.N, stage));
        } else {
          write_block(z, Block<T>(out, a.K, row, cols - c, m, a.K, stage));
        }
      }
      if (any) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed_cluster(free0 + buf * 8);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the products, loads, arrivals and reads of the cluster are over
  tc_fence_after();
  if (threadIdx.x == 0 && *gave_up != 0 && a.status != nullptr)
    atomicOr(a.status, MOE_FLAG_BARRIER_TIMEOUT);
  if (warp == kEpiWarps + 1) tmem_free(tmem, 512);
  // What follows waits for this launch alone, so it ends after the one before.
  if (a.beside_previous) pdl_wait();
}

}  // namespace experts
}  // namespace moe
