// tcgen05.cuh -- the PTX the grouped products are written in: mbarriers, clusters,
// TMA tile loads, tensor memory and tcgen05.mma.  Formats are those of the PTX ISA.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {
namespace experts {

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// One lane of a converged warp, the same one each time.  The asynchronous
// instructions take warp-uniform operands: behind this predicate the compiler
// knows that one thread runs them, behind `lane == 0` it does not and wraps
// each in a loop over the lanes (the grouped products ran 1.4x slower so).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// ---- mbarriers -------------------------------------------------------------

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
// The address of a peer block's copy of a shared variable of this block.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// `bar` as cluster_addr gave it.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
// Says only that this warp is through with reading, its values being in
// registers: unlike a release it does not wait until the global stores before it
// are performed, 1500 cycles.
__device__ __forceinline__ void mbar_arrive_relaxed_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ float cluster_load(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// Whether the phase is over, after sleeping for it up to kNapNs: an epilogue waits
// for tens of microseconds, and warps that poll all that time take power from the
// products (a long Mixtral-shaped gated product ran 1% slower).
constexpr uint32_t kNapNs = 20000;
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kNapNs)
      : "memory");
  return ok != 0;
}

// A wait gives up when kWaitNs pass without progress, or as soon as another wait of
// the block has: `gave_up` is the block's flag in shared memory.  A wait for one copy
// or one slice's products has no other progress than its own end.  A wait that spans
// a whole contraction (d_weight of one expert: as many slices as its rows fill, and
// rows may be counted up to 2^31) names the count of what a producer has issued,
// which moves with every slice: only where that stands still too has something gone
// wrong.  The count is in shared memory of this block or of another of the cluster.
constexpr unsigned long long kWaitNs = 2000000000ull;
constexpr uint32_t kNoProgress = 0xffffffffu;

#ifdef MOE_DEBUG_HOOKS
// The debug build's own limit, and the slices after which a producer stops (0: none);
// what lets copies in flight land keeps kWaitNs.
__device__ unsigned long long g_debug_wait_ns = kWaitNs;
__device__ int g_debug_slices = 0;
__device__ __forceinline__ unsigned long long wait_ns() { return g_debug_wait_ns; }
__device__ __forceinline__ bool withheld(uint32_t issued) {
  return g_debug_slices > 0 && issued >= static_cast<uint32_t>(g_debug_slices);
}
#else
__device__ __forceinline__ unsigned long long wait_ns() { return kWaitNs; }
__device__ __forceinline__ bool withheld(uint32_t) { return false; }
#endif

__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ uint32_t progress_at(uint32_t addr) {
  uint32_t v = 0;
  if (addr != kNoProgress)
    asm volatile("ld.volatile.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

static __device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity,
                                                   volatile int* gave_up, uint32_t progress) {
  unsigned long long t0 = now_ns();
  uint32_t seen = progress_at(progress);
  for (unsigned i = 0; i < (1u << 26); ++i) {
    if (mbar_try(bar, parity)) return true;
    if (*gave_up != 0) return false;
    if ((i & 63u) == 63u && now_ns() - t0 > wait_ns()) {
      const uint32_t at = progress_at(progress);
      if (at == seen) break;
      seen = at;
      t0 = now_ns();
      i = 0;
    }
  }
  *gave_up = 1;
  return false;
}

__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* gave_up,
                                          uint32_t progress = kNoProgress) {
#pragma unroll 1
  for (int i = 0; i < 8; ++i)
    if (mbar_try(bar, parity)) return true;
  return mbar_wait_slow(bar, parity, gave_up, progress);
}

// One lane waits, the whole warp learns the outcome and is ordered behind it.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* gave_up,
                                          uint32_t progress = kNoProgress) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, gave_up, progress);
  return __all_sync(0xffffffffu, ok);
}

// ---- TMA -------------------------------------------------------------------
// The loads of a pair of blocks: dst is this block's, bar either block's.

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, int w, int v, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(bar)
      : "memory");
}

// A load of one block of its own: no pair.
__device__ __forceinline__ void tma_load_4d_single(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// A plain copy of `bytes` (a multiple of 16, both sides 16-byte aligned) to
// this block's shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Orders this thread's ordinary writes to shared memory before what the
// asynchronous engines (tcgen05.mma) read afterwards.
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---- tensor memory and tcgen05 ---------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D (tensor memory) [+]= A (shared) B (shared), 16-bit operands, fp32 sums,
// over a pair of blocks: each holds half of A's rows, half of B's columns and
// the D rows of its A rows, at the same addresses in both.  Issued by the
// pair's first block.
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1 : 0)
      : "memory");
}
// The barrier at this address in the cluster's blocks of `mask` (the pair) gets one
// arrival when every tcgen05.mma issued before is done.
__device__ __forceinline__ void tc_commit(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}

// 32 columns of 16 of the warp's 32 lanes, as the fragments of mma.sync: lane
// (g, q) gets v[kAt + 4 i + 2 s + b] = D[lane 8 s + g][column 8 i + 2 q + b].
template <int kAt>
__device__ __forceinline__ void tmem_load_16x32(uint32_t addr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, "
      "%8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[kAt + 0]), "=f"(v[kAt + 1]), "=f"(v[kAt + 2]), "=f"(v[kAt + 3]),
        "=f"(v[kAt + 4]), "=f"(v[kAt + 5]), "=f"(v[kAt + 6]), "=f"(v[kAt + 7]),
        "=f"(v[kAt + 8]), "=f"(v[kAt + 9]), "=f"(v[kAt + 10]), "=f"(v[kAt + 11]),
        "=f"(v[kAt + 12]), "=f"(v[kAt + 13]), "=f"(v[kAt + 14]), "=f"(v[kAt + 15])
      : "r"(addr));
}
// 32 columns of the warp's 32 lanes: v[16 h + 4 i + 2 s + b] =
// D[lane 16 h + 8 s + g][column 8 i + 2 q + b].
__device__ __forceinline__ void tmem_load_32x32(uint32_t addr, float (&v)[32]) {
  tmem_load_16x32<0>(addr, v);
  tmem_load_16x32<16>(addr + (16u << 16), v);
}
// 64 columns of 16 of the warp's 32 lanes: v[4 i + 2 s + b] = D[lane 8 s + g][column
// 8 i + 2 q + b].
__device__ __forceinline__ void tmem_load_16x64(uint32_t addr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, "
      "%8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, "
      "%24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]),
        "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]),
        "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
        "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(addr));
}
// The loaded values pass through the wait, so that no use of them can be moved
// in front of it.
__device__ __forceinline__ void tmem_wait_load(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]),
                 "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31])::"memory");
}

// Four 8 x 8 matrices of 16-bit values, in fragments, to or from the rows whose
// addresses the lanes give (lane l: row l % 8 of matrix l / 8); transposed,
// what a fragment holds as row and column is column and row in memory.
template <bool kTranspose>
__device__ __forceinline__ void store_matrices(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                               uint32_t d) {
  if (kTranspose)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                     addr),
                 "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
  else
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                 "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void load_matrices_transposed(uint32_t addr, uint32_t& a, uint32_t& b,
                                                         uint32_t& c, uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}

// Shared memory descriptor of a 128-byte-swizzled operand tile.
//   K-major:  8 rows of 64 k-values make a 1024-byte block; sbo = the step to
//             the next 8 rows, lbo unused.
//   MN-major: 8 k-rows of 64 m- or n-values make a 1024-byte block; sbo = the
//             step to the next 8 k, lbo = the step to the next 64 m or n.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) |
         (static_cast<uint64_t>(lbo >> 4) << 16) | (static_cast<uint64_t>(sbo >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

// Instruction descriptor of kind::f16 with fp32 accumulators.
__device__ __forceinline__ uint32_t instr_desc(bool bf16, bool a_mn, bool b_mn, int m, int n) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) |
         (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

}  // namespace experts
}  // namespace moe
