// tcgen05.cuh -- the fifth-generation tensor cores and tensor-map TMA, as the
// FP8 products use them: E4M3 operands in shared memory (K-major rows of 128
// bytes in the 128-byte swizzle), fp32 accumulators in tensor memory.
#pragma once

#include <cstdint>

#include <cuda.h>

#include "tma.cuh"

namespace vg {

// ------------------------------------------------------ tensor-map copies

__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap *m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// One box of a 2-D tensor to this CTA's shared memory, counted on the barrier
// at cluster address `bar` (of either CTA of a pair); elements outside the
// tensor arrive as zeros (and are counted).  x times the element size must be
// a multiple of 16 bytes.
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *m, int32_t x, int32_t y,
                                                 uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(m), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// One lane of a converged warp, the same one each time.  The warps that issue
// copies and products run their loops as whole warps and elect the issuing
// lane at the instruction: with the loop itself on one lane the compiler must
// treat every operand as divergent (measured: 614 cycles of the issuing
// thread per scale block).
__device__ __forceinline__ bool elect_lane() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)::"memory");
  return r != 0;
}

// The same for a CTA that issues its products alone.
__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *m, int32_t x, int32_t y,
                                            uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(m), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// The same with an L2 policy (l2_evict_first()): data that is read once.
__device__ __forceinline__ uint64_t l2_evict_first() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_2d_hint(void *dst, const CUtensorMap *m, int32_t x, int32_t y,
                                                 uint64_t *bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
      "l"(m), "r"(x), "r"(y), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// Asks for one box to be brought into L2.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *m, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(m), "r"(x), "r"(y)
               : "memory");
}

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The cluster address of `p` in the shared memory of CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}

// Arrives on the barrier at a cluster address.  Relaxed: it hands over tensor
// memory that has been read (ordered by the tcgen05 fences), not memory that
// has been written; a release at cluster scope would cost about a thousand
// cycles here.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Four fp32 values at a cluster address.
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// All threads of the cluster's CTAs.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// One box from shared memory to a 2-D tensor; what lies outside the tensor is
// not written.  x and y must not be negative.  Then tma_store_commit().
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *m, const void *src, int32_t x,
                                             int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(m),
               "r"(x), "r"(y), "r"(smem_u32(src))
               : "memory");
}

// Closes this thread's group of stores (perhaps an empty one).
__device__ __forceinline__ void tma_store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Until at most N of this thread's groups still read shared memory.
template <int N>
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------ small async copies

// Four bytes from global to shared memory, or four zero bytes (nothing is
// read) where `live` is false.
__device__ __forceinline__ void copy_async4(void *dst, const void *src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(live ? 4u : 0u)
               : "memory");
}
// Arrives on `bar` once this thread's earlier small copies have landed.
__device__ __forceinline__ void copy_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copy_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ------------------------------------------------------------ tensor memory

// A whole warp allocates (a power of two >= 32 columns); the base address
// lands in shared memory.  The permit is given up: one allocation per CTA.
// PAIR: both CTAs of a pair call it, and the release, together; a kernel uses
// the pair's forms of all of these or of none.
#define VG_GROUP_FORM(PAIR, text_alone, text_pair, ...) \
  do {                                                  \
    if constexpr (PAIR) {                               \
      asm volatile(text_pair __VA_ARGS__);              \
    } else {                                            \
      asm volatile(text_alone __VA_ARGS__);             \
    }                                                   \
  } while (0)

template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t columns) {
  VG_GROUP_FORM(PAIR, "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;",
                "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;", ::"r"(smem_u32(slot)),
                "r"(columns)
                : "memory");
  VG_GROUP_FORM(PAIR, "tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;",
                "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;", ::
                    : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void tmem_dealloc(uint32_t base, uint32_t columns) {
  VG_GROUP_FORM(PAIR, "tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;",
                "tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;", ::"r"(base), "r"(columns)
                : "memory");
}

__device__ __forceinline__ void tcgen05_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tcgen05_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 32 lanes x 16 columns of fp32 accumulators, a lane a row, asynchronously;
// and the wait for them (below).
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_load_wait(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]),
                 "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]),
                 "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}

// 32 lanes x 32 columns of fp32 accumulators, a lane a row, asynchronously.
// A warp reads the 32 lanes that its index modulo four names.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
        "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr));
}

// Waits for this thread's tensor memory loads.  The registers are operands,
// so that nothing reads them earlier.
__device__ __forceinline__ void tmem_load_wait(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]),
                 "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]),
                 "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]),
                 "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                 "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]),
                 "+r"(v[31])
               :
               : "memory");
}

// ---------------------------------------------------------------- products

// Shared memory operand: rows of 128 bytes (128 E4M3 codes along K), the
// 128-byte swizzle, eight rows every 1024 bytes; base 1024-byte aligned.
// Stepping 32 bytes along the row (one product's K) adds 2.
__device__ __forceinline__ uint64_t operand_desc(uint32_t smem_addr) {
  constexpr uint64_t kLead = 1ull << 16;                 // unused under a swizzle
  constexpr uint64_t kStride = (uint64_t)(1024 >> 4) << 32;  // between groups of eight rows
  constexpr uint64_t kVersion = 1ull << 46;
  constexpr uint64_t kSwizzle128 = 2ull << 61;
  return ((uint64_t)(smem_addr >> 4) & 0x3FFFull) | kLead | kStride | kVersion | kSwizzle128;
}

// E4M3 x E4M3 -> fp32, both operands K-major, M x N.
__host__ __device__ constexpr uint32_t product_desc(uint32_t m, uint32_t n) {
  return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// D (tensor memory) = A B^T (+ D if accumulate) over K = 32, issued by one
// thread.  PAIR: of the pair's first CTA; rows 0..127 of A and D and the first
// half of B's rows are the first CTA's, the others the second's, at the same
// addresses of either.
template <bool PAIR>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t desc,
                                         bool accumulate) {
  VG_GROUP_FORM(PAIR,
                "{\n\t.reg .pred p;\n\t"
                "setp.ne.b32 p, %4, 0;\n\t"
                "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}",
                "{\n\t.reg .pred p;\n\t"
                "setp.ne.b32 p, %4, 0;\n\t"
                "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}", ::"r"(d),
                "l"(a), "l"(b), "r"(desc), "r"((uint32_t)accumulate)
                : "memory");
}

// Arrives on `bar` of both CTAs of the pair whose first cluster rank is `base`
// (or of this one alone) once this thread's earlier products have finished.
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar, uint32_t base) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)(3u << base))
      : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  VG_GROUP_FORM(PAIR, "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];",
                "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];", ::"r"(
                    smem_u32(bar))
                : "memory");
}

// ------------------------------------------------------------ register split

template <int N>
__device__ __forceinline__ void regs_decrease() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_increase() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace vg
