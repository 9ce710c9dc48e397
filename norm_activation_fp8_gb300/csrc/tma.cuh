// tma.cuh -- bulk (non-tensor) TMA copies global -> shared, completed on an
// mbarrier, plus the bounded waits the pipelined kernels use.
//
// cp.async.bulk needs 16-byte aligned source and destination and a size that
// is a multiple of 16 bytes; every row copied here is n bf16 with n % 8 == 0
// starting at a 16-byte aligned row of a 16-byte aligned tensor.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace vg {

// A wait gives up after this many failed try_wait polls (each poll may
// suspend the thread for a while): seconds, far beyond any healthy copy.
// (A test build lowers it.)
#ifndef VG_WAIT_LIMIT
#define VG_WAIT_LIMIT (1u << 22)
#endif
constexpr uint32_t kWaitLimit = VG_WAIT_LIMIT;

// Error bits a kernel leaves in its translation unit's status word.
constexpr uint32_t kErrWaitTimeout = 1u;

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

// Makes the initialised barriers visible to the async proxy (the TMA unit).
__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// Orders this thread's earlier generic-proxy shared memory accesses before
// later async-proxy (TMA) accesses to the same buffer.
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
               : "memory");
}

// Plain arrival (no transaction bytes), e.g. a consumer releasing a stage.
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// CLUSTER: the phase's arrivals come from the cluster's other CTAs too; behind
// it acquire_cluster_written() before what they wrote is used.
template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_try_wait(uint64_t *bar, uint32_t parity) {
  uint32_t done;
  if constexpr (CLUSTER)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  return done != 0;
}

// Orders what follows behind the writes to shared memory that the cluster's CTAs
// released (mbar_arrive_cluster_written()) before the arrivals that were seen.
__device__ __forceinline__ void acquire_cluster_written() {
  asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}

// Whether the phase with the given parity is over, without waiting: asked now,
// the answer taken later.  The answer rests in a predicate register N (0 or 1)
// that VG_LOOKS declares for the whole kernel: as a value of the same statement
// it would hold up what is issued in between, some 120 cycles.  Look 0 is for
// arrivals of this CTA, look 1 as mbar_try_wait<true>().
// The compiler does not know of the registers.  What keeps that sound: all three
// are volatile statements, which stay in the order they are written in; a kernel
// has VG_LOOKS once (a second copy would not assemble) and ahead of every look;
// and every path to a mbar_seen<N>() passes a mbar_look<N>().
#define VG_LOOKS asm volatile(".reg .pred vg_look0, vg_look1;")
template <int N>
__device__ __forceinline__ void mbar_look(uint64_t *bar, uint32_t parity) {
  if constexpr (N == 0)
    asm volatile("mbarrier.test_wait.parity.shared::cta.b64 vg_look0, [%0], %1;" ::"r"(smem_u32(bar)), "r"(parity)
                 : "memory");
  else
    asm volatile("mbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 vg_look1, [%0], %1;" ::"r"(
                     smem_u32(bar)),
                 "r"(parity)
                 : "memory");
}
template <int N>
__device__ __forceinline__ bool mbar_seen() {
  uint32_t done;
  if constexpr (N == 0)
    asm volatile("selp.u32 %0, 1, 0, vg_look0;" : "=r"(done)::"memory");
  else
    asm volatile("selp.u32 %0, 1, 0, vg_look1;" : "=r"(done)::"memory");
  return done != 0;
}

// Waits for the barrier's phase with the given parity; false after
// kWaitLimit polls.
template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_wait_bounded(uint64_t *bar, uint32_t parity) {
  for (uint32_t i = 0; i < kWaitLimit; ++i)
    if (mbar_try_wait<CLUSTER>(bar, parity)) return true;
  return false;
}

// Bulk copy of `bytes` from global to shared memory, counted on `bar`.
__device__ __forceinline__ void tma_load_bulk(void *dst_smem, const void *src, uint32_t bytes,
                                              uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst_smem)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Test-only builds (VG_TEST_FORCE_WAIT_TIMEOUT): a barrier that nothing
// arrives on.  A pipelined kernel waits on it after its first stage wait, so
// that wait runs out and the CTA takes its failure path while its other
// copies are in flight.  Product builds compile all of this away.
#ifdef VG_TEST_FORCE_WAIT_TIMEOUT
#define VG_NEVER_BARRIER __shared__ uint64_t vg_never_bar
#define VG_NEVER_BARRIER_INIT() mbar_init(&vg_never_bar, 1)
#define VG_FORCED_TIMEOUT(first) ((first) && !mbar_wait_bounded(&vg_never_bar, 0))
#else
#define VG_NEVER_BARRIER
#define VG_NEVER_BARRIER_INIT()
#define VG_FORCED_TIMEOUT(first) false
#endif

__device__ __forceinline__ uint4 lds128(const void *p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(smem_u32(p)));
  return v;
}

}  // namespace vg
