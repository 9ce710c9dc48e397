// gemm_common.cuh -- what the product kernels share: bounded waits of a warp,
// the tensor maps of row-major tensors, launches in clusters.
#pragma once

#include <atomic>

#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace vg {
namespace {

// Test-only builds (VG_TEST_FORCE_WAIT_TIMEOUT): a barrier that nothing
// arrives on, in the kernels' own shared memory (a static variable would move
// their 1024-byte aligned base).
#ifdef VG_TEST_FORCE_WAIT_TIMEOUT
#define VG_GEMM_NEVER uint64_t never;
#define VG_GEMM_NEVER_INIT(sm) mbar_init(&(sm).never, 1)
#define VG_GEMM_FORCED_TIMEOUT(sm, first) ((first) && !mbar_wait_bounded(&(sm).never, 0))
#else
#define VG_GEMM_NEVER
#define VG_GEMM_NEVER_INIT(sm)
#define VG_GEMM_FORCED_TIMEOUT(sm, first) false
#endif

// Waits for a barrier phase; a wait that gives up is recorded for the CTA,
// which reports it when it ends.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, volatile uint32_t *failed) {
  if (mbar_wait_bounded<CLUSTER>(bar, parity)) return true;
  *failed = 1;
  return false;
}

// The same for a whole warp, with one answer for all of it.
__device__ __forceinline__ bool warp_wait_phase(uint64_t *bar, uint32_t parity, volatile uint32_t *failed) {
  return __all_sync(0xFFFFFFFFu, wait_phase(bar, parity, failed));
}

// The same where a look at the phase (mbar_look) was taken some time ago.
// CLUSTER: behind what any CTA of the cluster wrote before it arrived.
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait_phase(bool seen, uint64_t *bar, uint32_t parity,
                                                volatile uint32_t *failed) {
  const bool ok =
      __all_sync(0xFFFFFFFFu, seen) || __all_sync(0xFFFFFFFFu, wait_phase<CLUSTER>(bar, parity, failed));
  if constexpr (CLUSTER) acquire_cluster_written();
  return ok;
}

// A barrier of `threads` threads that tells all of them whether any passed true.
__device__ __forceinline__ bool named_sync_or(int id, int threads, bool p) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(threads), "r"((uint32_t)p)
      : "memory");
  return any != 0;
}

// ------------------------------------------------------------------- host

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once.
EncodeTiled encoder() {
  static std::atomic<EncodeTiled> fn{nullptr};
  EncodeTiled f = fn.load(std::memory_order_acquire);
  if (f) return f;
  void *p = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
          cudaSuccess ||
      found != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<EncodeTiled>(p);
  fn.store(f, std::memory_order_release);
  return f;
}

// A tensor of `rank` dimensions, innermost first, read or written in boxes;
// strides in bytes, from the second dimension on.
// The encoder is a driver call and wants a context: a host thread whose first
// CUDA call this is has none yet, and setting its device makes it one.
inline bool make_map(CUtensorMap *m, CUtensorMapDataType type, const void *p, int rank,
                     const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box,
                     CUtensorMapSwizzle swizzle) {
  const cuuint32_t step[4] = {1, 1, 1, 1};
  const EncodeTiled f = encoder();
  if (!f) return false;
  const auto encode = [&] {
    return f(m, type, (cuuint32_t)rank, const_cast<void *>(p), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  int dev = 0;
  return encode() || (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode());
}

// A row-major [rows, cols] tensor in boxes of box_rows x box_cols.
inline bool make_map(CUtensorMap *m, CUtensorMapDataType type, int size, const void *p, int64_t rows,
                     int64_t cols, int box_rows, int box_cols, CUtensorMapSwizzle swizzle) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(cols * size)};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  return make_map(m, type, p, 2, dims, strides, box, swizzle);
}

// launch_pdl with thread-block clusters of `cluster` CTAs along x.
template <class... P, class... A>
cudaError_t launch_pdl_cluster(void (*kern)(P...), dim3 g, int cluster, dim3 b, size_t smem,
                               cudaStream_t s, A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = g;
  cfg.blockDim = b;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<A &&>(args)...);
}

// Opts `kern` in to large dynamic shared memory, once per kernel and device.
cudaError_t opt_in_once(std::atomic<uint64_t> &opted_in, const void *kern) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (opted_in.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = opt_in_dynamic_smem(kern);
  if (e == cudaSuccess) opted_in.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace
}  // namespace vg
