// cg_tma.cuh -- tensor maps, mbarriers and tiled copies, shared by the
// attention kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace cg {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's cuTensorMapEncodeTiled, found once (the library does not link against the driver).
inline EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// A map of rows of d elements with two strides, in boxes of 64 x n1 x n2.
inline bool make_map(CUtensorMap *map, const void *base, int d, int64_t size1, int64_t stride1, int n1, int64_t size2, int64_t stride2, int n2) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  // an extent of one needs no stride, but the map wants a positive one
  if (size1 == 1) stride1 = d;
  if (size2 == 1) stride2 = d;
  const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(size1), cuuint64_t(size2)};
  const cuuint64_t strides[2] = {cuuint64_t(2 * stride1), cuuint64_t(2 * stride2)};
  const cuuint32_t box[3] = {64, cuuint32_t(n1), cuuint32_t(n2)}, ones[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

__device__ inline uint32_t smem_of(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }

__device__ inline void bar_init(uint64_t *bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_of(bar)), "r"(count) : "memory");
}

// Makes initialised barriers visible to the async proxy.
__device__ inline void bar_init_fence() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }

__device__ inline void bar_expect(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_of(bar)), "r"(bytes) : "memory");
}

__device__ inline void bar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_of(bar)) : "memory");
}

__device__ inline bool bar_try(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{.reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p;}"
      : "=r"(ok)
      : "r"(smem_of(bar)), "r"(parity)
      : "memory");
  return ok;
}

// A wait ends when it takes this many cycles (about two seconds, where a tile
// takes microseconds), or when another wait of the CTA has ended so; false
// means that the memory system failed.
constexpr long long kWaitCycles = 4000000000ll;

__device__ inline bool bar_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *dead) {
  if (bar_try(bar, parity)) return true;
  const long long t0 = clock64();
  while (!bar_try(bar, parity)) {
    if (*dead) return false;
    if (clock64() - t0 > kWaitCycles) {
      *dead = 1;
      return false;
    }
  }
  return true;
}

__device__ inline void tma_2d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
               "l"(map), "r"(smem_of(bar)), "r"(x), "r"(y)
               : "memory");
}

__device__ inline void tma_3d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
               "l"(map), "r"(smem_of(bar)), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// Orders this thread's accesses of shared memory before later ones of the async proxy.
__device__ inline void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

}  // namespace cg
