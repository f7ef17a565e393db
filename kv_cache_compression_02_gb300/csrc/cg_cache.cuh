// cg_cache.cuh -- what the cache, prompt and page calls (cachegen_cache.h)
// share: argument checks, workspace sizes and small device helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>

#include "cachegen_cache.h"
#include "cg_layout.cuh"

namespace cg {

constexpr int kSMs = 152;  // of a GB300

inline bool is_aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Clears a call's status word.  The kernel that follows is launched early: it
// may begin while this one ends, when what ran before this one is done, and
// waits for it (status_cleared) before it sets a bit.
static __global__ void k_clear(uint32_t *status) {
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) *status = 0;
}

__device__ inline void status_cleared() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launches a kernel that may begin while the one before it ends.
template <typename... Args>
inline cudaError_t launch_early(void (*kernel)(Args...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const Args &...args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid, cfg.blockDim = block, cfg.dynamicSmemBytes = smem, cfg.stream = st;
  cfg.attrs = &early, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

inline cg_status launched() { return cudaGetLastError() == cudaSuccess ? CG_OK : CG_ERR_CUDA; }

inline bool cache_ok(const cg_cache *c) {
  return c && c->L >= 1 && c->H >= 1 && c->H <= 65535 && c->d >= 8 && c->d <= 128 && c->d % 8 == 0 &&
         c->block_tokens >= 1 && c->n_blocks >= 1 && c->n_blocks <= (1 << 28) && c->format >= CG_CACHE_F16 && c->format <= CG_CACHE_INT8 &&
         c->L <= (1 << 20) && int64_t(c->H) * c->block_tokens <= (int64_t(1) << 30);
}

inline bool cache8_ok(const cg_cache *c) { return cache_ok(c) && c->format != CG_CACHE_F16; }

// Bytes of a page of one pool.
inline uint64_t page_bytes(const cg_cache *c) {
  return uint64_t(c->H) * c->block_tokens * c->d * (c->format == CG_CACHE_F16 ? 2 : 1);
}

// A page's row for (head, slot): elements from the start of the pool.
__host__ __device__ inline int64_t page_row(int64_t page, int H, int h, int bt, int slot, int d) {
  return ((page * H + h) * bt + slot) * d;
}

template <int FMT>
struct QMax;
template <>
struct QMax<CG_CACHE_E4M3> {
  static constexpr float v = 448.0f;
};
template <>
struct QMax<CG_CACHE_INT8> {
  static constexpr float v = 127.0f;
};

// Four codes, nearest and halves to even.  e4m3 saturates; for int8 the values
// must be within 127.5 (an addition of 1.5 2^23 rounds them to integers, whose
// low bytes are the codes).
template <int FMT>
__device__ inline uint32_t codes_of(float a, float b, float c, float d) {
  if (FMT == CG_CACHE_E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return uint32_t(lo) | uint32_t(hi) << 16;
  }
  constexpr float kRound = 12582912.0f;
  const uint32_t ab = __byte_perm(__float_as_uint(__fadd_rn(a, kRound)), __float_as_uint(__fadd_rn(b, kRound)), 0x0040);
  const uint32_t cd = __byte_perm(__float_as_uint(__fadd_rn(c, kRound)), __float_as_uint(__fadd_rn(d, kRound)), 0x0040);
  return __byte_perm(ab, cd, 0x5410);
}

// The value a code stands for, without its scale.
template <int FMT>
__device__ inline float value_of(uint32_t c) {
  if (FMT == CG_CACHE_E4M3) return __half2float(__half(__nv_cvt_fp8_to_halfraw(__nv_fp8_storage_t(c), __NV_E4M3)));
  return float(int8_t(c));
}

// One element of a q, k or v row.
template <bool BF16>
__device__ inline float elem(uint16_t x) {
  if (BF16) return __uint_as_float(uint32_t(x) << 16);
  return __half2float(__ushort_as_half(x));
}

template <bool BF16>
__device__ inline uint16_t elem_of(float x) {
  if (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  return __half_as_ushort(__float2half_rn(x));
}

}  // namespace cg
