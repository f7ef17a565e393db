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

// The nearest code, halves to even, saturating.
template <int FMT>
__device__ inline uint32_t code_of(float x) {
  if (FMT == CG_CACHE_E4M3) return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
  return uint32_t(__float2int_rn(fminf(fmaxf(x, -127.0f), 127.0f))) & 0xffu;
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
