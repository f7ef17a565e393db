// cg_tc.cuh -- tcgen05 products, tensor memory and two-wide arithmetic, shared
// by the attention kernels that run on them.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "cg_tma.cuh"

namespace cg {

// ---- tcgen05 ----------------------------------------------------------------
// Operands in shared memory: rows of 128 bytes, swizzled; eight rows make 1024
// bytes.  For a K-major operand the stride between groups of eight rows is
// 1024; for V, whose rows are keys, 1024 is the stride between groups of eight
// keys and `lead` the one between groups of 64 channels.
constexpr uint32_t kOperandHi = 1024 >> 4 | 1u << 14 | 2u << 29;
__device__ inline uint32_t operand_lo(const void *p, uint32_t lead) { return smem_of(p) >> 4 | lead >> 4 << 16; }

__device__ inline void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{.reg .pred p; .reg .b64 a, b; setp.ne.u32 p, %5, 0; mov.b64 a, {%1, %3}; mov.b64 b, {%2, %3};"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;}" ::"r"(d), "r"(a), "r"(b), "r"(kOperandHi), "r"(idesc), "r"(uint32_t(add))
      : "memory");
}

__device__ inline void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{.reg .pred p; .reg .b64 b; setp.ne.u32 p, %5, 0; mov.b64 b, {%2, %3}; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;}" ::"r"(d),
      "r"(a), "r"(b), "r"(kOperandHi), "r"(idesc), "r"(uint32_t(add))
      : "memory");
}

// True in one thread of a warp that runs together.  (tcgen05 wants its operands
// in uniform registers; a branch on this keeps them there, one on a lane's
// number costs about 60 cycles an instruction.)
__device__ inline bool elected() {
  uint32_t ok;
  asm volatile("{.reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p;}" : "=r"(ok));
  return ok;
}

// The barrier gets an arrival when all products issued so far are done.
__device__ inline void mma_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_of(bar)) : "memory");
}

__device__ inline void tm_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ inline void tm_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ inline void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ inline void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define CG_R8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define CG_I8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])

// 32 columns of this thread's lane.
__device__ inline void tm_load(uint32_t addr, uint32_t *x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : CG_R8(x, 0), CG_R8(x, 8), CG_R8(x, 16), CG_R8(x, 24)
      : "r"(addr));
}

__device__ inline void tm_store32(uint32_t addr, const uint32_t *x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      CG_I8(x, 0), CG_I8(x, 8), CG_I8(x, 16), CG_I8(x, 24)
      : "memory");
}

__device__ inline void tm_store16(uint32_t addr, const uint32_t *x) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
               CG_I8(x, 0), CG_I8(x, 8)
               : "memory");
}

// ---- arithmetic ---------------------------------------------------------------
__device__ inline float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ inline float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ inline float2 fma2(float2 a, float2 b, float2 c) {
  float2 y;
  asm("{.reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};"
      " fma.rn.f32x2 d, a, b, c; mov.b64 {%0, %1}, d;}"
      : "=f"(y.x), "=f"(y.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return y;
}
__device__ inline float2 add2(float2 a, float2 b) {
  float2 y;
  asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d;}"
      : "=f"(y.x), "=f"(y.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
__device__ inline float2 mul2(float2 a, float2 b) {
  float2 y;
  asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mul.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d;}"
      : "=f"(y.x), "=f"(y.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}

template <bool BF16>
__device__ inline uint32_t pack(float lo, float hi) {
  uint32_t r;
  if (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace cg
