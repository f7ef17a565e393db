// cg_cache_write.cu -- cg_cache_write: new keys and values into 8-bit pages.
#include "cg_cache.cuh"

namespace cg {
namespace {

constexpr int kThreads = 128;
constexpr int kHeld = 8;  // vectors of 8 values that a thread keeps between its two passes

struct WriteArgs {
  const uint16_t *src[2];
  uint8_t *pool[2];
  float *scale[2];
  const int32_t *cu, *start, *table;
  int64_t st, sh;
  uint32_t *status;
  int H, d, bt, n_blocks, n_rows, max_new, stride, per_seq;
};

// Eight values; one that is not finite becomes 0 and sets `bad`.
template <bool BF16>
__device__ inline void finite8(uint4 w, float (&x)[8], bool &bad) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint16_t b = uint16_t(u[i >> 1] >> (16 * (i & 1)));
    constexpr uint16_t kExp = BF16 ? 0x7f80 : 0x7c00;
    const bool fin = (b & kExp) != kExp;
    bad |= !fin;
    x[i] = fin ? elem<BF16>(b) : 0.0f;
  }
}

template <int FMT>
__device__ inline uint2 codes8(const float (&x)[8], float r) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; i++) c[i] = code_of<FMT>(__fmul_rn(x[i], r));
  return make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
}

// One CTA per (page that gets rows, head, K or V): a pass for the largest
// magnitude, one that writes codes.  A page of up to 128 x 64 values stays in
// registers between the two; what is longer is read twice (the second time
// from L2).
template <int FMT, bool BF16>
__global__ void __launch_bounds__(kThreads) k_write(const WriteArgs a) {
  const int b = blockIdx.x / a.per_seq, p = blockIdx.x % a.per_seq;
  const int h = blockIdx.y >> 1, kv = blockIdx.y & 1;
  const int r0 = a.cu[b], r1 = a.cu[b + 1], pos = a.start[b];
  const int n = r1 - r0;
  if (r0 < 0 || r1 > a.n_rows || n < 0 || n > a.max_new || pos < 0 || int64_t(pos) + n > int64_t(a.stride) * a.bt) {
    if (p == 0 && threadIdx.x == 0) atomicOr(a.status, kStBadArg);
    return;
  }
  const int blk = pos / a.bt + p;
  const int64_t first = int64_t(blk) * a.bt;
  const int64_t t0 = max(int64_t(pos), first), t1 = min(int64_t(pos) + n, first + a.bt);
  if (t0 >= t1) return;
  const int page = a.table[int64_t(b) * a.stride + blk];
  if (uint32_t(page) >= uint32_t(a.n_blocks)) {
    if (threadIdx.x == 0) atomicOr(a.status, kStBadArg);
    return;
  }
  const int vpr = a.d >> 3, nv = int(t1 - t0) * vpr, s0 = int(t0 - first);
  const uint16_t *src = a.src[kv] + (r0 + t0 - pos) * a.st + h * a.sh;
  uint8_t *dst = a.pool[kv] + page_row(page, a.H, h, a.bt, 0, a.d);
  float *scale = a.scale[kv] + int64_t(page) * a.H + h;

  uint4 held[kHeld];
  float top = 0.0f;
  bool bad = false;
  auto load = [&](int i) { return *reinterpret_cast<const uint4 *>(src + int64_t(i / vpr) * a.st + (i % vpr) * 8); };
  auto max8 = [&](uint4 w) {
    float x[8];
    finite8<BF16>(w, x, bad);
#pragma unroll
    for (int i = 0; i < 8; i++) top = fmaxf(top, fabsf(x[i]));
  };
#pragma unroll
  for (int k = 0; k < kHeld; k++)
    if (int(threadIdx.x) + k * kThreads < nv) held[k] = load(threadIdx.x + k * kThreads);
#pragma unroll
  for (int k = 0; k < kHeld; k++)
    if (int(threadIdx.x) + k * kThreads < nv) max8(held[k]);
  for (int i = threadIdx.x + kHeld * kThreads; i < nv; i += kThreads) max8(load(i));

  __shared__ float s_top[kThreads / 32];
  const float before = s0 > 0 ? *scale : 0.0f;
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));  // not negative: ordered as integers
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
  if (__syncthreads_or(bad) && threadIdx.x == 0) atomicOr(a.status, kStNonfinite);
#pragma unroll
  for (int w = 0; w < kThreads / 32; w++) top = fmaxf(top, s_top[w]);
  float now = __fmul_rn(top, 1.0f / QMax<FMT>::v);
  if (now < 0x1p-100f) now = 0.0f;
  if (s0 > 0) now = fmaxf(now, before);
  if (s0 > 0 && now > before) {  // the rows that were there, in the larger step
    const float ratio = __fdiv_rn(before, now);
    for (int i = threadIdx.x; i < s0 * vpr; i += kThreads) {
      uint2 *at = reinterpret_cast<uint2 *>(dst + int64_t(i) * 8);
      const uint2 c = *at;
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; j++) x[j] = value_of<FMT>(((j < 4 ? c.x : c.y) >> (8 * (j & 3))) & 0xffu);
      *at = codes8<FMT>(x, ratio);
    }
  }
  if (threadIdx.x == 0) *scale = now;
  const float r = now > 0.0f ? __fdiv_rn(1.0f, now) : 0.0f;
  auto store = [&](int i, uint4 w) {
    float x[8];
    finite8<BF16>(w, x, bad);
    *reinterpret_cast<uint2 *>(dst + int64_t(s0) * a.d + int64_t(i) * 8) = codes8<FMT>(x, r);
  };
#pragma unroll
  for (int k = 0; k < kHeld; k++)
    if (int(threadIdx.x) + k * kThreads < nv) store(threadIdx.x + k * kThreads, held[k]);
  for (int i = threadIdx.x + kHeld * kThreads; i < nv; i += kThreads) store(i, load(i));
}

}  // namespace
}  // namespace cg

extern "C" cg_status cg_cache_write(const cg_cache *cache, const cg_rows *rows, const void *k_dev, const void *v_dev,
                                    const int32_t *cu_new_dev, const int32_t *start_dev, const int32_t *table_dev,
                                    void *k_pool, void *v_pool, float *k_scale, float *v_scale, void *ws_dev,
                                    size_t ws_bytes, void *stream) {
  using namespace cg;
  if (!cache8_ok(cache) || !rows || !k_dev || !v_dev || !cu_new_dev || !start_dev || !table_dev || !k_pool ||
      !v_pool || !k_scale || !v_scale || !ws_dev)
    return CG_ERR_INVALID_ARG;
  if (rows->n_seq < 1 || rows->n_rows < 0 || rows->max_new < 0 || rows->table_stride < 1 || rows->reserved != 0 ||
      (rows->dtype != CG_F16 && rows->dtype != CG_BF16) || rows->stride_token % 8 || rows->stride_head % 8)
    return CG_ERR_INVALID_ARG;
  if (!is_aligned(k_dev, 16) || !is_aligned(v_dev, 16) || !is_aligned(k_pool, 16) || !is_aligned(v_pool, 16) ||
      !is_aligned(k_scale, 4) || !is_aligned(v_scale, 4) || !is_aligned(cu_new_dev, 4) ||
      !is_aligned(start_dev, 4) || !is_aligned(table_dev, 4) || !is_aligned(ws_dev, 256) || ws_bytes < 256)
    return CG_ERR_INVALID_ARG;
  // a run of max_new tokens touches at most this many pages
  const int64_t per_seq = (int64_t(rows->max_new) + 2 * int64_t(cache->block_tokens) - 2) / cache->block_tokens;
  const int64_t gx = per_seq * rows->n_seq;
  if (gx > 0x7fffffff || 2 * int64_t(cache->H) > 65535) return CG_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(ws_dev, 0, 256, st) != cudaSuccess) return CG_ERR_CUDA;
  if (rows->max_new == 0 || gx == 0) return CG_OK;
  WriteArgs a{};
  a.src[0] = static_cast<const uint16_t *>(k_dev), a.src[1] = static_cast<const uint16_t *>(v_dev);
  a.pool[0] = static_cast<uint8_t *>(k_pool), a.pool[1] = static_cast<uint8_t *>(v_pool);
  a.scale[0] = k_scale, a.scale[1] = v_scale;
  a.cu = cu_new_dev, a.start = start_dev, a.table = table_dev;
  a.st = rows->stride_token, a.sh = rows->stride_head;
  a.status = static_cast<uint32_t *>(ws_dev);
  a.H = cache->H, a.d = cache->d, a.bt = cache->block_tokens, a.n_blocks = cache->n_blocks;
  a.n_rows = rows->n_rows, a.max_new = rows->max_new, a.stride = rows->table_stride, a.per_seq = int(per_seq);
  const dim3 grid(unsigned(gx), unsigned(2 * cache->H));
  const bool e4m3 = cache->format == CG_CACHE_E4M3, bf16 = rows->dtype == CG_BF16;
  if (e4m3 && bf16) k_write<CG_CACHE_E4M3, true><<<grid, kThreads, 0, st>>>(a);
  if (e4m3 && !bf16) k_write<CG_CACHE_E4M3, false><<<grid, kThreads, 0, st>>>(a);
  if (!e4m3 && bf16) k_write<CG_CACHE_INT8, true><<<grid, kThreads, 0, st>>>(a);
  if (!e4m3 && !bf16) k_write<CG_CACHE_INT8, false><<<grid, kThreads, 0, st>>>(a);
  return launched();
}
