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

// The exponent of Inf and NaN, in both halves of a word.
template <bool BF16>
constexpr uint32_t kExp = BF16 ? 0x7f807f80u : 0x7c007c00u;

// The larger magnitudes of two pairs: as integers, without the signs, 16-bit
// floats are in the order of their magnitudes, Inf and NaN above all.
__device__ inline uint32_t max_pair(uint32_t top, uint4 w) {
  top = __vmaxu2(top, __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu));
  return __vmaxu2(top, __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
}

// Values that are not finite become 0.
template <bool BF16>
__device__ inline uint4 finite(uint4 w) {
  auto one = [](uint32_t x) {
    const uint32_t bad = __vcmpeq2(x & kExp<BF16>, kExp<BF16>);
    return x & ~bad;
  };
  return make_uint4(one(w.x), one(w.y), one(w.z), one(w.w));
}

template <bool BF16>
__device__ inline float2 pair(uint32_t w) {
  if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

template <int FMT, bool BF16>
__device__ inline uint2 codes8(uint4 w, float r) {
  const float2 a = pair<BF16>(w.x), b = pair<BF16>(w.y), c = pair<BF16>(w.z), d = pair<BF16>(w.w);
  return make_uint2(codes_of<FMT>(__fmul_rn(a.x, r), __fmul_rn(a.y, r), __fmul_rn(b.x, r), __fmul_rn(b.y, r)),
                    codes_of<FMT>(__fmul_rn(c.x, r), __fmul_rn(c.y, r), __fmul_rn(d.x, r), __fmul_rn(d.y, r)));
}

// One CTA per (page that gets rows, head, K or V): a pass for the largest
// magnitude, one that writes codes.  A page of up to 128 x 64 values stays in
// registers between the two; what is longer is read twice (the second time
// from L2).  Bound by HBM: what is in flight counts, so that eight CTAs share
// an SM with 64 registers a thread (32768 tokens of 8 heads, fp16 to int8: 36 us
// or 5.5 TB/s; 49 us with the 112 registers that the compiler would take).
template <int FMT, bool BF16>
__global__ void __launch_bounds__(kThreads, 8) k_write(const WriteArgs a) {
  const int b = blockIdx.x / a.per_seq, p = blockIdx.x % a.per_seq;
  const int h = blockIdx.y >> 1, kv = blockIdx.y & 1;
  const int r0 = a.cu[b], r1 = a.cu[b + 1], pos = a.start[b];
  const int64_t n = int64_t(r1) - r0;
  status_cleared();
  auto report = [&](uint32_t bit) { atomicOr(a.status, bit); };
  if (r0 < 0 || r1 > a.n_rows || n < 0 || n > a.max_new || pos < 0 || int64_t(pos) + n > int64_t(a.stride) * a.bt) {
    if (p == 0 && threadIdx.x == 0) report(kStBadArg);
    return;
  }
  const int blk = pos / a.bt + p;
  const int64_t first = int64_t(blk) * a.bt;
  const int64_t t0 = max(int64_t(pos), first), t1 = min(int64_t(pos) + n, first + a.bt);
  if (t0 >= t1) return;
  const int page = a.table[int64_t(b) * a.stride + blk];
  if (uint32_t(page) >= uint32_t(a.n_blocks)) {
    if (threadIdx.x == 0) report(kStBadArg);
    return;
  }
  const int vpr = a.d >> 3, nv = int(t1 - t0) * vpr, s0 = int(t0 - first);
  const uint16_t *src = (kv ? a.src[1] : a.src[0]) + (r0 + t0 - pos) * a.st + h * a.sh;
  uint8_t *dst = (kv ? a.pool[1] : a.pool[0]) + page_row(page, a.H, h, a.bt, 0, a.d);
  float *scale = (kv ? a.scale[1] : a.scale[0]) + int64_t(page) * a.H + h;

  uint4 held[kHeld];
  uint32_t top2 = 0;
  auto load = [&](int i) { return *reinterpret_cast<const uint4 *>(src + int64_t(i / vpr) * a.st + (i % vpr) * 8); };
#pragma unroll
  for (int k = 0; k < kHeld; k++)
    held[k] = int(threadIdx.x) + k * kThreads < nv ? load(threadIdx.x + k * kThreads) : make_uint4(0, 0, 0, 0);
  const float before = s0 > 0 ? *scale : 0.0f;
#pragma unroll
  for (int k = 0; k < kHeld; k++)
    top2 = max_pair(top2, held[k]);
  for (int i = threadIdx.x + kHeld * kThreads; i < nv; i += kThreads) top2 = max_pair(top2, load(i));

  __shared__ uint32_t s_top[kThreads / 32];
  auto join = [&](uint32_t pair) {  // over the CTA
    const uint32_t t = __reduce_max_sync(0xffffffffu, max(pair & 0xffffu, pair >> 16));
    if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = t;
    __syncthreads();
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w++) m = max(m, s_top[w]);
    return m;
  };
  uint32_t top = join(top2);
  const bool bad = top >= (kExp<BF16> & 0xffffu);
  if (bad) {  // rare: once more, without them
    if (threadIdx.x == 0) report(kStNonfinite);
    top2 = 0;
#pragma unroll
    for (int k = 0; k < kHeld; k++)
      held[k] = finite<BF16>(held[k]), top2 = max_pair(top2, held[k]);
    for (int i = threadIdx.x + kHeld * kThreads; i < nv; i += kThreads) top2 = max_pair(top2, finite<BF16>(load(i)));
    __syncthreads();
    top = join(top2);
  }
  float now = __fmul_rn(pair<BF16>(top).x, 1.0f / QMax<FMT>::v);
  if (now < 0x1p-100f) now = 0.0f;
  if (s0 > 0) now = fmaxf(now, before);
  if (s0 > 0 && now > before) {  // the rows that were there, in the larger step
    const float ratio = __fdiv_rn(before, now);
    for (int i = threadIdx.x; i < s0 * vpr * 2; i += kThreads) {
      uint32_t *at = reinterpret_cast<uint32_t *>(dst + int64_t(i) * 4);
      const uint32_t c = *at;
      *at = codes_of<FMT>(__fmul_rn(value_of<FMT>(c & 0xff), ratio), __fmul_rn(value_of<FMT>(c >> 8 & 0xff), ratio),
                          __fmul_rn(value_of<FMT>(c >> 16 & 0xff), ratio), __fmul_rn(value_of<FMT>(c >> 24), ratio));
    }
  }
  if (threadIdx.x == 0) *scale = now;
  const float r = now > 0.0f ? __fdiv_rn(1.0f, now) : 0.0f;
  uint2 *to = reinterpret_cast<uint2 *>(dst + int64_t(s0) * a.d);
#pragma unroll
  for (int k = 0; k < kHeld; k++)
    if (int(threadIdx.x) + k * kThreads < nv) to[threadIdx.x + k * kThreads] = codes8<FMT, BF16>(held[k], r);
  for (int i = threadIdx.x + kHeld * kThreads; i < nv; i += kThreads) {
    const uint4 w = load(i);
    to[i] = codes8<FMT, BF16>(bad ? finite<BF16>(w) : w, r);
  }
}

}  // namespace
}  // namespace cg

extern "C" cg_status cg_cache_write(const cg_cache *cache, const cg_rows *rows, const void *k_dev, const void *v_dev,
                                    const int32_t *cu_new_dev, const int32_t *start_dev, const int32_t *table_dev,
                                    void *k_pool, void *v_pool, float *k_scale, float *v_scale, void *ws_dev,
                                    size_t ws_bytes, void *stream) {
  using namespace cg;
  // k and v may be NULL where there are no rows
  if (!cache8_ok(cache) || !rows || ((!k_dev || !v_dev) && rows->n_rows > 0) || !cu_new_dev || !start_dev || !table_dev || !k_pool ||
      !v_pool || !k_scale || !v_scale || !ws_dev)
    return CG_ERR_INVALID_ARG;
  if (rows->n_seq < 1 || rows->n_rows < 0 || rows->max_new < 0 || rows->table_stride < 1 || rows->reserved != 0 ||
      (rows->dtype != CG_F16 && rows->dtype != CG_BF16) || rows->stride_token % 8 || rows->stride_head % 8)
    return CG_ERR_INVALID_ARG;
  if (!is_aligned(k_dev, 16) || !is_aligned(v_dev, 16) || !is_aligned(k_pool, 16) || !is_aligned(v_pool, 16) ||
      !is_aligned(k_scale, 4) || !is_aligned(v_scale, 4) || !is_aligned(cu_new_dev, 4) ||
      !is_aligned(start_dev, 4) || !is_aligned(table_dev, 4) || !is_aligned(ws_dev, 256) || ws_bytes < 256)
    return CG_ERR_INVALID_ARG;
  // the kernel counts a page's vectors of 4 and 8 values of a head in 32 bits
  if (int64_t(cache->block_tokens) * cache->d > int64_t(1) << 32) return CG_ERR_INVALID_ARG;
  // a run of max_new tokens touches at most this many pages; a CTA at least looks at a sequence's offsets
  const int64_t touched = (int64_t(rows->max_new) + 2 * int64_t(cache->block_tokens) - 2) / cache->block_tokens, per_seq = touched ? touched : 1;
  const int64_t gx = per_seq * rows->n_seq;
  if (gx > 0x7fffffff || 2 * int64_t(cache->H) > 65535) return CG_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  k_clear<<<1, 32, 0, st>>>(static_cast<uint32_t *>(ws_dev));
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
  auto *const kernel = e4m3 ? (bf16 ? k_write<CG_CACHE_E4M3, true> : k_write<CG_CACHE_E4M3, false>)
                            : (bf16 ? k_write<CG_CACHE_INT8, true> : k_write<CG_CACHE_INT8, false>);
  const cudaError_t e = launch_early(kernel, grid, dim3(kThreads), 0, st, a);
  return e == cudaSuccess ? launched() : CG_ERR_CUDA;
}
