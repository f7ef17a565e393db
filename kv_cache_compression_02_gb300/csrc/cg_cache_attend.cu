// cg_cache_attend.cu -- cg_cache_attend: new tokens attend over 8-bit pages.
#include "cg_cache.cuh"

namespace cg {
namespace {

constexpr int kThreads = 128;

struct AttendArgs {
  const uint16_t *q;
  const uint8_t *kp, *vp;
  const float *ks, *vs;
  const int32_t *table, *len;
  uint16_t *out;
  float *lse;
  uint32_t *status;
  int64_t q_seq, q_tok, q_head;
  int B, T, Hq, H, d, bt, n_blocks, stride;
  float scale_log2;  // scale * log2(e)
};

// One CTA per output row; each warp takes every fourth position and keeps its
// own running maximum, sum and output.
template <int FMT, bool BF16>
__global__ void __launch_bounds__(kThreads) k_attend(const AttendArgs a) {
  const int b = blockIdx.x / a.T, t = blockIdx.x % a.T, hq = blockIdx.y, h = hq / (a.Hq / a.H);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t len = a.len[b];
  const int64_t most = int64_t(a.stride) * a.bt;
  if (len < 0 || len > most) {
    if (threadIdx.x == 0) atomicOr(a.status, kStBadArg);
    len = len < 0 ? 0 : most;
  }
  const int64_t seen = len - a.T + t + 1;
  const uint16_t *q = a.q + b * a.q_seq + t * a.q_tok + hq * a.q_head;
  float qf[4], o[4] = {0.0f, 0.0f, 0.0f, 0.0f}, m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; i++) qf[i] = 4 * lane + i < a.d ? elem<BF16>(q[4 * lane + i]) : 0.0f;
  for (int64_t j = warp; j < seen; j += kThreads / 32) {
    const int page = a.table[int64_t(b) * a.stride + j / a.bt];
    if (uint32_t(page) >= uint32_t(a.n_blocks)) {
      if (lane == 0) atomicOr(a.status, kStBadArg);
      continue;
    }
    const int64_t row = page_row(page, a.H, h, a.bt, int(j % a.bt), a.d);
    uint32_t kc = 0, vc = 0;
    if (4 * lane < a.d) {
      kc = *reinterpret_cast<const uint32_t *>(a.kp + row + 4 * lane);
      vc = *reinterpret_cast<const uint32_t *>(a.vp + row + 4 * lane);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++) s += qf[i] * value_of<FMT>((kc >> (8 * i)) & 0xffu);
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale_log2 * a.ks[int64_t(page) * a.H + h];
    const float top = fmaxf(m, s), keep = exp2f(m - top), p = exp2f(s - top), w = p * a.vs[int64_t(page) * a.H + h];
    l = l * keep + p;
#pragma unroll
    for (int i = 0; i < 4; i++) o[i] = o[i] * keep + w * value_of<FMT>((vc >> (8 * i)) & 0xffu);
    m = top;
  }
  __shared__ float s_m[4], s_l[4], s_o[4][128];
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
  for (int i = 0; i < 4; i++) s_o[warp][4 * lane + i] = o[i];
  __syncthreads();
  float top = -INFINITY, sum = 0.0f, x = 0.0f;
  for (int w = 0; w < 4; w++) top = fmaxf(top, s_m[w]);
  if (seen > 0)
    for (int w = 0; w < 4; w++) {
      const float f = s_m[w] == -INFINITY ? 0.0f : exp2f(s_m[w] - top);
      sum += f * s_l[w];
      x += f * s_o[w][threadIdx.x];
    }
  const int64_t r = (int64_t(b) * a.T + t) * a.Hq + hq;
  if (int(threadIdx.x) < a.d) a.out[r * a.d + threadIdx.x] = elem_of<BF16>(sum == 0.0f ? 0.0f : x / sum);
  if (threadIdx.x == 0 && a.lse) a.lse[r] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

bool attend_ok(const cg_cache *c, const cg_attend *t) {
  if (!cache8_ok(c) || !t || t->n_seq < 1 || t->q_tokens < 1 || t->Hq < 1 || t->Hq % c->H || t->table_stride < 1 ||
      (t->dtype != CG_F16 && t->dtype != CG_BF16) || !std::isfinite(t->scale) || !(t->scale > 0.0f))
    return false;
  for (int64_t s : t->q_stride)
    if (s % 8) return false;
  return t->n_seq <= (1 << 20) && t->q_tokens <= (1 << 16) && t->Hq <= 65535 &&
         int64_t(t->n_seq) * t->q_tokens <= 0x7fffffff;
}

}  // namespace
}  // namespace cg

extern "C" size_t cg_cache_workspace_bytes(const cg_cache *cache, const cg_attend *attend) {
  return cg::attend_ok(cache, attend) ? 256 : 0;
}

extern "C" cg_status cg_cache_attend(const cg_cache *cache, const cg_attend *attend, const void *q_dev,
                                     const void *k_pool, const void *v_pool, const float *k_scale,
                                     const float *v_scale, const int32_t *table_dev, const int32_t *len_dev,
                                     void *out_dev, float *lse_dev, void *ws_dev, size_t ws_bytes, void *stream) {
  using namespace cg;
  if (!attend_ok(cache, attend) || !q_dev || !k_pool || !v_pool || !k_scale || !v_scale || !table_dev || !len_dev ||
      !out_dev || !ws_dev)
    return CG_ERR_INVALID_ARG;
  if (!is_aligned(q_dev, 16) || !is_aligned(k_pool, 16) || !is_aligned(v_pool, 16) || !is_aligned(out_dev, 16) ||
      !is_aligned(k_scale, 4) || !is_aligned(v_scale, 4) || !is_aligned(table_dev, 4) || !is_aligned(len_dev, 4) ||
      !is_aligned(lse_dev, 4) || !is_aligned(ws_dev, 256) ||
      ws_bytes < cg_cache_workspace_bytes(cache, attend))
    return CG_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(ws_dev, 0, 256, st) != cudaSuccess) return CG_ERR_CUDA;
  AttendArgs a{};
  a.q = static_cast<const uint16_t *>(q_dev);
  a.kp = static_cast<const uint8_t *>(k_pool), a.vp = static_cast<const uint8_t *>(v_pool);
  a.ks = k_scale, a.vs = v_scale, a.table = table_dev, a.len = len_dev;
  a.out = static_cast<uint16_t *>(out_dev), a.lse = lse_dev;
  a.status = static_cast<uint32_t *>(ws_dev);
  a.q_seq = attend->q_stride[0], a.q_tok = attend->q_stride[1], a.q_head = attend->q_stride[2];
  a.B = attend->n_seq, a.T = attend->q_tokens, a.Hq = attend->Hq, a.H = cache->H, a.d = cache->d;
  a.bt = cache->block_tokens, a.n_blocks = cache->n_blocks, a.stride = attend->table_stride;
  a.scale_log2 = attend->scale * 1.4426950408889634f;
  const dim3 grid(unsigned(a.B * a.T), unsigned(a.Hq));
  const bool e4m3 = cache->format == CG_CACHE_E4M3, bf16 = attend->dtype == CG_BF16;
  if (e4m3 && bf16) k_attend<CG_CACHE_E4M3, true><<<grid, kThreads, 0, st>>>(a);
  if (e4m3 && !bf16) k_attend<CG_CACHE_E4M3, false><<<grid, kThreads, 0, st>>>(a);
  if (!e4m3 && bf16) k_attend<CG_CACHE_INT8, true><<<grid, kThreads, 0, st>>>(a);
  if (!e4m3 && !bf16) k_attend<CG_CACHE_INT8, false><<<grid, kThreads, 0, st>>>(a);
  return launched();
}
