// cg_prompt.cu -- cg_prompt_attend: causal attention of packed prompts.
#include "cg_cache.cuh"

namespace cg {
namespace {

constexpr int kThreads = 128;

struct PromptArgs {
  const uint16_t *q, *k, *v;
  const int32_t *cu_q, *cu_k;
  uint16_t *out;
  float *lse;
  uint32_t *status;
  int64_t qs[2], ks[2], vs[2];
  int n_seq, Hq, H, d, max_q, max_k, n_q, n_k;
  float scale_log2;  // scale * log2(e)
};

// One CTA per (query row of a sequence, head); each warp takes every fourth
// key and keeps its own running maximum, sum and output.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_prompt(const PromptArgs a) {
  const int b = blockIdx.y, i = blockIdx.x, hq = blockIdx.z, h = hq / (a.Hq / a.H);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q0 = a.cu_q[b], nq = a.cu_q[b + 1] - q0, k0 = a.cu_k[b], nk = a.cu_k[b + 1] - k0;
  if (q0 < 0 || nq < 0 || nq > a.max_q || nq > a.n_q - q0 || k0 < 0 || nk < 0 || nk > a.max_k || nk > a.n_k - k0) {
    if (i == 0 && hq == 0 && threadIdx.x == 0) atomicOr(a.status, kStBadArg);
    return;
  }
  if (i >= nq) return;
  const int seen = i + nk - nq + 1;
  const uint16_t *q = a.q + int64_t(q0 + i) * a.qs[0] + hq * a.qs[1];
  float qf[4], o[4] = {0.0f, 0.0f, 0.0f, 0.0f}, m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int x = 0; x < 4; x++) qf[x] = 4 * lane + x < a.d ? elem<BF16>(q[4 * lane + x]) : 0.0f;
  for (int j = warp; j < seen; j += kThreads / 32) {
    uint2 kc = make_uint2(0, 0), vc = make_uint2(0, 0);
    if (4 * lane < a.d) {
      kc = *reinterpret_cast<const uint2 *>(a.k + int64_t(k0 + j) * a.ks[0] + h * a.ks[1] + 4 * lane);
      vc = *reinterpret_cast<const uint2 *>(a.v + int64_t(k0 + j) * a.vs[0] + h * a.vs[1] + 4 * lane);
    }
    float s = 0.0f;
#pragma unroll
    for (int x = 0; x < 4; x++) s += qf[x] * elem<BF16>(uint16_t((x < 2 ? kc.x : kc.y) >> (16 * (x & 1))));
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale_log2;
    const float top = fmaxf(m, s), keep = exp2f(m - top), p = exp2f(s - top);
    l = l * keep + p;
#pragma unroll
    for (int x = 0; x < 4; x++) o[x] = o[x] * keep + p * elem<BF16>(uint16_t((x < 2 ? vc.x : vc.y) >> (16 * (x & 1))));
    m = top;
  }
  __shared__ float s_m[4], s_l[4], s_o[4][128];
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
  for (int x = 0; x < 4; x++) s_o[warp][4 * lane + x] = o[x];
  __syncthreads();
  float top = -INFINITY, sum = 0.0f, x = 0.0f;
  for (int w = 0; w < 4; w++) top = fmaxf(top, s_m[w]);
  if (seen > 0)
    for (int w = 0; w < 4; w++) {
      const float f = s_m[w] == -INFINITY ? 0.0f : exp2f(s_m[w] - top);
      sum += f * s_l[w];
      x += f * s_o[w][threadIdx.x];
    }
  const int64_t r = int64_t(q0 + i) * a.Hq + hq;
  if (int(threadIdx.x) < a.d) a.out[r * a.d + threadIdx.x] = elem_of<BF16>(sum == 0.0f ? 0.0f : x / sum);
  if (threadIdx.x == 0 && a.lse) a.lse[r] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

bool prompt_ok(const cg_prompt *p) {
  if (!p || p->n_seq < 1 || p->n_seq > 65535 || p->H < 1 || p->Hq < 1 || p->Hq > 65535 || p->Hq % p->H ||
      p->Hq / p->H > 128 || p->d < 8 || p->d > 128 || p->d % 8 || (p->dtype != CG_F16 && p->dtype != CG_BF16) ||
      p->max_q < 0 || p->max_k < 0 || p->n_q < 0 || p->n_k < 0 || !std::isfinite(p->scale) || !(p->scale > 0.0f))
    return false;
  for (int i = 0; i < 2; i++)
    if (p->q_stride[i] % 8 || p->k_stride[i] % 8 || p->v_stride[i] % 8) return false;
  return true;
}

}  // namespace
}  // namespace cg

extern "C" size_t cg_prompt_workspace_bytes(const cg_prompt *prompt) { return cg::prompt_ok(prompt) ? 256 : 0; }

extern "C" cg_status cg_prompt_attend(const cg_prompt *prompt, const void *q_dev, const void *k_dev,
                                      const void *v_dev, const int32_t *cu_q_dev, const int32_t *cu_k_dev,
                                      void *out_dev, float *lse_dev, void *ws_dev, size_t ws_bytes, void *stream) {
  using namespace cg;
  if (!prompt_ok(prompt) || !q_dev || !k_dev || !v_dev || !cu_q_dev || !cu_k_dev || !out_dev || !ws_dev)
    return CG_ERR_INVALID_ARG;
  if (!is_aligned(q_dev, 16) || !is_aligned(k_dev, 16) || !is_aligned(v_dev, 16) || !is_aligned(out_dev, 16) ||
      !is_aligned(cu_q_dev, 4) || !is_aligned(cu_k_dev, 4) || !is_aligned(lse_dev, 4) || !is_aligned(ws_dev, 256) ||
      ws_bytes < cg_prompt_workspace_bytes(prompt))
    return CG_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(ws_dev, 0, 256, st) != cudaSuccess) return CG_ERR_CUDA;
  if (prompt->max_q == 0) return CG_OK;
  PromptArgs a{};
  a.q = static_cast<const uint16_t *>(q_dev), a.k = static_cast<const uint16_t *>(k_dev);
  a.v = static_cast<const uint16_t *>(v_dev);
  a.cu_q = cu_q_dev, a.cu_k = cu_k_dev;
  a.out = static_cast<uint16_t *>(out_dev), a.lse = lse_dev, a.status = static_cast<uint32_t *>(ws_dev);
  for (int i = 0; i < 2; i++) a.qs[i] = prompt->q_stride[i], a.ks[i] = prompt->k_stride[i], a.vs[i] = prompt->v_stride[i];
  a.n_seq = prompt->n_seq, a.Hq = prompt->Hq, a.H = prompt->H, a.d = prompt->d;
  a.max_q = prompt->max_q, a.max_k = prompt->max_k, a.n_q = prompt->n_q, a.n_k = prompt->n_k;
  a.scale_log2 = prompt->scale * 1.4426950408889634f;
  const dim3 grid(unsigned(a.max_q), unsigned(a.n_seq), unsigned(a.Hq));
  if (prompt->dtype == CG_BF16)
    k_prompt<true><<<grid, kThreads, 0, st>>>(a);
  else
    k_prompt<false><<<grid, kThreads, 0, st>>>(a);
  return launched();
}
