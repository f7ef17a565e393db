// cg_cache_attend.cu -- cg_cache_attend: new tokens attend over 8-bit pages (the
// kernels are in cg_attend.cuh).
#include "cg_attend.cuh"

extern "C" size_t cg_cache_workspace_bytes(const cg_cache *cache, const cg_attend *attend) {
  using namespace cg;
  if (!attend_ok(cache, attend)) return 0;
  return size_t(attend_bytes(cache, attend));
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
  return run_attend<false>(AttendArgs{}, cache, attend, q_dev, k_pool, v_pool, k_scale, v_scale, table_dev, len_dev, out_dev, lse_dev,
                           static_cast<uint8_t *>(ws_dev), static_cast<cudaStream_t>(stream));
}
