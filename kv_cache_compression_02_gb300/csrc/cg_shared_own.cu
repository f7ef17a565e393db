// cg_shared_own.cu -- cg_cache_attend's kernels for cg_shared_attend: what each
// sequence has behind the pages that it shares.
#include "cg_shared.cuh"

#include "cg_attend.cuh"

namespace cg {

bool attend_args_ok(const cg_cache *cache, const cg_attend *attend) { return attend_ok(cache, attend); }

uint64_t attend_own_bytes(const cg_cache *cache, const cg_attend *attend) { return attend_bytes(cache, attend); }

cg_status attend_own(const cg_cache *cache, const cg_attend *attend, const int32_t *first, float *own, float *own_ml, const void *q_dev,
                     const void *k_pool, const void *v_pool, const float *k_scale, const float *v_scale, const int32_t *table_dev,
                     const int32_t *len_dev, void *out_dev, float *lse_dev, uint8_t *ws, cudaStream_t st) {
  AttendArgs a{};
  a.first = first, a.own = own, a.own_ml = own_ml;
  return run_attend<true>(a, cache, attend, q_dev, k_pool, v_pool, k_scale, v_scale, table_dev, len_dev, out_dev, lse_dev, ws, st);
}

}  // namespace cg
