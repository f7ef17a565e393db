// cg_shared.cuh -- what cg_shared_attend's own kernels (cg_shared.cu) need of
// those that it has in common with cg_cache_attend (cg_shared_own.cu).
#pragma once

#include <cuda_runtime.h>

#include "cachegen_cache.h"

namespace cg {

bool attend_args_ok(const cg_cache *cache, const cg_attend *attend);
uint64_t attend_own_bytes(const cg_cache *cache, const cg_attend *attend);

// New tokens attend over what each sequence has behind its first `first` pages.
// A sequence without such pages gets its outputs; of the others the rows go, not
// normalised, to own [n_seq][T][Hq][d] with maximum and sum in own_ml.
cg_status attend_own(const cg_cache *cache, const cg_attend *attend, const int32_t *first, float *own, float *own_ml, const void *q_dev,
                     const void *k_pool, const void *v_pool, const float *k_scale, const float *v_scale, const int32_t *table_dev,
                     const int32_t *len_dev, void *out_dev, float *lse_dev, uint8_t *ws, cudaStream_t st);

}  // namespace cg
