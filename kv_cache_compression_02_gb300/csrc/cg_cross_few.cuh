// cg_cross_few.cuh -- cg_cross_attend where a sequence has few query rows for a KV head.
#pragma once

#include <cuda_runtime.h>

#include "cachegen_cache.h"

namespace cg {

// Up to this many rows (queries x Hq / H) the keys are what is to be moved, and
// tiles of 128 rows would be nearly empty: 64 sequences of one query and 16
// heads on 100 to 1500 keys take 28 us here, 66 us on those; 40 of up to 12 rows
// on 333 to 901 keys 14.6 us and 25.7 us (ten calls in a graph).
constexpr int kFewRows = 16;

uint64_t few_bytes(const cg_prompt &p);  // of the workspace

cg_status cross_few(const cg_prompt &p, const void *q_dev, const void *k_dev, const void *v_dev, const int32_t *cu_q_dev,
                    const int32_t *k_begin_dev, const int32_t *k_len_dev, void *out_dev, float *lse_dev, uint8_t *ws, cudaStream_t st);

}  // namespace cg
