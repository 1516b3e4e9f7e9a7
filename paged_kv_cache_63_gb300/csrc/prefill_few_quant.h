// prefill_few_quant.h -- the multi-token call over a quantised cache for few rows.
#pragma once

#include "internal.h"
#include "pagedattn.h"
#include "scored_softmax.cuh"

namespace pa {

// Whether the call, of at most max_query_len new tokens a sequence, goes to the kernel for few rows.
bool few_rows(const pa_problem_t *p, const ScoreArgs &s, int max_query_len);

// Launches it; `p` as filled for the other kernels.
pa_status_t launch_few_quant(const pa_problem_t *problem, const PrefillQuantArgs &p,
                             const void *query, int max_query_len, const pa_quant_cache_t *cache,
                             cudaStream_t stream);

}  // namespace pa
