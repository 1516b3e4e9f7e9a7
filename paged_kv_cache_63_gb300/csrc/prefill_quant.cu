#include "internal.h"
extern "C" pa_status_t pa_prefill_quant(const pa_problem_t *, const pa_score_t *, const void *, const int32_t *, int64_t, int32_t, const pa_quant_cache_t *, const int32_t *, const int32_t *, float, void *, const pa_options_t *, void *) { return PA_ERR_UNSUPPORTED; }
