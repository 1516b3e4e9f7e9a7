// prefill_scored.cu -- host entry point of multi-token attention under a score rule.
#include "prefill_launch.cuh"

extern "C" pa_status_t pa_prefill_scored(const pa_problem_t *problem, const pa_score_t *score,
                                         const void *query, const int32_t *query_start,
                                         int64_t total_tokens, int32_t max_query_len,
                                         const void *key_cache, const void *value_cache,
                                         const int32_t *block_tables,
                                         const int32_t *context_lengths, float scale, void *out,
                                         const pa_options_t *options, void *stream) {
  using namespace pa;
  PrefillScoredArgs a = {};
  pa_status_t st = check_problem_public(problem);
  if (st != PA_OK) return st;
  if (!score) return PA_ERR_INVALID_ARG;
  st = resolve_score(score, scale, &a.s);
  if (st != PA_OK) return st;
  if (!a.s.out_half) return PA_ERR_UNSUPPORTED;
  PrefillLaunch l;
  st = setup_prefill(problem, query, query_start, total_tokens, max_query_len, key_cache,
                     value_cache, block_tables, context_lengths, scale, out, options, &l, &a);
  if (st != PA_OK || l.grid.x == 0) return st;
  // a masked score is an infinity times the scale, so the scale is never 0: with this one every
  // finite dot product (below 2^41) still scores 0 in fp32 next to the maximum
  if (a.scale_log2 == 0.f) a.scale_log2 = 1e-30f;
  a.out16 = static_cast<uint16_t *>(out);
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  // Only with first_tokens may a row see nothing. The code for such rows slows calls that have
  // none by its size alone: eight prompts of 2048 (head_dim 128, a window of 1024) took 312 us
  // with it and 281 without, two of 4096 at head_dim 256 443 and 403.
  return a.s.first ? launch_prefill<true, true>(problem->head_dim, a, l, on)
                   : launch_prefill<true, false>(problem->head_dim, a, l, on);
}
