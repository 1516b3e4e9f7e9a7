// prefill_scored.cu -- host entry point of multi-token attention under a score rule.
#include "prefill_launch.cuh"

namespace pa {
namespace {

// Launches the kernel compiled for the rule's parts.
template <int kParts>
pa_status_t launch_parts(int parts, int head_dim, const PrefillScoredArgs &a,
                         const PrefillLaunch &l, cudaStream_t stream) {
  if (parts == kParts) return launch_prefill<true, kParts>(head_dim, a, l, stream);
  if constexpr (kParts > 0) return launch_parts<kParts - 1>(parts, head_dim, a, l, stream);
  return PA_ERR_UNSUPPORTED;  // not reached
}

}  // namespace
}  // namespace pa

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
  if (total_tokens == 0) {  // no rows, so no addresses of any (an empty tensor's is null)
    query = key_cache;
    out = const_cast<void *>(value_cache);  // not written
  }
  PrefillLaunch l;
  st = setup_prefill(problem, query, query_start, total_tokens, max_query_len, key_cache,
                     value_cache, block_tables, context_lengths, scale, out, options, &l, &a);
  if (st != PA_OK || l.grid.x == 0) return st;
  // a masked score is an infinity times the scale, so the scale is never 0: with this one every
  // finite dot product (below 2^41) still scores 0 in fp32 next to the maximum
  if (a.scale_log2 == 0.f) a.scale_log2 = 1e-30f;
  a.out16 = static_cast<uint16_t *>(out);
  const int parts = (a.s.cap_in != 0.f ? kRuleCap : 0) | (a.s.slopes ? kRuleSlopes : 0) |
                    (a.s.first ? kRuleFirst : 0);
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  if (a.s.cap_wide) return launch_parts_wide(parts | kRuleWide, problem->head_dim, a, l, on);
  return launch_parts<kRuleParts - 1>(parts, problem->head_dim, a, l, on);
}
