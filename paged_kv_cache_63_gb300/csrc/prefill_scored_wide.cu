// prefill_scored_wide.cu -- the multi-token kernels of a score rule with a wide cap.
#include "prefill_launch.cuh"

namespace pa {

namespace {

// Every combination of parts has a cap.
template <int kParts>
pa_status_t launch_wide(int parts, int head_dim, const PrefillScoredArgs &a,
                        const PrefillLaunch &l, cudaStream_t stream) {
  if (parts == kParts) return launch_prefill<true, kParts>(head_dim, a, l, stream);
  if constexpr (kParts > (kRuleCap | kRuleWide))
    return launch_wide<kParts - 2>(parts, head_dim, a, l, stream);
  return PA_ERR_UNSUPPORTED;  // not reached
}

}  // namespace

pa_status_t launch_parts_wide(int parts, int head_dim, const PrefillScoredArgs &a,
                              const PrefillLaunch &l, cudaStream_t stream) {
  return launch_wide<kRuleCap | kRuleSlopes | kRuleFirst | kRuleWide>(parts, head_dim, a, l,
                                                                      stream);
}

}  // namespace pa
