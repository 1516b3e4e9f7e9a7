// prefill_launch.cuh -- host-side set-up and launch of the multi-token kernels: the two-tile
// kernel for head_dim 64 and 128, the single-tile kernel for 256, plain or under a score rule.
#pragma once

#include "internal.h"
#include "pagedattn.h"
#include "prefill2_scored_kernel.cuh"
#include "prefill_scored_kernel.cuh"

namespace pa {

struct PrefillLaunch {
  CUtensorMap tq, tk, tv;
  dim3 grid;  // x = 0: nothing to do
};

// Checks the arguments of a multi-token call and fills its tensor maps, grid and kernel
// arguments but the output (defined in prefill.cu). `args` comes in zeroed.
pa_status_t setup_prefill(const pa_problem_t *problem, const void *query,
                          const int32_t *query_start, int64_t total_tokens, int32_t max_query_len,
                          const void *key_cache, const void *value_cache,
                          const int32_t *block_tables, const int32_t *context_lengths, float scale,
                          const void *out, const pa_options_t *options, PrefillLaunch *l,
                          PrefillArgs *args);

// head_dim 64 / 128: two query tiles per CTA (a.n_qtiles counts pairs, grid.z too)
template <int HD, bool kScored, int kParts>
cudaError_t launch_prefill2_hd(const PrefillArgsOf<kScored> &a, const PrefillLaunch &l,
                               cudaStream_t stream) {
  static std::atomic<bool> set[kMaxLaunchDevices];
  constexpr int smem = Prefill2Cfg<HD>::kSmem + 1024;
  void (*kern)(PrefillArgsOf<kScored>, CUtensorMap, CUtensorMap, CUtensorMap);
  if constexpr (kScored)
    kern = prefill2_scored_kernel<HD, kParts>;
  else
    kern = prefill2_kernel<HD>;
  const cudaError_t e = allow_smem(kern, smem, set);
  if (e != cudaSuccess) return e;
  if constexpr (kScored)
    return launch_early(kern, l.grid, kPrefill2Threads, smem, stream, a, l.tq, l.tk, l.tv);
  kern<<<l.grid, kPrefill2Threads, smem, stream>>>(a, l.tq, l.tk, l.tv);
  return cudaGetLastError();
}

template <int HD, bool kScored, int kParts>
cudaError_t launch_prefill_hd(const PrefillArgsOf<kScored> &a, const PrefillLaunch &l,
                              cudaStream_t stream) {
  static std::atomic<bool> set[kMaxLaunchDevices];
  constexpr int smem = PrefillCfg<HD>::kSmem + 1024;
  void (*kern)(PrefillArgsOf<kScored>, CUtensorMap, CUtensorMap, CUtensorMap);
  if constexpr (kScored)
    kern = prefill_scored_kernel<HD, kParts>;
  else
    kern = prefill_kernel<HD>;
  const cudaError_t e = allow_smem(kern, smem, set);
  if (e != cudaSuccess) return e;
  if constexpr (kScored)
    return launch_early(kern, l.grid, kScoredThreads, smem, stream, a, l.tq, l.tk, l.tv);
  kern<<<l.grid, kPrefillThreads, smem, stream>>>(a, l.tq, l.tk, l.tv);
  return cudaGetLastError();
}

template <bool kScored, int kParts = 0>
pa_status_t launch_prefill(int head_dim, const PrefillArgsOf<kScored> &a, const PrefillLaunch &l,
                           cudaStream_t stream) {
  cudaError_t e;
  switch (head_dim) {
    case 64: e = launch_prefill2_hd<64, kScored, kParts>(a, l, stream); break;
    case 128: e = launch_prefill2_hd<128, kScored, kParts>(a, l, stream); break;
    case 256: e = launch_prefill_hd<256, kScored, kParts>(a, l, stream); break;
    default: return PA_ERR_UNSUPPORTED;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// Launches the scored kernel compiled for the parts of a rule with a wide cap
// (prefill_scored_wide.cu).
pa_status_t launch_parts_wide(int parts, int head_dim, const PrefillScoredArgs &a,
                              const PrefillLaunch &l, cudaStream_t stream);

}  // namespace pa
