// prefill.cu -- host entry point of the causal multi-token (prefill) kernels, and the argument
// checks and tensor maps that it shares with the one under a score rule.
#include <cmath>

#include "prefill_launch.cuh"

namespace pa {

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

pa_status_t setup_prefill(const pa_problem_t *problem, const void *query,
                          const int32_t *query_start, int64_t total_tokens, int32_t max_query_len,
                          const void *key_cache, const void *value_cache,
                          const int32_t *block_tables, const int32_t *context_lengths, float scale,
                          const void *out, const pa_options_t *options, PrefillLaunch *l,
                          PrefillArgs *args, bool codes) {
  l->grid = dim3(0, 0, 0);
  pa_status_t st = check_problem_public(problem);
  if (st != PA_OK) return st;
  if (options && (options->schedule || options->math || options->combine || options->workers ||
                  options->stages || options->warps_per_cta || options->tile_tokens ||
                  (options->test_flags & ~PA_TEST_EXPIRE_WAITS)))
    return PA_ERR_INVALID_ARG;
  if (!query || !query_start || !key_cache || !value_cache || !block_tables ||
      !context_lengths || !out || !std::isfinite(scale))
    return PA_ERR_INVALID_ARG;
  if (total_tokens < 0 || total_tokens >= (int64_t(1) << 31) || max_query_len < 0)
    return PA_ERR_INVALID_ARG;
  if (!aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(query_start) & 3u) ||
      (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
      (reinterpret_cast<uintptr_t>(context_lengths) & 3u))
    return PA_ERR_MISALIGNED;
  const int g = problem->query_heads / problem->kv_heads;
  if (g > 128) return PA_ERR_UNSUPPORTED;
  if (problem->batch == 0 || total_tokens == 0 || max_query_len == 0) return PA_OK;  // empty grid
  if (problem->batch > 65535 || problem->kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  int smem_optin = 0;  // only the device check matters: both kernels fit any sm_103
  st = current_device_smem(&smem_optin);
  if (st != PA_OK) return st;

  const int hd = problem->head_dim;
  const int tn = hd == 256 ? 64 : 128;
  const int qt = 128 / g;
  const long long n_qtiles = (static_cast<long long>(max_query_len) + qt - 1) / qt;
  if (n_qtiles > 65535) return PA_ERR_UNSUPPORTED;

  PrefillArgs &a = *args;
  a.qs = query_start;
  a.bt = block_tables;
  a.ctx = context_lengths;
  a.err = device_error_word();
  if (!a.err) return PA_ERR_CUDA;
  a.total = total_tokens;
  a.batch = problem->batch;
  a.qh = problem->query_heads;
  a.kvh = problem->kv_heads;
  a.ps = problem->page_size;
  a.ps_shift = 0;
  while ((1 << a.ps_shift) < a.ps) ++a.ps_shift;
  a.maxp = problem->max_pages_per_sequence;
  a.num_pages = problem->num_physical_pages;
  a.layout = problem->cache_layout;
  a.g = g;
  a.qt = qt;
  a.n_qtiles = static_cast<int>(n_qtiles);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.expire = (options && (options->test_flags & PA_TEST_EXPIRE_WAITS)) ? 1 : 0;
  a.out_v8 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0 ? 1 : 0;

  const int rows = a.ps < tn ? a.ps : tn;
  st = encode_query_map(&l->tq, query, total_tokens, a.qh, hd, g, qt);
  if (st != PA_OK) return st;
  st = encode_cache_map_rows(&l->tk, key_cache, problem, rows, codes);
  if (st != PA_OK) return st;
  st = encode_cache_map_rows(&l->tv, value_cache, problem, rows, codes);
  if (st != PA_OK) return st;

  if (hd != 256) a.n_qtiles = (a.n_qtiles + 1) / 2;  // pairs of query tiles
  l->grid = dim3(a.kvh, a.batch, a.n_qtiles);
  return PA_OK;
}

}  // namespace pa

extern "C" pa_status_t pa_prefill(const pa_problem_t *problem, const void *query,
                                  const int32_t *query_start, int64_t total_tokens,
                                  int32_t max_query_len, const void *key_cache,
                                  const void *value_cache, const int32_t *block_tables,
                                  const int32_t *context_lengths, float scale, float *out,
                                  const pa_options_t *options, void *stream) {
  using namespace pa;
  PrefillLaunch l;
  PrefillArgs a = {};
  pa_status_t st = setup_prefill(problem, query, query_start, total_tokens, max_query_len,
                                 key_cache, value_cache, block_tables, context_lengths, scale, out,
                                 options, &l, &a);
  if (st != PA_OK || l.grid.x == 0) return st;
  a.out = out;
  return launch_prefill<false>(problem->head_dim, a, l, static_cast<cudaStream_t>(stream));
}
