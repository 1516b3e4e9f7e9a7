// decode_quant.cu -- one decode step over a quantised paged cache (pa_decode_quant), with the score
// rules of pa_decode_scored.
//
// Mathematics, for query head h of sequence b at position p = context - 1, codes c and scales f of
// the cached rows (quant.cuh):
//   s_t = rule(scale f^K_t q . c^K_t);   out = sum_t softmax(s)_t f^V_t c^V_t
// over the tokens that the rule lets the query see. Bound: HBM -- 2 (head_dim + 1) bytes a token and
// K/V head are read once, 4 g flops a code pair (g query heads a K/V head).
//
// The work is laid out as in decode_scored.cu (span_split.cuh): a warp is a worker with a ring of
// K/V tiles loaded by TMA, the tiles of all units are cut into equal ranges, and the states of units
// that workers share are joined by the same kernel. A tile is twice the tokens in the same bytes, and
// the instructions a tile takes decide how near the kernel comes to the memory:
//  * Scores are products of 16 tokens by 8 heads, outputs of 16 elements by 8 heads (m16n8k16), so
//    that all rows of an instruction carry work. Codes are converted to fp16, exactly, as they become
//    operands: a word of four keys' elements is two words of the first product (the queries are held
//    in the same order). Values' bytes are transposed by ldmatrix, so that a lane holds four tokens of
//    one element, and the tokens are dealt to the rows of both products so that these are the ones
//    whose weights the lane has. (Products of the codes themselves, the query split into three e4m3
//    numbers, took 168 us for 64 sequences of 1500 seen tokens with 32 heads of their own: the
//    compiler converts both operands for each product.)
//  * A key's scale multiplies its score in fp32; a value's scale multiplies its probability, relative
//    to the tile's smallest, whose own power of two multiplies the tile's output, or its codes where a
//    tile's scales lie far apart (code_walk.cuh, kScaleSpan). Scales come by 8-byte asynchronous copies
//    that arrive on the tile's barrier: a page may hold fewer of them than the 16 bytes of a TMA copy.
//  * Probabilities keep 22 bits (two fp16 numbers, a product each) and sums are fp32, as in
//    decode_scored.cu.
// 64 sequences of 1500 seen tokens, 32 heads of 128 of their own: 134.2 us, 0.88 of the copy bandwidth;
// four contexts of 100000, 24 / 4 heads of 256: 137 us, 0.90.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "code_walk.cuh"

namespace pa {

template <int HD>
__device__ __forceinline__ void code_begin(CodeState<HD> &st, const ScoredArgs &a, int b, int h0,
                                           int nh) {
  const int lane = threadIdx.x & 31;
  const int h = lane >> 2, pair = 2 * (lane & 3);
  const uint2 *src = reinterpret_cast<const uint2 *>(
      a.k.q + (static_cast<long long>(b) * a.k.qh + h0 + h) * HD);
#pragma unroll
  for (int k = 0; k < HD / 16; ++k) {
    const uint2 q = h < nh ? __ldg(src + k * 4 + (lane & 3)) : make_uint2(0u, 0u);
    st.q[k][0] = q.x;
    st.q[k][1] = q.y;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    st.slope2[j] = a.s.slopes && pair + j < nh ? __ldg(a.s.slopes + h0 + pair + j) * kLog2e : 0.f;
    st.m[j] = -INFINITY;
    st.lsum[j] = 0.f;
  }
#pragma unroll
  for (int k = 0; k < HD / 16; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) st.o[k][i] = 0.f;
}

template <int HD, int T>
__global__ void __launch_bounds__(kQuantWarps * 32, 1)
    decode_quant_kernel(const __grid_constant__ QuantDecodeArgs sa,
                        const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv) {
  using G = CodeGeom<HD, T>;
  const KernelArgs &a = sa.k;
  extern __shared__ uint8_t dsm[];
  __shared__ __align__(8) uint64_t bars[kQuantWarps * kMaxStages];
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int worker = (blockIdx.x * (blockDim.x >> 5) + warp) / a.group;
  const int member = warp % a.group;
  const int S = a.stages;
  const uint32_t base = (smem_addr(dsm) + kSmemAlign - 1) & ~static_cast<uint32_t>(kSmemAlign - 1);
  const uint32_t wbase = base + warp * a.warp_smem;
  // the scales lie behind all warps' rings
  const uint32_t wscales = base + (blockDim.x >> 5) * a.warp_smem + warp * S * G::kScaleBytes;
  const uint32_t bar0 = smem_addr(&bars[warp * kMaxStages]);

  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(bar0 + 8 * s, 33);
    fence_barrier_init();
    prefetch_tensormap(&tk);
    prefetch_tensormap(&tv);
  }
  __syncwarp();
  wait_for_stream();

  {
    // warm L2 with the small inputs every warp reads first
    const long long nthreads = static_cast<long long>(gridDim.x) * blockDim.x;
    const long long tid = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    const long long ctx_lines = (static_cast<long long>(a.batch) * 4 + 127) / 128;
    const long long bt_lines = (static_cast<long long>(a.batch) * a.maxp * 4 + 127) / 128;
    const long long q_lines = (static_cast<long long>(a.batch) * a.qh * a.hd * 2 + 127) / 128;
    for (long long i = tid; i < ctx_lines + bt_lines + q_lines; i += nthreads) {
      const char *p =
          i < ctx_lines ? reinterpret_cast<const char *>(a.ctx) + i * 128
          : i < ctx_lines + bt_lines
              ? reinterpret_cast<const char *>(a.bt) + (i - ctx_lines) * 128
              : reinterpret_cast<const char *>(a.q) + (i - ctx_lines - bt_lines) * 128;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
    }
  }

  // ---- the worker's range
  SpanCursor c;
  long long total = 0, nworkers = 0;
  if (a.mode == MODE_BALANCED) {
    if (worker >= a.workers) return;
    const bool any = span_balanced_start(sa, worker, T, c, total, nworkers);
    // sequences that see nothing: worker b mod workers zeroes their rows; lanes test 32
    // candidates at once
    for (long long b0 = worker; b0 < a.batch; b0 += 32ll * a.workers) {
      const long long bl = b0 + static_cast<long long>(lane) * a.workers;
      unsigned empty = __ballot_sync(
          0xffffffffu, bl < a.batch && span_tiles(load_span(sa, static_cast<int>(bl)), T) == 0);
      while (empty) {
        const int j = __ffs(empty) - 1;
        empty &= empty - 1;
        const int b = static_cast<int>(b0 + static_cast<long long>(j) * a.workers);
        for (int us = member; us < a.ups; us += a.group)
          zero_rows_out<HD>(sa, unit_info(a, b, us));
      }
    }
    if (!any) return;
  } else {  // MODE_SINGLE
    if (worker >= a.batch * a.upg) return;
    c.b = worker / a.upg;
    c.us = worker % a.upg;
    c.sp = load_span(sa, c.b);
    c.tok = span_start(c.sp, T);
    c.left = span_tiles(c.sp, T);
    c.ug0 = 0;
    if (c.left == 0) {
      zero_rows_out<HD>(sa, unit_info(a, c.b, c.us * a.group + member));
      return;
    }
  }

  // ---- pipeline
  const uint64_t pol = l2_evict_first_policy();
  SpanCursor ic = c;
  BtWindow win;
  win.b = -1;
  win.base = 0;
  win.cur = win.nxt = -1;
  // the stage and phase parity of the next tile to consume, the stage of the next one to issue,
  // and the tiles in flight
  int cs = 0, is = 0, flying = 0;
  uint32_t cphase = 0, extra = a.tx_extra;
  int ius = ic.us, ikv = (ic.us * a.group + member) / a.sub;  // K/V head of the cursor's unit
  auto issue = [&]() {
    if (ic.us != ius) {
      ius = ic.us;
      ikv = (ic.us * a.group + member) / a.sub;
    }
    issue_code_tile<HD, T>(sa, &tk, &tv, ic, ikv, win, wbase + is * G::kStageBytes,
                           wscales + is * G::kScaleBytes, bar0 + 8 * is, pol, extra);
    extra = 0;
    is = is + 1 == S ? 0 : is + 1;
    ++flying;
    advance(sa, ic, T);
  };
  CodeState<HD> st = {};
  CodeLane<HD, T> lane_addr;
  lane_addr.init();
  UnitInfo cur;
  cur.b = -1;
  cur.us = -1;
  cur.h0 = cur.nh = 0;
  long long cur_ug0 = 0;
  int cur_tiles = 0;
  bool aborted = false;

  auto finish_unit = [&]() {
    bool whole = true;
    const long long unit = static_cast<long long>(cur.b) * a.ups + cur.us;
    if (a.mode == MODE_BALANCED)
      whole = worker_of(cur_ug0, total, nworkers) ==
              worker_of(cur_ug0 + cur_tiles - 1, total, nworkers);
    const int element = lane >> 2;
    float sum[2] = {st.lsum[0], st.lsum[1]};
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
      sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], o);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int h = 2 * (lane & 3) + j;
      const float l = sum[j];
      if (h >= cur.nh) break;
      if (whole) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const long long at = (static_cast<long long>(cur.b) * a.qh + cur.h0 + h) * HD + element;
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          store_out1(sa.s, sa.out, at + k * 16, st.o[k][j] * inv);
          store_out1(sa.s, sa.out, at + k * 16 + 8, st.o[k][2 + j] * inv);
        }
      } else {
        // partial state relative to the head's reference, for the joining kernel
        const long long slot = slot_of(unit, worker, a.group) * kMaxHeads + h;
        if (element == 0)
          *reinterpret_cast<float2 *>(a.ws_ml + slot * 2) = make_float2(st.m[j], l);
        float *dst = a.ws_acc + slot * HD + element;
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          dst[k * 16] = st.o[k][j];
          dst[k * 16 + 8] = st.o[k][2 + j];
        }
      }
    }
  };

  // ---- main loop: fill the ring, wait for the next tile, compute
  for (;;) {
    const bool done = c.left <= 0;
    // the joining kernel may come up now (it waits for this grid before it reads any state)
    if (done) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const bool change = done || c.b != cur.b || c.us * a.group + member != cur.us;
    if (change && cur.b >= 0) finish_unit();
    if (done) break;
#pragma unroll 1
    while (flying < S && ic.left > 0) issue();
    if (change) {
      cur = unit_info(a, c.b, c.us * a.group + member);
      cur_ug0 = c.ug0;
      cur_tiles = span_tiles(c.sp, T);
      code_begin<HD>(st, sa, cur.b, cur.h0, cur.nh);
    }
    if (!mbar_wait(bar0 + 8 * cs, cphase, a.err)) {
      aborted = true;
      break;
    }
    code_tile<HD, T>(st, lane_addr, wbase + cs * G::kStageBytes, wscales + cs * G::kScaleBytes, c, sa,
                     OneQuery{c.sp});
    fence_proxy_async();
    __syncwarp();
    if (++cs == S) {
      cs = 0;
      cphase ^= 1u;
    }
    --flying;
    advance(sa, c, T);
  }
  if (aborted) {
    // let the copies still in flight land before the shared memory is given up
    for (; flying > 0; --flying) {
      mbar_wait(bar0 + 8 * cs, cphase, a.err);
      if (++cs == S) {
        cs = 0;
        cphase ^= 1u;
      }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
}

namespace {

// What pa_decode_quant launches, in pa_plan's terms. `score`: null, or the resolved rule.
pa_status_t quant_plan(const pa_problem_t *p, const pa_options_t *o, int sm_count,
                       const ScoreArgs *score, pa_plan_t *pl) {
  if (o && (o->stages < 0 || o->stages > kMaxStages || o->warps_per_cta < 0 ||
            o->warps_per_cta > kMaxWarpsPerCta))
    return PA_ERR_INVALID_ARG;
  pa_options_t rest = o ? *o : pa_options_t{};
  rest.stages = rest.warps_per_cta = 0;  // what they take of shared memory is another here
  pa_status_t st = pa_plan(p, &rest, sm_count, pl);  // its checks, and the split into units
  if (st != PA_OK) return st;
  if (o && (o->math || o->combine || o->tile_tokens)) return PA_ERR_UNSUPPORTED;
  const int g = p->query_heads / p->kv_heads;
  const int sub = (g + kMaxHeads - 1) / kMaxHeads;
  pl->tile_tokens = quant_tile(p->head_dim);
  pl->warps_per_cta = o && o->warps_per_cta ? o->warps_per_cta : kQuantWarps;
  pl->stages = o && o->stages ? o->stages : kQuantStages;
  pl->smem_bytes = quant_smem(p->head_dim, pl->warps_per_cta, pl->stages);
  if (pl->smem_bytes > kMaxDecodeSmem) return PA_ERR_UNSUPPORTED;
  int a = p->kv_heads * sub, b = pl->warps_per_cta;
  while (b) {
    const int t = a % b;
    a = b;
    b = t;
  }
  pl->group = a;
  const int64_t capacity = static_cast<int64_t>(sm_count) * pl->warps_per_cta;
  pl->schedule = o ? o->schedule : PA_SCHEDULE_AUTO;
  if (pl->schedule == PA_SCHEDULE_AUTO) {
    const int64_t most = static_cast<int64_t>(p->max_pages_per_sequence) * p->page_size;
    const int T = pl->tile_tokens;
    int64_t tiles = (most + T - 1) / T;
    if (score && score->window > 0 && score->window < most)
      tiles = std::min(tiles, (int64_t{score->window} + 2 * T - 2) / T);
    // as for pa_decode_scored: few tiles to a unit are walked faster than shared and joined, and
    // units alone fill the GPU where there are many
    pl->schedule = tiles <= 3 || (pl->units >= 4 * capacity && most <= 1024)
                       ? PA_SCHEDULE_SINGLE
                       : PA_SCHEDULE_BALANCED;
  }
  pl->workers = pl->units;
  pl->workspace_bytes = 0;
  pl->combine = PA_COMBINE_KERNEL;
  if (pl->schedule == PA_SCHEDULE_BALANCED) {
    pl->workers = o && o->workers ? o->workers : static_cast<int>(capacity);
    pl->workers = (pl->workers + pl->group - 1) / pl->group * pl->group;
    const int64_t slots = static_cast<int64_t>(pl->units) + pl->workers;
    pl->workspace_bytes = (slots * kMaxHeads * 2 * 4 + 255) / 256 * 256 +
                          slots * kMaxHeads * p->head_dim * 4;
  }
  pl->ctas = (std::max(pl->workers, 1) + pl->warps_per_cta - 1) / pl->warps_per_cta;
  return PA_OK;
}

template <int HD, int T>
cudaError_t launch_quant(const QuantDecodeArgs &a, const CUtensorMap &tk, const CUtensorMap &tv,
                         const pa_plan_t &pl, cudaStream_t stream) {
  static std::atomic<bool> set[kMaxLaunchDevices];
  auto kern = decode_quant_kernel<HD, T>;
  const cudaError_t e = allow_smem(kern, kMaxDecodeSmem, set);
  if (e != cudaSuccess) return e;
  return launch_early(kern, dim3(pl.ctas), pl.warps_per_cta * 32, static_cast<int>(pl.smem_bytes),
                      stream, a, tk, tv);
}

}  // namespace

}  // namespace pa

extern "C" pa_status_t pa_quant_workspace_size(const pa_problem_t *problem,
                                               const pa_options_t *options, size_t *bytes) {
  using namespace pa;
  if (!bytes) return PA_ERR_INVALID_ARG;
  pa_plan_t pl;
  pa_status_t st = quant_plan(problem, options, 1, nullptr, &pl);  // shapes and options refused
  if (st != PA_OK) return st;
  int smem = 0;
  st = current_device_smem(&smem);
  if (st != PA_OK) return st;
  st = quant_plan(problem, options, device_sm_count(), nullptr, &pl);
  if (st == PA_OK) *bytes = problem->batch == 0 ? 0 : static_cast<size_t>(pl.workspace_bytes);
  return st;
}

extern "C" pa_status_t pa_decode_quant(const pa_problem_t *problem, const pa_score_t *score,
                                       const void *query, const pa_quant_cache_t *cache,
                                       const int32_t *block_tables, const int32_t *context_lengths,
                                       float scale, void *out, const pa_options_t *options,
                                       void *workspace, size_t workspace_bytes, void *stream) {
  using namespace pa;
  pa_status_t st = check_problem_public(problem);
  if (st != PA_OK) return st;
  st = check_quant_cache(cache);
  if (st != PA_OK) return st;
  st = validate_call(problem, options, query, cache->key, cache->value, block_tables,
                     context_lengths, scale, static_cast<const float *>(out));
  if (st != PA_OK) return st;
  QuantDecodeArgs a;
  std::memset(&a, 0, sizeof(a));
  st = resolve_score(score, scale, &a.s);
  if (st != PA_OK) return st;
  pa_plan_t pl;
  st = quant_plan(problem, options, 1, &a.s, &pl);  // shapes and options that are refused
  if (st != PA_OK) return st;
  if (problem->batch == 0) return PA_OK;
  int smem_optin = 0;
  st = current_device_smem(&smem_optin);
  if (st != PA_OK) return st;
  st = quant_plan(problem, options, device_sm_count(), &a.s, &pl);
  if (st != PA_OK) return st;
  if (pl.workspace_bytes > 0) {
    if (!workspace || workspace_bytes < static_cast<size_t>(pl.workspace_bytes))
      return PA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return PA_ERR_MISALIGNED;
  }

  alignas(64) CUtensorMap tk, tv;
  const int hd = problem->head_dim;
  const int rows = std::min(problem->page_size, pl.tile_tokens);
  const int blocks = rows == pl.tile_tokens && hd > 128 ? hd / 128 : 1;
  st = encode_code_map(&tk, cache->key, problem, rows, blocks);
  if (st != PA_OK) return st;
  st = encode_code_map(&tv, cache->value, problem, rows, blocks);
  if (st != PA_OK) return st;
  st = fill_scored_args(problem, pl, query, block_tables, context_lengths, scale, out, workspace,
                        &a);
  if (st != PA_OK) return st;
  KernelArgs &k = a.k;
  k.warp_smem = pl.stages * 2 * pl.tile_tokens * hd;
  if (options && (options->test_flags & PA_TEST_EXPIRE_WAITS)) k.tx_extra = 16;
  a.k_scale = cache->key_scale;
  a.v_scale = cache->value_scale;

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (hd) {
    case 64: e = launch_quant<64, 64>(a, tk, tv, pl, s); break;
    case 128: e = launch_quant<128, 32>(a, tk, tv, pl, s); break;
    default: e = launch_quant<256, 16>(a, tk, tv, pl, s); break;
  }
  if (e == cudaSuccess && k.mode == MODE_BALANCED)
    e = launch_join_states(a, pl.units, k.nh_unit, combine_warps_per_pair(pl.units, pl.workers),
                           pl.tile_tokens, s);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
