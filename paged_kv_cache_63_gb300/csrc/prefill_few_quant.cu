// prefill_few_quant.cu -- few new tokens over a quantised cache (pa_prefill_quant), as drafted tokens are
// checked or a short prompt goes on.
//
// Mathematics as in prefill2_scored_kernel.cuh. There a work item is 128 rows (new tokens by the query
// heads of a K/V head) whose softmax walks through the keys 64 at a time, 0.55 us each; of 7 tokens by 4
// heads a hundred rows are padding, and 8 sequences with 8 K/V heads are work for 64 of 152
// multiprocessors. Here a CTA takes eight rows of a sequence and K/V head, its twelve warps a twelfth of
// the keys each, by the decode step's walk (code_walk.cuh) with a mask for each row, and their states are
// joined in shared memory; where such CTAs leave multiprocessors idle, up to eight of them form a cluster
// that shares the keys and joins through its shared memories. K and V are read once for each eight rows,
// from L2 after the first (CTAs of the same keys run side by side: loads marked to stay in L2, as in
// prefill2_scored_kernel.cuh, took 959.6 us against 959.7 for 64 new tokens of 100000, 32/8 heads of
// 128, and 23.4 against 23.0 for the eight sequences below). Bound: the walk's chain of loads and products, about 1 us a tile and warp. Eight
// sequences of up to 4096 tokens, 2 to 7 of them new, 32/8 heads of 128: 23.0 us against 42.4; one of
// 100000, one new token: 68 against 1200.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cstring>

#include "code_walk.cuh"
#include "prefill_few_quant.h"

namespace pa {

struct FewArgs : QuantDecodeArgs {
  const int32_t *qs;
  long long total;
  int parts;  // CTAs of a cluster, which share the keys of its eight rows
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// A float of shared memory of the cluster's block `rank`, at the place that `p` has in this block's.
__device__ __forceinline__ float load_of_block(const float *p, int rank) {
  float x;
  asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
               "ld.shared::cluster.f32 %0, [a];\n\t}"
               : "=f"(x)
               : "r"(smem_addr(p)), "r"(rank)
               : "memory");
  return x;
}

// What the lane's two rows (2 (l % 4) and the next) see; lo_max and end_min are over all eight rows.
struct FewRows {
  int lo[2], end[2], pos[2];
  int lo_max, end_min;
  __device__ __forceinline__ bool masks(int from, int to) const {
    return from < lo_max || end_min < to;
  }
  __device__ __forceinline__ bool sees(int j, int t) const { return t >= lo[j] && t < end[j]; }
  __device__ __forceinline__ float distance(int j, int t) const {
    return -static_cast<float>(abs(pos[j] - t));
  }
};

template <int HD, int T>
__global__ void __launch_bounds__(kQuantWarps * 32, 1)
    prefill_few_quant_kernel(const __grid_constant__ FewArgs fa, const __grid_constant__ CUtensorMap tk,
                             const __grid_constant__ CUtensorMap tv) {
  using G = CodeGeom<HD, T>;
  constexpr int S = kQuantStages, kRow = HD + 4;  // floats of a joined row: no two lanes on a bank
  static_assert(kMaxHeads * kRow * 4 <= S * G::kStageBytes, "a warp's state fits its ring");
  const KernelArgs &a = fa.k;
  extern __shared__ uint8_t dsm[];
  __shared__ __align__(8) uint64_t bars[kQuantWarps * S];
  __shared__ float part[kQuantWarps][kMaxHeads][2];
  __shared__ float joined[kMaxHeads * HD], joined_ml[kMaxHeads][2];  // of a cluster's block
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kv = blockIdx.x / fa.parts, b = blockIdx.z;
  const int rank = blockIdx.x - kv * fa.parts;  // in the cluster
  const uint32_t base = (smem_addr(dsm) + kSmemAlign - 1) & ~static_cast<uint32_t>(kSmemAlign - 1);
  const uint32_t ring = base + warp * S * G::kStageBytes;
  const uint32_t scales = base + kQuantWarps * S * G::kStageBytes + warp * S * G::kScaleBytes;
  const uint32_t bar0 = smem_addr(&bars[warp * S]);
  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(bar0 + 8 * s, 33);
    fence_barrier_init();
    prefetch_tensormap(&tk);
    prefetch_tensormap(&tv);
  }
  __syncwarp();
  wait_for_stream();

  // ---- the CTA's rows: n tokens by g heads, eight from row0 on (the last row stands in for those past it)
  const int q0 = __ldg(fa.qs + b), q1 = __ldg(fa.qs + b + 1), ctx = __ldg(a.ctx + b);
  const int n = q1 - q0;
  unsigned bad = 0;
  if (ctx < 0 || static_cast<long long>(ctx) > static_cast<long long>(a.maxp) << a.ps_shift)
    bad = PA_DEVERR_CONTEXT;
  else if (q0 < 0 || n < 0 || q1 > fa.total || n > ctx)
    bad = PA_DEVERR_QUERY_START;
  if (bad) {
    if (threadIdx.x == 0) atomicOr(a.err, bad);
    return;
  }
  const int row0 = blockIdx.y * kMaxHeads;
  // (n may be more than the call promised, which is not computed)
  const long long all = static_cast<long long>(n) * a.g;
  if (row0 >= all) return;
  const int rows = static_cast<int>(min(all, static_cast<long long>(INT_MAX)));
  const int prefix = fa.s.prefix ? min(__ldg(fa.s.prefix + b), ctx) : 0;
  auto row_of = [&](int i) { return min(row0 + i, rows - 1); };
  FewRows rs;
  CodeState<HD> st = {};
  SpanCursor c;
  {
    const int i = lane >> 2, r = row_of(i);  // queries: the row that the lane gives elements of
    const uint2 *src = reinterpret_cast<const uint2 *>(
        a.q + (static_cast<long long>(q0 + r / a.g) * a.qh + kv * a.g + r % a.g) * HD);
#pragma unroll
    for (int k = 0; k < HD / 16; ++k) {
      const uint2 q = __ldg(src + k * 4 + (lane & 3));
      st.q[k][0] = q.x;
      st.q[k][1] = q.y;
    }
  }
  int lo_min = INT_MAX, end_max = 0;
  rs.lo_max = 0;
  rs.end_min = INT_MAX;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = row_of(2 * (lane & 3) + j), pos = ctx - n + r / a.g;
    rs.pos[j] = pos;
    rs.lo[j] = fa.s.window > 0 && pos >= fa.s.window ? pos - fa.s.window + 1 : 0;
    rs.end[j] = pos < prefix ? prefix : pos + 1;
    st.slope2[j] = fa.s.slopes ? __ldg(fa.s.slopes + kv * a.g + r % a.g) * kLog2e : 0.f;
    st.m[j] = -INFINITY;
    lo_min = min(lo_min, rs.lo[j]);
    end_max = max(end_max, rs.end[j]);
    rs.lo_max = max(rs.lo_max, rs.lo[j]);
    rs.end_min = min(rs.end_min, rs.end[j]);
  }
  // a token between the first and the last that some row sees is seen by some row: each sees its own
  c.sp.lo = __reduce_min_sync(0xffffffffu, lo_min);
  c.sp.end = __reduce_max_sync(0xffffffffu, end_max);
  rs.lo_max = __reduce_max_sync(0xffffffffu, rs.lo_max);
  rs.end_min = __reduce_min_sync(0xffffffffu, rs.end_min);

  // ---- the warp's tiles
  const long long tiles = span_tiles(c.sp, T);
  const int walks = fa.parts * kQuantWarps, walk = rank * kQuantWarps + warp;
  const int from = static_cast<int>(tiles * walk / walks);
  c.b = b;
  c.us = 0;
  c.ug0 = 0;
  c.tok = span_start(c.sp, T) + from * T;
  c.left = static_cast<int>(tiles * (walk + 1) / walks) - from;
  SpanCursor ic = c;
  BtWindow win;
  win.b = -1;
  win.base = 0;
  win.cur = win.nxt = -1;
  CodeLane<HD, T> lane_addr;
  lane_addr.init();
  const uint64_t pol = l2_evict_first_policy();
  int cs = 0, is = 0, flying = 0;
  uint32_t cphase = 0, extra = a.tx_extra;
  while (c.left > 0) {
#pragma unroll 1
    while (flying < S && ic.left > 0) {
      issue_code_tile<HD, T>(fa, &tk, &tv, ic, kv, win, ring + is * G::kStageBytes,
                             scales + is * G::kScaleBytes, bar0 + 8 * is, pol, extra);
      extra = 0;
      is = is + 1 == S ? 0 : is + 1;
      ++flying;
      ic.tok += T;
      --ic.left;
    }
    if (!mbar_wait(bar0 + 8 * cs, cphase, a.err)) break;
    code_tile<HD, T>(st, lane_addr, ring + cs * G::kStageBytes, scales + cs * G::kScaleBytes, c, fa,
                     rs);
    fence_proxy_async();
    __syncwarp();
    if (++cs == S) {
      cs = 0;
      cphase ^= 1u;
    }
    --flying;
    c.tok += T;
    --c.left;
  }
  // after a wait that gave up: the copies in flight land before their memory is used again
  for (; flying > 0; --flying) {
    mbar_wait(bar0 + 8 * cs, cphase, a.err);
    if (++cs == S) {
      cs = 0;
      cphase ^= 1u;
    }
  }

  // ---- join: each warp leaves its state in its ring
  float sum[2] = {st.lsum[0], st.lsum[1]};
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
    sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], o);
  }
  float *states = reinterpret_cast<float *>(dsm + (base - smem_addr(dsm)));
  constexpr int kState = S * G::kStageBytes / 4;  // floats from warp to warp
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = 2 * (lane & 3) + j, element = lane >> 2;
    if (element == 0) {
      part[warp][i][0] = st.m[j];
      part[warp][i][1] = sum[j];
    }
    float *dst = states + warp * kState + i * kRow + element;
#pragma unroll
    for (int k = 0; k < HD / 16; ++k) {
      dst[k * 16] = st.o[k][j];
      dst[k * 16 + 8] = st.o[k][2 + j];
    }
  }
  __syncthreads();
  const int live = min(kMaxHeads, rows - row0);
  constexpr int kThreads = kQuantWarps * 32;
  auto store = [&](int at, float o, float l) {
    const int r = row0 + at / HD;
    store_out1(fa.s, fa.out,
               (static_cast<long long>(q0 + r / a.g) * a.qh + kv * a.g + r % a.g) * HD + at % HD,
               l > 0.f ? o / l : 0.f);
  };
  for (int at = threadIdx.x; at < live * HD; at += kThreads) {
    const int i = at / HD, element = at % HD;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kQuantWarps; ++w) m = fmaxf(m, part[w][i][0]);
    float l = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < kQuantWarps; ++w) {
      // a warp without tiles, or whose tokens the row does not see: 0
      const float mw = part[w][i][0], f = mw == -INFINITY ? 0.f : fast_exp2(mw - m);
      l = fmaf(part[w][i][1], f, l);
      o = fmaf(states[w * kState + i * kRow + element], f, o);
    }
    if (fa.parts == 1) {
      store(at, o, l);
    } else {
      joined[at] = o;
      if (element == 0) {
        joined_ml[i][0] = m;
        joined_ml[i][1] = l;
      }
    }
  }
  if (fa.parts == 1) return;
  cluster_sync();  // every block of the cluster gets here: they have the same rows
  for (int at = threadIdx.x + rank * kThreads; at < live * HD; at += fa.parts * kThreads) {
    const float *ml = joined_ml[at / HD];
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int p = 0; p < fa.parts; ++p) m = fmaxf(m, load_of_block(ml, p));
    for (int p = 0; p < fa.parts; ++p) {
      const float mp = load_of_block(ml, p), f = mp == -INFINITY ? 0.f : fast_exp2(mp - m);
      l = fmaf(load_of_block(ml + 1, p), f, l);
      o = fmaf(load_of_block(joined + at, p), f, o);
    }
    store(at, o, l);
  }
  cluster_sync();  // no block leaves while others read its memory
}

namespace {

template <int HD, int T>
cudaError_t launch_few(const FewArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, dim3 grid,
                       cudaStream_t stream) {
  static std::atomic<bool> set[kMaxLaunchDevices];
  auto kern = prefill_few_quant_kernel<HD, T>;
  const int smem = quant_smem(HD, kQuantWarps, kQuantStages);
  const cudaError_t e = allow_smem(kern, smem, set);
  if (e != cudaSuccess) return e;
  return launch_early_in_clusters(static_cast<unsigned>(a.parts), kern, grid, kQuantWarps * 32, smem,
                                  stream, a, tk, tv);
}

}  // namespace

// A CTA here takes about half the time of a work item of 128 rows there, so this kernel is taken while
// its CTAs are at most twice the larger of the other's items and the multiprocessors. Measured here |
// there (no clusters), us, on contexts of 4000, 32/8 heads of 128: one sequence, 1 to 32 new tokens 24 |
// 54 to 59, 64 of them 47 | 70; eight sequences, 8 tokens 47 | 58, 16 (past the rule) 90 | 58; 64
// sequences of up to 600 tokens, 4 new 44 | 47, 8 (past it) 80 | 47; head_dim 256, 24/4 heads, two
// sequences, 42 new 90 | 91. On contexts of 100 the two are within 3 us. First tokens may leave tokens
// that no row sees between others, which only the other kernels clear.
bool few_rows(const pa_problem_t *p, const ScoreArgs &s, int max_query_len) {
  if (s.first) return false;
  const long long rows = static_cast<long long>(max_query_len) * (p->query_heads / p->kv_heads);
  const long long heads = static_cast<long long>(p->kv_heads) * p->batch;
  const long long ctas = (rows + kMaxHeads - 1) / kMaxHeads * heads;
  const long long items = (rows + 127) / 128 * heads;
  return ctas <= 2 * std::max<long long>(device_sm_count(), items);
}

pa_status_t launch_few_quant(const pa_problem_t *problem, const PrefillQuantArgs &p,
                             const void *query, int max_query_len, const pa_quant_cache_t *cache,
                             cudaStream_t stream) {
  FewArgs a;
  std::memset(&a, 0, sizeof(a));
  a.s = p.s;
  a.out = p.out16;
  a.k_scale = p.k_scale;
  a.v_scale = p.v_scale;
  a.qs = p.qs;
  a.total = p.total;
  KernelArgs &k = a.k;
  k.q = static_cast<const uint16_t *>(query);
  k.bt = p.bt;
  k.ctx = p.ctx;
  k.err = p.err;
  k.batch = p.batch;
  k.qh = p.qh;
  k.kvh = p.kvh;
  k.hd = problem->head_dim;
  k.ps = p.ps;
  k.ps_shift = p.ps_shift;
  k.maxp = p.maxp;
  k.num_pages = p.num_pages;
  k.layout = p.layout;
  k.g = p.g;
  k.scale_log2 = p.scale_log2;
  k.tx_extra = p.expire ? 16 : 0;

  alignas(64) CUtensorMap tk, tv;
  const int hd = problem->head_dim, tile = quant_tile(hd);
  const int rows = problem->page_size < tile ? problem->page_size : tile;
  const int blocks = rows == tile && hd > 128 ? hd / 128 : 1;
  pa_status_t st = encode_code_map(&tk, cache->key, problem, rows, blocks);
  if (st != PA_OK) return st;
  st = encode_code_map(&tv, cache->value, problem, rows, blocks);
  if (st != PA_OK) return st;
  const long long rows_most = static_cast<long long>(max_query_len) * p.g;
  const long long groups = (rows_most + kMaxHeads - 1) / kMaxHeads;
  const long long ctas = groups * p.kvh * p.batch;
  // Multiprocessors left idle share the keys, where the tables hold 32 tiles and more: one sequence of
  // 4000 tokens, 32/8 heads of 128, 1, 2, 4, 8 blocks to a cluster: 23.4, 16.1, 10.9, 9.1 us; of 1000:
  // 8.8, 8.6, 7.0, 6.9; of 300 (not shared) 5.5, 7.1, 6.9, 6.9. Clusters of 8 only on half of the
  // multiprocessors: 16 of them do not run at once (head_dim 256, four sequences of 4000: 22 against 17).
  const int sms = device_sm_count();
  const long long most = static_cast<long long>(p.maxp) << p.ps_shift;
  a.parts = 1;
  if (most >= 32 * quant_tile(problem->head_dim))
    while (a.parts < 8 && (a.parts < 4 ? 2 : 4) * a.parts * ctas <= sms) a.parts *= 2;
  const dim3 grid(static_cast<unsigned>(p.kvh * a.parts), static_cast<unsigned>(groups), p.batch);
  cudaError_t e;
  switch (hd) {
    case 64: e = launch_few<64, 64>(a, tk, tv, grid, stream); break;
    case 128: e = launch_few<128, 32>(a, tk, tv, grid, stream); break;
    default: e = launch_few<256, 16>(a, tk, tv, grid, stream); break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
