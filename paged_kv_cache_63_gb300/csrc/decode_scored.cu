// decode_scored.cu -- one decode step with a score rule (pa_decode_scored): scores capped by a
// tanh, a bias by distance, a sliding window or a first visible token per sequence.
//
// Mathematics, for query head h of sequence b at position p = context - 1:
//   s_t = scale q . K_t;  s_t = cap tanh(s_t / cap);  s_t -= slope_h (p - t)
//   out = sum_t softmax(s)_t V_t over max(0, p - window + 1, first_b) <= t <= p
// Bound: HBM -- the seen K and V are read once, 2 g flops a byte (g query heads a K/V head).
//
// The work is laid out as in decode_kernel.cuh: a warp is a worker with a private ring of K/V
// tiles loaded by TMA, warps of a CTA take neighbouring units over the same tokens, and the
// concatenated tiles of all units are cut into equal ranges, one per worker, whose (reference
// maximum, sum, unnormalised output) states are joined by log-sum-exp. What differs:
//  * A unit's tiles are those of its seen tokens only: tokens before the window or the document
//    cost nothing, and their pages are never read.
//  * The joining always runs in a kernel of its own (a programmatic dependent). It needs no
//    flags and no numbers of calls, so a captured call replays as it stands.
//  * The probabilities keep 22 bits: the m16n8k16 tile has 16 rows for 8 heads, so rows 0..7
//    take a probability rounded to fp16 and rows 8..15 the remainder, at no further tensor
//    instruction; tile results are added to the output in fp32 registers, so a long context
//    does not lose bits to the tensor cores' accumulator either.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "row_maps.h"
#include "span_split.cuh"

namespace pa {

// Issue the TMA loads of the tile at cursor c into a stage (warp-uniform). Pieces (min(page
// size, T) rows) that hold no seen token are not loaded. A tile of one piece is one load each
// for K and V; the column blocks of smaller pieces lie apart in the stage and are loaded alone.
template <int HD, int T>
__device__ __forceinline__ void issue_span_tile(const ScoredArgs &sa, const CUtensorMap *tk,
                                                const CUtensorMap *tv, const SpanCursor &c, int kv,
                                                BtWindow &w, uint32_t stage, uint32_t bar,
                                                uint64_t pol, uint32_t extra_tx) {
  const KernelArgs &a = sa.k;
  constexpr int kMaxPieces = T / 8;
  const int R = a.ps < T ? a.ps : T;
  const int npages = (c.sp.end + a.ps - 1) >> a.ps_shift;
  const bool hm = a.layout == PA_LAYOUT_HEAD_MAJOR;
  auto place = [&](int tok, int &row, int &head) {  // false: the page id is outside the pool
    const int page = bt_page(a, w, c.b, tok >> a.ps_shift, npages);
    const int slot = tok & (a.ps - 1);
    row = hm ? slot : (page << a.ps_shift) + slot;
    head = hm ? page * a.kvh + kv : kv;
    if (page >= 0 && page < a.num_pages) return true;
    if ((threadIdx.x & 31) == 0) atomicOr(a.err, PA_DEVERR_PAGE_ID);
    return false;
  };
  if (R == T) {
    int row, head;
    const bool good = place(c.tok, row, head);
    expect_bytes_warp(bar, (good ? Geom<HD, T>::kStageBytes : 0u) + extra_tx);
    if (good) {
      tma_rows_warp(stage, tk, bar, row, head, 0, pol);
      tma_rows_warp(stage + Geom<HD, T>::kHalfBytes, tv, bar, row, head, 0, pol);
    }
    return;
  }
  int row[kMaxPieces], head[kMaxPieces];  // row < 0 marks a piece not loaded
  uint32_t bytes = 0;
#pragma unroll
  for (int p = 0; p < kMaxPieces; ++p) {
    const int tok = c.tok + p * R;
    head[p] = 0;
    if (p * R < T && tok < c.sp.end && tok + R > c.sp.lo && place(tok, row[p], head[p]))
      bytes += static_cast<uint32_t>(R * HD * 4);
    else
      row[p] = -1;
  }
  expect_bytes_warp(bar, bytes + extra_tx);
#pragma unroll
  for (int p = 0; p < kMaxPieces; ++p) {
    if (row[p] < 0) continue;
#pragma unroll
    for (int blk = 0; blk < HD / 64; ++blk) {
      const uint32_t dst = stage + blk * (T * 128) + p * R * 128;
      tma_rows_warp(dst, tk, bar, row[p], head[p], blk, pol);
      tma_rows_warp(dst + Geom<HD, T>::kHalfBytes, tv, bar, row[p], head[p], blk, pol);
    }
  }
}

// Running state of a unit; a lane's row (head) is lane / 4.
template <int HD>
struct SpanState {
  float m, lsum;
  float slope2;              // the head's slope * log2 e
  float o[HD / 8][2];        // O[lane / 4][8 nt + 2 (lane % 4) + {0, 1}]
  uint32_t qa[HD / 16][2];   // A fragments of q
};

template <int HD>
__device__ __forceinline__ void span_begin(SpanState<HD> &st, const ScoredArgs &a, int b, int h0,
                                           int nh) {
  const int lane = threadIdx.x & 31;
  const int h = lane >> 2;
  const int c = (lane & 3) * 2;
  const uint32_t *src = reinterpret_cast<const uint32_t *>(
      a.k.q + (static_cast<long long>(b) * a.k.qh + h0 + h) * HD);
#pragma unroll
  for (int ks = 0; ks < HD / 16; ++ks) {
    st.qa[ks][0] = h < nh ? __ldg(src + (ks * 16 + c) / 2) : 0u;
    st.qa[ks][1] = h < nh ? __ldg(src + (ks * 16 + 8 + c) / 2) : 0u;
  }
  st.slope2 = a.s.slopes && h < nh ? __ldg(a.s.slopes + h0 + h) * kLog2e : 0.f;
  st.m = -INFINITY;
  st.lsum = 0.f;
#pragma unroll
  for (int nt = 0; nt < HD / 8; ++nt) st.o[nt][0] = st.o[nt][1] = 0.f;
}

// Zero V rows [from, to) of a stage: a zero probability must not meet a non-finite value in a
// row that holds no seen token.
template <int HD, int T>
__device__ __forceinline__ void zero_rows(uint32_t stv, int from, int to) {
  const int lane = threadIdx.x & 31;
  const int n = (to - from) * (HD / 8);
  for (int i = lane; i < n; i += 32) {
    const int row = from + i / (HD / 8);
    const int chunk = i % (HD / 8);
    sts128(stv + (chunk >> 3) * (T * 128) + row * 128 + (chunk & 7) * 16, make_uint4(0, 0, 0, 0));
  }
}

template <int HD, int T>
__device__ __forceinline__ void span_tile(SpanState<HD> &st, const MmaLane<HD, T> &ln,
                                          uint32_t stage, const SpanCursor &c,
                                          const ScoredArgs &a) {
  constexpr int NCH = T / 16;
  const int lane = threadIdx.x & 31;
  const int tok0 = c.tok;
  uint32_t kb[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) kb[j] = stage + ln.k[j];

  // S[h][t]: two n8 tiles per 16-token chunk, each in two chains (even and odd k steps), which
  // halves the dependent chain and the accumulator's rounding
  float x[NCH][2][2];
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch) {
    float s[2][2][2] = {};
#pragma unroll
    for (int ks = 0; ks < HD / 16; ++ks) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4(kb[ks & 3] + (ks >> 2) * (T * 128) + ch * 2048, b0, b1, b2, b3);
      mma_rows8(s[ks & 1][0][0], s[ks & 1][0][1], st.qa[ks][0], st.qa[ks][1], b0, b1);
      mma_rows8(s[ks & 1][1][0], s[ks & 1][1][1], st.qa[ks][0], st.qa[ks][1], b2, b3);
    }
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) x[ch][nt][j] = s[0][nt][j] + s[1][nt][j];
  }

  // the score rule, in base-2 units; the row's scores live in lanes lane & ~3 .. lane | 3
  const bool partial = tok0 < c.sp.lo || c.sp.end - tok0 < T;
  const float away0 = static_cast<float>(tok0 + 2 * (lane & 3) - (c.sp.end - 1));
  float mt = -INFINITY;
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float y = x[ch][nt][j];
        y = a.s.cap_in != 0.f ? a.s.cap_out * tanhf(y * a.s.cap_in) : y * a.k.scale_log2;
        if (a.s.slopes) y = fmaf(st.slope2, away0 + static_cast<float>(ch * 16 + nt * 8 + j), y);
        if (partial) {
          const int tok = tok0 + ch * 16 + nt * 8 + 2 * (lane & 3) + j;
          y = tok >= c.sp.lo && tok < c.sp.end ? y : -INFINITY;
        }
        x[ch][nt][j] = y;
        mt = fmaxf(mt, y);
      }
  mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
  mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
  if (__any_sync(0xffffffffu, mt > st.m + (kLift + kRescaleSlack))) {
    const float mn = fmaxf(st.m, mt - kLift);
    const float alpha = mn == -INFINITY ? 1.f : fast_exp2(st.m - mn);
    st.m = mn;
    st.lsum *= alpha;
#pragma unroll
    for (int nt = 0; nt < HD / 8; ++nt) {
      st.o[nt][0] *= alpha;
      st.o[nt][1] *= alpha;
    }
  }
  const float m = st.m == -INFINITY ? 0.f : st.m;  // no score above -inf yet
  float psum = 0.f;
  uint32_t hi[NCH][2], lo[NCH][2];
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const float p0 = fast_exp2(x[ch][nt][0] - m);
      const float p1 = fast_exp2(x[ch][nt][1] - m);
      hi[ch][nt] = pack_half2(p0, p1);
      const float2 r = half2_bits_to_float2(hi[ch][nt]);
      lo[ch][nt] = pack_half2(p0 - r.x, p1 - r.y);
      psum += p0 + p1;
    }
  st.lsum += psum;

  if (partial) {
    const uint32_t stv = stage + Geom<HD, T>::kHalfBytes;
    if (tok0 < c.sp.lo) zero_rows<HD, T>(stv, 0, c.sp.lo - tok0);
    if (c.sp.end - tok0 < T) zero_rows<HD, T>(stv, c.sp.end - tok0, T);
    __syncwarp();
  }
#pragma unroll
  for (int dt = 0; dt < HD / 16; ++dt) {
    float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ch = 0; ch < NCH; ++ch) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4_trans(stage + ln.v[dt & 3] + (dt >> 2) * (T * 128) + ch * 2048, b0, b1, b2, b3);
      mma_rows16(d0, hi[ch][0], lo[ch][0], hi[ch][1], lo[ch][1], b0, b1);
      mma_rows16(d1, hi[ch][0], lo[ch][0], hi[ch][1], lo[ch][1], b2, b3);
    }
    st.o[2 * dt][0] += d0[0] + d0[2];
    st.o[2 * dt][1] += d0[1] + d0[3];
    st.o[2 * dt + 1][0] += d1[0] + d1[2];
    st.o[2 * dt + 1][1] += d1[1] + d1[3];
  }
}

// Eight warps leave a thread 255 registers: enough at head_dim 64 and 128 (156 and 203); at 256,
// where the output alone takes 64 and the query 32, 112 bytes spill, which the stream hides (0.97
// of the copy bandwidth).
template <int HD, int T>
__global__ void __launch_bounds__(kMaxWarpsPerCta * 32, 1)
    decode_scored_kernel(const __grid_constant__ ScoredArgs sa,
                         const __grid_constant__ CUtensorMap tk,
                         const __grid_constant__ CUtensorMap tv) {
  using G = Geom<HD, T>;
  const KernelArgs &a = sa.k;
  extern __shared__ uint8_t dsm[];
  __shared__ __align__(8) uint64_t bars[kMaxWarpsPerCta * kMaxStages];
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int worker = (blockIdx.x * (blockDim.x >> 5) + warp) / a.group;
  const int member = warp % a.group;
  const int S = a.stages;
  const uint32_t wbase =
      ((smem_addr(dsm) + kSmemAlign - 1) & ~static_cast<uint32_t>(kSmemAlign - 1)) +
      warp * a.warp_smem;
  const uint32_t bar0 = smem_addr(&bars[warp * kMaxStages]);

  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(bar0 + 8 * s, 1);
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
    for (long long base = worker; base < a.batch; base += 32ll * a.workers) {
      const long long bl = base + static_cast<long long>(lane) * a.workers;
      unsigned empty = __ballot_sync(
          0xffffffffu, bl < a.batch && span_tiles(load_span(sa, static_cast<int>(bl)), T) == 0);
      while (empty) {
        const int j = __ffs(empty) - 1;
        empty &= empty - 1;
        const int b = static_cast<int>(base + static_cast<long long>(j) * a.workers);
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
  // ring positions: the stage and phase parity of the next tile to consume, the stage of the
  // next one to issue, and the tiles in flight; divisions stay out of the loop (with them a
  // tile's bookkeeping took 500 cycles more)
  int cs = 0, is = 0, flying = 0;
  uint32_t cphase = 0, extra = a.tx_extra;
  int ius = ic.us, ikv = (ic.us * a.group + member) / a.sub;  // K/V head of the cursor's unit
  auto issue = [&]() {
    if (ic.us != ius) {
      ius = ic.us;
      ikv = (ic.us * a.group + member) / a.sub;
    }
    issue_span_tile<HD, T>(sa, &tk, &tv, ic, ikv, win, wbase + is * G::kStageBytes, bar0 + 8 * is,
                           pol, extra);
    extra = 0;
    is = is + 1 == S ? 0 : is + 1;
    ++flying;
    advance(sa, ic, T);
  };
  while (flying < S - 1 && ic.left > 0) issue();

  SpanState<HD> st = {};
  MmaLane<HD, T> lane_addr;
  lane_addr.init();
  UnitInfo cur;
  cur.b = -1;
  cur.us = -1;
  cur.h0 = cur.nh = 0;
  long long cur_ug0 = 0;
  int cur_tiles = 0;
  bool aborted = false;

  auto finish_unit = [&]() {
    float l = st.lsum;
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const int h = lane >> 2;
    bool whole = true;
    const long long unit = static_cast<long long>(cur.b) * a.ups + cur.us;
    if (a.mode == MODE_BALANCED)
      whole = worker_of(cur_ug0, total, nworkers) ==
              worker_of(cur_ug0 + cur_tiles - 1, total, nworkers);
    if (h >= cur.nh) return;
    if (whole) {
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const long long base =
          (static_cast<long long>(cur.b) * a.qh + cur.h0 + h) * HD + 2 * (lane & 3);
#pragma unroll
      for (int nt = 0; nt < HD / 8; ++nt)
        store_out2(sa.s, sa.out, base + nt * 8, st.o[nt][0] * inv, st.o[nt][1] * inv);
      return;
    }
    // partial state relative to the row's reference, for the joining kernel
    const long long slot = slot_of(unit, worker, a.group) * kMaxHeads + h;
    if ((lane & 3) == 0)
      *reinterpret_cast<float2 *>(a.ws_ml + slot * 2) = make_float2(st.m, l);
    float *dst = a.ws_acc + slot * HD + 2 * (lane & 3);
#pragma unroll
    for (int nt = 0; nt < HD / 8; ++nt)
      *reinterpret_cast<float2 *>(dst + nt * 8) = make_float2(st.o[nt][0], st.o[nt][1]);
  };

  // ---- main loop: refill the slot freed last iteration, wait for the next tile, compute
  while (c.left > 0) {
    if (c.b != cur.b || c.us * a.group + member != cur.us) {
      if (cur.b >= 0) finish_unit();
      cur = unit_info(a, c.b, c.us * a.group + member);
      cur_ug0 = c.ug0;
      cur_tiles = span_tiles(c.sp, T);
      span_begin<HD>(st, sa, cur.b, cur.h0, cur.nh);
    }
    if (ic.left > 0) issue();
    if (!mbar_wait(bar0 + 8 * cs, cphase, a.err)) {
      aborted = true;
      break;
    }
    span_tile<HD, T>(st, lane_addr, wbase + cs * G::kStageBytes, c, sa);
    fence_proxy_async();
    __syncwarp();
    if (++cs == S) {
      cs = 0;
      cphase ^= 1u;
    }
    --flying;
    advance(sa, c, T);
  }
  // the joining kernel may come up now (it waits for this grid before it reads any state)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (aborted) {
    // let the copies still in flight land before the shared memory is given up
    for (; flying > 0; --flying) {
      mbar_wait(bar0 + 8 * cs, cphase, a.err);
      if (++cs == S) {
        cs = 0;
        cphase ^= 1u;
      }
    }
    return;
  }
  finish_unit();
}

// The unit that is cut where worker w (not the first) starts and at no worker before it: its
// sequence, group unit and number of contributors, w - 1 the first of them (n = 0: there is none).
struct Cut {
  int b, us, n;
};

// Warp-collective.
__device__ inline Cut cut_at(const ScoredArgs &sa, int w, int T) {
  SpanCursor c = {};
  long long total, nworkers;
  Cut cut = {0, 0, 0};
  if (span_balanced_start(sa, w, T, c, total, nworkers) &&
      c.ug0 < worker_start(w, total, nworkers) && worker_of(c.ug0, total, nworkers) == w - 1) {
    cut.b = c.b;
    cut.us = c.us;
    cut.n = static_cast<int>(worker_of(c.ug0 + span_tiles(c.sp, T) - 1, total, nworkers) - w + 2);
  }
  return cut;
}

// Joins the states of units that several workers share: out = sum_k 2^(m_k - M) acc_k /
// sum_k 2^(m_k - M) l_k, contributors in their order. W warps take one (unit, head) pair, a
// CTA of eight warps 8 / W pairs. Its CTAs come up when the decode kernel's have finished their
// tiles, which had waited for everything before them in the stream: so a warp redoes the split
// from the inputs before its own wait, and after it the pair costs about one memory round trip.
// kCuts: with more units than workers the CTAs go through the workers' starts, where alone a unit
// can be cut, instead of all units, `chunks` CTAs to a start: a pass over the batch's lengths for
// each unit grows with the square of the batch (the call on sequences of 64 tokens, 64/8 heads of
// 128, that is 1216 workers: 160 of them 24.9 us by units and 22.6 by starts, 512 80 and 42, 4096
// 2502 and 315). Registers: up to 64 the CTAs come up beside the decode kernel's last ones, 2 us
// earlier; at head_dim 256 that would spill (four contexts of 100000: 244.4 against 243.7 us).
template <int HD, int W, bool kCuts>
__global__ void __launch_bounds__(256, HD == 256 && !kCuts ? 3 : 4)
    join_scored_kernel(const __grid_constant__ ScoredArgs sa, int heads, long long pairs, int chunks,
                       int T) {
  constexpr int DPL = HD / 32;
  constexpr int P = 8 / W;
  constexpr int KB = HD >= 256 ? 4 : 8;
  const KernelArgs &a = sa.k;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int sub = warp % W;
  long long unit = 0, c0 = 0;
  int h = 0, n = 0;
  UnitInfo u = {0, 0, 0, 0};
  if constexpr (kCuts) {
    __shared__ Cut cut;
    const int w = blockIdx.x / chunks + 1;
    const int i = (blockIdx.x - (w - 1) * chunks) * P + warp;  // of the group's units and heads
    if (warp == 0) {
      const Cut found = cut_at(sa, w, T);
      if (lane == 0) cut = found;
    }
    __syncthreads();
    if (cut.n > 0 && i < a.group * heads) {
      c0 = w - 1;
      h = i % heads;
      u = unit_info(a, cut.b, cut.us * a.group + i / heads);
      unit = static_cast<long long>(u.b) * a.ups + u.us;
      if (h < u.nh) n = cut.n;
    }
  } else {
    const long long pair = static_cast<long long>(blockIdx.x) * P + warp / W;
    const bool valid = pair < pairs;  // warp-uniform
    unit = valid ? pair / heads : 0;
    h = valid ? static_cast<int>(pair % heads) : 0;
    const int b = static_cast<int>(unit / a.ups);
    const int us = static_cast<int>(unit % a.ups);
    long long all = 0, before = 0;
    for (int bb = lane; bb < a.batch; bb += 32) {
      const long long t = span_tiles(load_span(sa, bb), T);
      all += t;
      if (bb < b) before += t;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    const long long total = all * a.upg;
    const long long nworkers = total < a.workers ? total : a.workers;
    const int nt = span_tiles(load_span(sa, b), T);
    if (valid && nt > 0) {
      const long long ug0 = before * a.upg + static_cast<long long>(us / a.group) * nt;
      c0 = worker_of(ug0, total, nworkers);
      n = static_cast<int>(worker_of(ug0 + nt - 1, total, nworkers) - c0 + 1);
      u = unit_info(a, b, us);
      // a unit with one worker was finished by it; heads past the unit's own do not exist
      if (n <= 1 || h >= u.nh) n = 0;
    }
  }
  wait_for_stream();
  if constexpr (W == 1) {
    if (n == 0) return;  // no barrier below for a warp per pair
  }
  const int mine = n > sub ? (n - sub + W - 1) / W : 0;  // contributors sub, sub + W, ...
  auto ml_of = [&](int j) {
    const long long slot = slot_of(unit, c0 + sub + W * j, a.group);
    return __ldcg(reinterpret_cast<const float2 *>(a.ws_ml + (slot * kMaxHeads + h) * 2));
  };
  const float *acc_base = a.ws_acc + static_cast<long long>(h) * HD + lane * DPL;
  float2 v[KB][DPL / 2];
  auto load_batch = [&](int j0) {
#pragma unroll
    for (int tt = 0; tt < KB; ++tt) {
      if (j0 + tt < mine) {
        const float *src =
            acc_base + slot_of(unit, c0 + sub + W * (j0 + tt), a.group) * kMaxHeads * HD;
#pragma unroll
        for (int i = 0; i < DPL / 2; ++i)
          v[tt][i] = __ldcg(reinterpret_cast<const float2 *>(src + 2 * i));
      } else {
#pragma unroll
        for (int i = 0; i < DPL / 2; ++i) v[tt][i] = make_float2(0.f, 0.f);
      }
    }
  };
  float2 first = make_float2(-INFINITY, 0.f);  // (m, l) of contributor `lane`
  if (lane < mine) first = ml_of(lane);
  load_batch(0);
  float mx = first.y > 0.f ? first.x : -INFINITY;
  for (int j = lane + 32; j < mine; j += 32) {
    const float2 ml = ml_of(j);
    if (ml.y > 0.f) mx = fmaxf(mx, ml.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  __shared__ float s_max[8];
  __shared__ float s_l[8];
  __shared__ __align__(16) float s_acc[W > 1 ? 8 : 1][HD];
  float M = mx;
  if constexpr (W > 1) {
    if (lane == 0) s_max[warp] = mx;
    __syncthreads();
    M = s_max[warp - sub];
#pragma unroll
    for (int w = 1; w < W; ++w) M = fmaxf(M, s_max[warp - sub + w]);
  }
  float O[DPL];
#pragma unroll
  for (int i = 0; i < DPL; ++i) O[i] = 0.f;
  float L = 0.f;
  for (int j0 = 0; j0 < mine; j0 += 32) {
    float2 ml = first;
    if (j0 > 0) ml = j0 + lane < mine ? ml_of(j0 + lane) : make_float2(-INFINITY, 0.f);
    const float wk = ml.y > 0.f ? fast_exp2(ml.x - M) : 0.f;
    L += wk * ml.y;
    const int cnt = min(32, mine - j0);
    for (int t0 = 0; t0 < cnt; t0 += KB) {
      if (j0 + t0 > 0) load_batch(j0 + t0);
#pragma unroll
      for (int tt = 0; tt < KB; ++tt) {
        const float w = __shfl_sync(0xffffffffu, wk, (t0 + tt) & 31);
#pragma unroll
        for (int i = 0; i < DPL / 2; ++i) {
          O[2 * i] += w * v[tt][i].x;
          O[2 * i + 1] += w * v[tt][i].y;
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if constexpr (W > 1) {
#pragma unroll
    for (int i = 0; i < DPL; ++i) s_acc[warp][lane * DPL + i] = O[i];
    if (lane == 0) s_l[warp] = L;
    __syncthreads();
    if (sub != 0) return;
    L = s_l[warp];
#pragma unroll
    for (int i = 0; i < DPL; ++i) O[i] = s_acc[warp][lane * DPL + i];
#pragma unroll
    for (int w = 1; w < W; ++w) {
      L += s_l[warp + w];
#pragma unroll
      for (int i = 0; i < DPL; ++i) O[i] += s_acc[warp + w][lane * DPL + i];
    }
  }
  if (n == 0) return;
  const float inv = L > 0.f ? 1.f / L : 0.f;
  const long long dst = (static_cast<long long>(u.b) * a.qh + u.h0 + h) * HD + lane * DPL;
#pragma unroll
  for (int i = 0; i < DPL; i += 2)
    store_out2(sa.s, sa.out, dst + i, O[i] * inv, O[i + 1] * inv);
}

pa_status_t resolve_score(const pa_score_t *score, float scale, ScoreArgs *s) {
  std::memset(s, 0, sizeof(*s));
  if (!score) return PA_OK;
  if (!(score->softcap >= 0.f) || !std::isfinite(score->softcap) || score->window < 0 ||
      score->out_type < PA_OUT_FP32 || score->out_type > PA_OUT_FP16 || score->reserved != 0)
    return PA_ERR_INVALID_ARG;
  if (score->softcap > 0.f) {
    s->cap_in = static_cast<float>(static_cast<double>(scale) / score->softcap);
    s->cap_out = static_cast<float>(score->softcap * 1.4426950408889634);
    // a cap so small or large against the scale that the quotient is no normal number, or that the
    // exponential form's multiple of it is none
    if (scale != 0.f && (!std::isnormal(s->cap_in) || !std::isfinite(4.f * s->cap_in)))
      return PA_ERR_INVALID_ARG;
    if (!std::isfinite(s->cap_out)) return PA_ERR_INVALID_ARG;
    // tanh's polynomial as one of the raw dot product v = t / cap_in. Under a large cap the highest
    // coefficients fall below the normal floats: one that does is left out, for arguments so small
    // that its term would be below 2^-24 of the sum.
    const double in = static_cast<double>(scale) / score->softcap;
    double power = in * score->softcap * 1.4426950408889634, z_max = 0.25;
    for (int k = 0; k < 4; ++k, power *= in * in) {
      const float c = static_cast<float>(kTanhFit[k] * power);
      if (std::isnormal(c))
        s->cap_poly[k] = c;
      else
        z_max = k == 0 ? -1. : std::min(z_max, std::pow(0x1p-24 / std::fabs(kTanhFit[k]), 1. / k));
    }
    s->cap_poly_max = z_max < 0. ? -1.f : static_cast<float>(std::min(z_max / (in * in), 3e38));
    s->cap_wide = s->cap_in != 0.f && score->softcap > 256.f;
  }
  const uintptr_t ptrs = reinterpret_cast<uintptr_t>(score->slopes) |
                         reinterpret_cast<uintptr_t>(score->first_tokens) |
                         reinterpret_cast<uintptr_t>(score->prefix_lengths);
  if (ptrs & 3u) return PA_ERR_MISALIGNED;
  s->slopes = score->slopes;
  s->first = score->first_tokens;
  s->prefix = score->prefix_lengths;
  s->window = score->window;
  s->out_half = score->out_type == PA_OUT_FP16;
  return PA_OK;
}

namespace {

template <int HD, int T>
cudaError_t launch_scored(const ScoredArgs &a, const CUtensorMap &tk, const CUtensorMap &tv,
                          const pa_plan_t &pl, cudaStream_t stream) {
  static std::atomic<bool> set[kMaxLaunchDevices];
  auto kern = decode_scored_kernel<HD, T>;
  const cudaError_t e = allow_smem(kern, kMaxDecodeSmem, set);
  if (e != cudaSuccess) return e;
  return launch_early(kern, dim3(pl.ctas), pl.warps_per_cta * 32, static_cast<int>(pl.smem_bytes),
                      stream, a, tk, tv);
}

template <int HD, int W>
cudaError_t launch_join(const ScoredArgs &a, int units, int heads, int tile, cudaStream_t stream) {
  const long long pairs = static_cast<long long>(units) * heads;
  constexpr int P = 8 / W;
  return launch_early(join_scored_kernel<HD, W, false>,
                      dim3(static_cast<unsigned>((pairs + P - 1) / P)), 256, 0, stream, a, heads,
                      pairs, 1, tile);
}

template <int HD>
cudaError_t launch_join_hd(const ScoredArgs &a, int units, int heads, int warps, int tile,
                           cudaStream_t stream) {
  if (units > a.k.workers * a.k.group) {  // (warps is 1)
    const int chunks = (a.k.group * heads + 7) / 8;
    if (a.k.workers == 1) return cudaSuccess;  // nothing is shared
    return launch_early(join_scored_kernel<HD, 1, true>,
                        dim3(static_cast<unsigned>((a.k.workers - 1) * chunks)), 256, 0, stream, a,
                        heads, 0ll, chunks, tile);
  }
  switch (warps) {
    case 1: return launch_join<HD, 1>(a, units, heads, tile, stream);
    case 2: return launch_join<HD, 2>(a, units, heads, tile, stream);
    case 4: return launch_join<HD, 4>(a, units, heads, tile, stream);
    default: return launch_join<HD, 8>(a, units, heads, tile, stream);
  }
}

}  // namespace

int device_sm_count() {
  static std::atomic<int> known[kMaxLaunchDevices];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxLaunchDevices) return 0;
  n = known[dev].load(std::memory_order_relaxed);
  if (n == 0 && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
    known[dev].store(n, std::memory_order_relaxed);
  return n;
}

pa_status_t fill_scored_args(const pa_problem_t *problem, const pa_plan_t &pl, const void *query,
                             const int32_t *block_tables, const int32_t *context_lengths,
                             float scale, void *out, void *workspace, ScoredArgs *a) {
  const int g = problem->query_heads / problem->kv_heads;
  KernelArgs &k = a->k;
  k.q = static_cast<const uint16_t *>(query);
  k.bt = block_tables;
  k.ctx = context_lengths;
  k.err = device_error_word();
  if (!k.err) return PA_ERR_CUDA;
  k.batch = problem->batch;
  k.qh = problem->query_heads;
  k.kvh = problem->kv_heads;
  k.hd = problem->head_dim;
  k.ps = problem->page_size;
  while ((1 << k.ps_shift) < k.ps) ++k.ps_shift;
  k.maxp = problem->max_pages_per_sequence;
  k.num_pages = problem->num_physical_pages;
  k.layout = problem->cache_layout;
  k.g = g;
  k.sub = (g + kMaxHeads - 1) / kMaxHeads;
  k.nh_unit = (g + k.sub - 1) / k.sub;
  k.ups = k.kvh * k.sub;
  k.group = pl.group;
  k.upg = k.ups / k.group;
  k.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  k.mode = pl.schedule == PA_SCHEDULE_SINGLE ? MODE_SINGLE : MODE_BALANCED;
  k.workers = pl.workers / pl.group;
  k.stages = pl.stages;
  a->out = out;
  if (k.mode == MODE_BALANCED) {
    const int64_t slots = static_cast<int64_t>(pl.units) + pl.workers;
    char *base = static_cast<char *>(workspace);
    k.ws_ml = reinterpret_cast<float *>(base);
    k.ws_acc = reinterpret_cast<float *>(base + (slots * kMaxHeads * 2 * 4 + 255) / 256 * 256);
  }
  return PA_OK;
}

cudaError_t launch_join_states(const ScoredArgs &a, int units, int heads, int warps, int tile,
                               cudaStream_t stream) {
  switch (a.k.hd) {
    case 64: return launch_join_hd<64>(a, units, heads, warps, tile, stream);
    case 128: return launch_join_hd<128>(a, units, heads, warps, tile, stream);
    default: return launch_join_hd<256>(a, units, heads, warps, tile, stream);
  }
}

}  // namespace pa

extern "C" pa_status_t pa_decode_scored(const pa_problem_t *problem, const pa_score_t *score,
                                        const void *query, const void *key_cache,
                                        const void *value_cache, const int32_t *block_tables,
                                        const int32_t *context_lengths, float scale, void *out,
                                        const pa_options_t *options, void *workspace,
                                        size_t workspace_bytes, void *stream) {
  using namespace pa;
  pa_status_t st = validate_call(problem, options, query, key_cache, value_cache, block_tables,
                                 context_lengths, scale, static_cast<const float *>(out));
  if (st != PA_OK) return st;
  ScoredArgs a;
  std::memset(&a, 0, sizeof(a));
  st = resolve_score(score, scale, &a.s);
  if (st != PA_OK) return st;
  if (options && (options->math == PA_MATH_SIMT || options->combine == PA_COMBINE_FUSED))
    return PA_ERR_UNSUPPORTED;
  // With at most three tiles to a unit one worker walks them faster than several share and join
  // them (head_dim 64, two sequences: 7.0 against 9.0 us; from four tiles on 9.7 against 9.4).
  pa_options_t single = {};
  pa_plan_t pl;
  st = pa_plan(problem, options, 1, &pl);  // shapes and options the plan refuses
  if (st != PA_OK) return st;
  if (!options || options->schedule == PA_SCHEDULE_AUTO) {
    int64_t most = static_cast<int64_t>(problem->max_pages_per_sequence) * problem->page_size;
    int64_t tiles = (most + pl.tile_tokens - 1) / pl.tile_tokens;
    if (a.s.window > 0 && a.s.window < most)  // a window may start anywhere in a tile
      tiles = std::min(tiles, (int64_t{a.s.window} + 2 * pl.tile_tokens - 2) / pl.tile_tokens);
    if (tiles <= 3) {
      if (options) single = *options;
      single.schedule = PA_SCHEDULE_SINGLE;
      options = &single;
    }
  }
  if (problem->batch == 0) return PA_OK;
  int smem_optin = 0;
  st = current_device_smem(&smem_optin);
  if (st != PA_OK) return st;
  st = pa_plan(problem, options, device_sm_count(), &pl);
  if (st != PA_OK) return st;
  // At head_dim 128 a warp with one tile on the way beside the one it works on is faster than
  // with two (32 heads of their own over 2048 tokens, 64 sequences: 191 against 202 us; 8 K/V
  // heads over 28613 tokens, 4 sequences: 76 against 81; never slower). Eight warps keep the
  // multiprocessor to one CTA either way, so the split and the workspace stay the plan's.
  if (problem->head_dim == 128 && pl.tile_tokens == 16 && pl.warps_per_cta == kMaxWarpsPerCta &&
      pl.stages > 2 && (!options || options->stages == 0)) {
    pl.stages = 2;
    pl.smem_bytes = kSmemAlign + kMaxWarpsPerCta * warp_smem_bytes(128, 1, kMaxHeads, 2, 16);
  }
  if (pl.workspace_bytes > 0) {
    if (!workspace || workspace_bytes < static_cast<size_t>(pl.workspace_bytes))
      return PA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return PA_ERR_MISALIGNED;
  }

  alignas(64) CUtensorMap tk, tv;
  const int hd = problem->head_dim;
  const int rows = problem->page_size < pl.tile_tokens ? problem->page_size : pl.tile_tokens;
  const int blocks = rows == pl.tile_tokens ? hd / 64 : 1;
  st = encode_row_map(&tk, key_cache, problem, rows, blocks);
  if (st != PA_OK) return st;
  st = encode_row_map(&tv, value_cache, problem, rows, blocks);
  if (st != PA_OK) return st;
  st = fill_scored_args(problem, pl, query, block_tables, context_lengths, scale, out, workspace,
                        &a);
  if (st != PA_OK) return st;
  KernelArgs &k = a.k;
  k.warp_smem = warp_smem_bytes(hd, 1, kMaxHeads, pl.stages, pl.tile_tokens);
  if (options && (options->test_flags & PA_TEST_EXPIRE_WAITS)) k.tx_extra = 16;

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
  if (hd == 64 && pl.tile_tokens == 32)
    e = launch_scored<64, 32>(a, tk, tv, pl, s);
  else if (hd == 128 && pl.tile_tokens == 16)
    e = launch_scored<128, 16>(a, tk, tv, pl, s);
  else if (hd == 128 && pl.tile_tokens == 32)
    e = launch_scored<128, 32>(a, tk, tv, pl, s);
  else if (hd == 256 && pl.tile_tokens == 16)
    e = launch_scored<256, 16>(a, tk, tv, pl, s);
  if (e != cudaSuccess) return PA_ERR_CUDA;
  if (k.mode == MODE_BALANCED) {
    e = launch_join_states(a, pl.units, k.nh_unit, combine_warps_per_pair(pl.units, pl.workers),
                           pl.tile_tokens, s);
    if (e != cudaSuccess) return PA_ERR_CUDA;
  }
  return PA_OK;
}
