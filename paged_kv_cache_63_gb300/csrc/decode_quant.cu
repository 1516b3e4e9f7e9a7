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
// that workers share are joined by the same kernel. A tile is twice the tokens in the same bytes.
//  * Codes stay bytes until they are operands: ldmatrix brings four codes of a token to a lane, and
//    the products run over the head's elements in the order in which they come. A word of four keys
//    converts to the two words that m16n8k16 takes for B (the query's fragments are loaded in the
//    same order); a word of two tokens by two elements of V (ldmatrix.trans on pairs of codes)
//    becomes a word for the even and one for the odd elements. The conversion is exact, one
//    instruction a pair.
//  * A key's scale multiplies its score in fp32; a value's scale, a power of two, its fp16 elements
//    (exact, quant.cuh). Scales come by 8-byte asynchronous copies that arrive on the tile's
//    barrier: a page may hold fewer of them than the 16 bytes of a TMA copy.
//  * Probabilities keep 22 bits and sums are fp32, as in decode_scored.cu.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "quant.cuh"
#include "row_maps.h"
#include "span_split.cuh"

namespace pa {

struct QuantDecodeArgs : ScoredArgs {
  const uint8_t *k_scale, *v_scale;
};

template <int HD, int T>
struct CodeGeom {
  static constexpr int kBlock = HD < 128 ? HD : 128;  // bytes of a column block's row
  static constexpr int kHalfBytes = T * HD;           // the K (or V) part of a stage
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int kScaleBytes = 2 * T;           // a stage's scales: K's, then V's
  // byte offset of 16-byte chunk `chunk` of tile row `row` (row_maps.h, encode_code_map)
  static __device__ __forceinline__ uint32_t at(int row, int chunk) {
    if constexpr (HD < 128)
      return static_cast<uint32_t>(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
    else
      return static_cast<uint32_t>((chunk >> 3) * (T * 128) + row * 128 +
                                   (((chunk & 7) ^ (row & 7)) << 4));
  }
};

__device__ __forceinline__ void copy8_async(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

// The barrier's arrival of this lane, once its asynchronous copies so far have landed.
__device__ __forceinline__ void arrive_after_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}

// Issue the loads of the tile at cursor c into a stage (warp-uniform), as issue_span_tile does. The
// barrier takes 33 arrivals: the announcement of the bytes, and each lane's copies of scales.
template <int HD, int T>
__device__ __forceinline__ void issue_code_tile(const QuantDecodeArgs &qa, const CUtensorMap *tk,
                                                const CUtensorMap *tv, const SpanCursor &c, int kv,
                                                BtWindow &w, uint32_t stage, uint32_t scales,
                                                uint32_t bar, uint64_t pol, uint32_t extra_tx) {
  using G = CodeGeom<HD, T>;
  const KernelArgs &a = qa.k;
  constexpr int kMaxPieces = T / 8;
  const int lane = threadIdx.x & 31;
  const int R = a.ps < T ? a.ps : T;
  const int npages = (c.sp.end + a.ps - 1) >> a.ps_shift;
  const bool hm = a.layout == PA_LAYOUT_HEAD_MAJOR;
  int page_of_lane = -1;  // the page of the eight scales that this lane copies
  auto place = [&](int tok, int &page, int &row, int &head) {  // false: id outside the pool
    page = bt_page(a, w, c.b, tok >> a.ps_shift, npages);
    const int slot = tok & (a.ps - 1);
    row = hm ? slot : (page << a.ps_shift) + slot;
    head = hm ? page * a.kvh + kv : kv;
    if (page >= 0 && page < a.num_pages) return true;
    if (lane == 0) atomicOr(a.err, PA_DEVERR_PAGE_ID);
    return false;
  };
  if (R == T) {
    int page, row, head;
    const bool good = place(c.tok, page, row, head);
    expect_bytes_warp(bar, (good ? G::kStageBytes : 0u) + extra_tx);
    if (good) {
      page_of_lane = page;
      tma_rows_warp(stage, tk, bar, row, head, 0, pol);
      tma_rows_warp(stage + G::kHalfBytes, tv, bar, row, head, 0, pol);
    }
  } else {
    int row[kMaxPieces], head[kMaxPieces];  // row < 0 marks a piece not loaded
    uint32_t bytes = 0;
#pragma unroll
    for (int p = 0; p < kMaxPieces; ++p) {
      const int tok = c.tok + p * R;
      int page;
      head[p] = 0;
      if (p * R < T && tok < c.sp.end && tok + R > c.sp.lo && place(tok, page, row[p], head[p])) {
        bytes += static_cast<uint32_t>(R * HD * 2);
        if ((lane & 15) * 8 >> a.ps_shift == p) page_of_lane = page;
      } else {
        row[p] = -1;
      }
    }
    expect_bytes_warp(bar, bytes + extra_tx);
#pragma unroll
    for (int p = 0; p < kMaxPieces; ++p) {
      if (row[p] < 0) continue;
#pragma unroll
      for (int blk = 0; blk < HD / G::kBlock; ++blk) {
        const uint32_t dst = stage + blk * (T * G::kBlock) + p * R * G::kBlock;
        tma_rows_warp(dst, tk, bar, row[p], head[p], blk, pol);
        tma_rows_warp(dst + G::kHalfBytes, tv, bar, row[p], head[p], blk, pol);
      }
    }
  }
  const int i = (lane & 15) * 8;  // token of the tile
  if (i < T) {
    const bool is_v = lane >= 16;
    const int page = max(page_of_lane, 0);
    const uint8_t *src = (is_v ? qa.v_scale : qa.k_scale) +
                         scale_place(page, kv, (c.tok + i) & (a.ps - 1), a.kvh, a.ps);
    copy8_async(scales + (is_v ? T : 0) + i, src, page_of_lane >= 0 ? 8u : 0u);
  }
  arrive_after_copies(bar);
}

// Running state of a unit (as SpanState of decode_scored.cu). A lane's row (head) is lane / 4; it
// holds elements 16 k + 4 (lane % 4) .. + 3 of the query and of the output.
template <int HD>
struct CodeState {
  float m, lsum;
  float slope2;
  float o[HD / 16][4];
  uint32_t qa[HD / 16][2];
};

template <int HD>
__device__ __forceinline__ void code_begin(CodeState<HD> &st, const ScoredArgs &a, int b, int h0,
                                           int nh) {
  const int lane = threadIdx.x & 31;
  const int h = lane >> 2;
  const uint2 *src = reinterpret_cast<const uint2 *>(
      a.k.q + (static_cast<long long>(b) * a.k.qh + h0 + h) * HD);
#pragma unroll
  for (int ks = 0; ks < HD / 16; ++ks) {
    const uint2 q = h < nh ? __ldg(src + ks * 4 + (lane & 3)) : make_uint2(0u, 0u);
    st.qa[ks][0] = q.x;
    st.qa[ks][1] = q.y;
  }
  st.slope2 = a.s.slopes && h < nh ? __ldg(a.s.slopes + h0 + h) * kLog2e : 0.f;
  st.m = -INFINITY;
  st.lsum = 0.f;
#pragma unroll
  for (int k = 0; k < HD / 16; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) st.o[k][j] = 0.f;
}

// Zero V rows [from, to) of a stage: a zero probability must not meet a NaN code.
template <int HD, int T>
__device__ __forceinline__ void zero_code_rows(uint32_t stv, int from, int to) {
  const int lane = threadIdx.x & 31;
  const int n = (to - from) * (HD / 16);
  for (int i = lane; i < n; i += 32)
    sts128(stv + CodeGeom<HD, T>::at(from + i / (HD / 16), i % (HD / 16)), make_uint4(0, 0, 0, 0));
}

template <int HD, int T>
__device__ __forceinline__ void code_tile(CodeState<HD> &st, uint32_t stage, uint32_t scales,
                                          const SpanCursor &c, const ScoredArgs &a) {
  using G = CodeGeom<HD, T>;
  constexpr int NT = T / 8;
  const int lane = threadIdx.x & 31;
  const int mi = lane >> 3, rr = lane & 7, col = 2 * (lane & 3);
  const int tok0 = c.tok;

  // S[h][t], eight tokens at a time, 64 elements a load; two chains
  float x[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float s[2][2] = {};
#pragma unroll
    for (int cq = 0; cq < HD / 64; ++cq) {
      uint32_t w[4];
      ldsm_x4(stage + G::at(rr, (cq & 1) * 4 + mi) + (cq >> 1) * (T * 128) + nt * 8 * G::kBlock,
              w[0], w[1], w[2], w[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mma_rows8(s[i & 1][0], s[i & 1][1], st.qa[cq * 4 + i][0], st.qa[cq * 4 + i][1],
                  half2_of_low(w[i]), half2_of_high(w[i]));
    }
    // a scale that no written row has belongs to a token that is masked below
    const uint32_t f = lds16(scales + nt * 8 + col);
    x[nt][0] = (s[0][0] + s[1][0]) * __uint_as_float(f << 23 & 0x7f800000u);
    x[nt][1] = (s[0][1] + s[1][1]) * __uint_as_float(f << 15 & 0x7f800000u);
  }

  // the score rule, in base-2 units; the row's scores live in lanes lane & ~3 .. lane | 3
  const bool partial = tok0 < c.sp.lo || c.sp.end - tok0 < T;
  const float away0 = static_cast<float>(tok0 + col - (c.sp.end - 1));
  float mt = -INFINITY;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float y = x[nt][j];
      y = a.s.cap_in != 0.f ? a.s.cap_out * tanhf(y * a.s.cap_in) : y * a.k.scale_log2;
      if (a.s.slopes) y = fmaf(st.slope2, away0 + static_cast<float>(nt * 8 + j), y);
      if (partial) {
        const int tok = tok0 + nt * 8 + col + j;
        y = tok >= c.sp.lo && tok < c.sp.end ? y : -INFINITY;
      }
      x[nt][j] = y;
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
    for (int k = 0; k < HD / 16; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) st.o[k][j] *= alpha;
  }
  const float m = st.m == -INFINITY ? 0.f : st.m;  // no score above -inf yet
  float psum = 0.f;
  uint32_t hi[NT], lo[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float p0 = fast_exp2(x[nt][0] - m);
    const float p1 = fast_exp2(x[nt][1] - m);
    hi[nt] = pack_half2(p0, p1);
    const float2 r = half2_bits_to_float2(hi[nt]);
    lo[nt] = pack_half2(p0 - r.x, p1 - r.y);
    psum += p0 + p1;
  }
  st.lsum += psum;

  uint32_t vf[NT];  // the values' scales
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const uint32_t f = lds16(scales + T + nt * 8 + col);
    vf[nt] = half2_of_scales(f & 0xffu, f >> 8);
  }
  if (partial) {
    const uint32_t stv = stage + G::kHalfBytes;
    if (tok0 < c.sp.lo) zero_code_rows<HD, T>(stv, 0, c.sp.lo - tok0);
    if (c.sp.end - tok0 < T) zero_code_rows<HD, T>(stv, c.sp.end - tok0, T);
    __syncwarp();
  }
#pragma unroll
  for (int cp = 0; cp < HD / 32; ++cp) {  // 32 elements: two chunks of 16
    float d[2][2][4] = {};                // [chunk][even, odd elements]
#pragma unroll
    for (int ch = 0; ch < NT / 2; ++ch) {
      uint32_t w[4];  // chunk 0 tokens 0..7, 8..15, chunk 1 likewise
      ldsm_x4_trans(stage + G::kHalfBytes + G::at((mi & 1) * 8 + rr, (2 * cp & 7) + (mi >> 1)) +
                        (cp >> 2) * (T * 128) + ch * 16 * G::kBlock,
                    w[0], w[1], w[2], w[3]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t u = __byte_perm(w[2 * k], 0, 0x3120), z = __byte_perm(w[2 * k + 1], 0, 0x3120);
        mma_rows16(d[k][0], hi[2 * ch], lo[2 * ch], hi[2 * ch + 1], lo[2 * ch + 1],
                   mul_half2(half2_of_low(u), vf[2 * ch]), mul_half2(half2_of_low(z), vf[2 * ch + 1]));
        mma_rows16(d[k][1], hi[2 * ch], lo[2 * ch], hi[2 * ch + 1], lo[2 * ch + 1],
                   mul_half2(half2_of_high(u), vf[2 * ch]),
                   mul_half2(half2_of_high(z), vf[2 * ch + 1]));
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        st.o[2 * cp + k][j] += d[k][j][0] + d[k][j][2];
        st.o[2 * cp + k][2 + j] += d[k][j][1] + d[k][j][3];
      }
  }
}

template <int HD, int T>
__global__ void __launch_bounds__(kMaxWarpsPerCta * 32, 1)
    decode_quant_kernel(const __grid_constant__ QuantDecodeArgs sa,
                        const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv) {
  using G = CodeGeom<HD, T>;
  const KernelArgs &a = sa.k;
  extern __shared__ uint8_t dsm[];
  __shared__ __align__(8) uint64_t bars[kMaxWarpsPerCta * kMaxStages];
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
  while (flying < S - 1 && ic.left > 0) issue();

  CodeState<HD> st = {};
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
      const long long at =
          (static_cast<long long>(cur.b) * a.qh + cur.h0 + h) * HD + 4 * (lane & 3);
#pragma unroll
      for (int k = 0; k < HD / 16; ++k) {
        store_out2(sa.s, sa.out, at + k * 16, st.o[k][0] * inv, st.o[k][1] * inv);
        store_out2(sa.s, sa.out, at + k * 16 + 2, st.o[k][2] * inv, st.o[k][3] * inv);
      }
      return;
    }
    // partial state relative to the row's reference, for the joining kernel
    const long long slot = slot_of(unit, worker, a.group) * kMaxHeads + h;
    if ((lane & 3) == 0)
      *reinterpret_cast<float2 *>(a.ws_ml + slot * 2) = make_float2(st.m, l);
    float *dst = a.ws_acc + slot * HD + 4 * (lane & 3);
#pragma unroll
    for (int k = 0; k < HD / 16; ++k)
      *reinterpret_cast<float4 *>(dst + k * 16) =
          make_float4(st.o[k][0], st.o[k][1], st.o[k][2], st.o[k][3]);
  };

  // ---- main loop: refill the slot freed last iteration, wait for the next tile, compute
  while (c.left > 0) {
    if (c.b != cur.b || c.us * a.group + member != cur.us) {
      if (cur.b >= 0) finish_unit();
      cur = unit_info(a, c.b, c.us * a.group + member);
      cur_ug0 = c.ug0;
      cur_tiles = span_tiles(c.sp, T);
      code_begin<HD>(st, sa, cur.b, cur.h0, cur.nh);
    }
    if (ic.left > 0) issue();
    if (!mbar_wait(bar0 + 8 * cs, cphase, a.err)) {
      aborted = true;
      break;
    }
    code_tile<HD, T>(st, wbase + cs * G::kStageBytes, wscales + cs * G::kScaleBytes, c, sa);
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

namespace {

constexpr int kQuantStages = 3;

int quant_tile(int head_dim) { return head_dim == 64 ? 64 : head_dim == 128 ? 32 : 16; }

int quant_smem(int head_dim, int warps, int stages) {
  const int t = quant_tile(head_dim);
  return kSmemAlign + warps * stages * 2 * t * (head_dim + 1);
}

// What pa_decode_quant launches, in pa_plan's terms. `score`: null, or the resolved rule.
pa_status_t quant_plan(const pa_problem_t *p, const pa_options_t *o, int sm_count,
                       const ScoreArgs *score, pa_plan_t *pl) {
  pa_status_t st = pa_plan(p, o, sm_count, pl);  // its checks, and the split into units
  if (st != PA_OK) return st;
  if (o && (o->math || o->combine || o->tile_tokens)) return PA_ERR_UNSUPPORTED;
  const int g = p->query_heads / p->kv_heads;
  const int sub = (g + kMaxHeads - 1) / kMaxHeads;
  pl->tile_tokens = quant_tile(p->head_dim);
  pl->warps_per_cta = o && o->warps_per_cta ? o->warps_per_cta : kMaxWarpsPerCta;
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
