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
//    to the tile's largest, whose own power of two multiplies the tile's output. Scales come by
//    8-byte asynchronous copies that arrive on the tile's barrier: a page may hold fewer of them than
//    the 16 bytes of a TMA copy.
//  * Probabilities keep 22 bits (two fp16 numbers, a product each) and sums are fp32, as in
//    decode_scored.cu.
// 64 sequences of 1500 seen tokens, 32 heads of 128 of their own: 133.5 us, 0.89 of the copy bandwidth;
// four contexts of 100000, 24 / 4 heads of 256: 135.3 us, 0.91.
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

// Warps of a CTA, one CTA to a multiprocessor: the tiles in flight, two to a warp, are those of
// decode_scored.cu's eight warps, but a warp's chain of loads, products and shuffles is long for the
// half tile of bytes it brings (eight warps: 162 us against 134 for 64 sequences of 1500 seen tokens,
// 32 heads of 128 of their own; sixteen with tiles of 16 tokens, which the registers allow: 178).
constexpr int kQuantWarps = 12;

template <int HD, int T>
struct CodeGeom {
  static constexpr int kBlock = HD < 128 ? HD : 128;  // bytes of a column block's row
  static constexpr int kHalfBytes = T * HD;           // the K (or V) part of a stage
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int kScaleBytes = 2 * T;           // a stage's scales: K's, then V's
  static constexpr int kShift = T == 16 ? 4 : T == 32 ? 5 : 6;
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

// D(16x8, fp32) = A(16x16, fp16) B(16x8, fp16) + D; fresh: + 0.
__device__ __forceinline__ void mma_halves(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                           uint32_t b1, bool fresh) {
  if (fresh)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two 16x16 matrices of bytes, transposed: of each, r[2 m] has column lane / 4 and r[2 m + 1] column
// 8 + lane / 4 in rows 4 (lane % 4) .. + 3, lowest byte first. Lanes 0..15 give the rows' addresses
// of the first matrix, 16..31 of the second.
template <int kOff>
__device__ __forceinline__ void ldsm_bytes_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4+%5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(kOff));
}

// Issue the loads of the tile at cursor c into a stage. Pieces (min(page size, T) rows) that hold no
// seen token are not loaded; lane p looks at piece p. The barrier takes 33 arrivals: the announcement
// of the bytes, and each lane's copies of scales. Warp-collective. (Written as loops: what all warps
// run has to fit the instruction cache.)
template <int HD, int T>
__device__ __forceinline__ void issue_code_tile(const QuantDecodeArgs &qa, const CUtensorMap *tk,
                                                const CUtensorMap *tv, const SpanCursor &c, int kv,
                                                BtWindow &w, uint32_t stage, uint32_t scales,
                                                uint32_t bar, uint64_t pol, uint32_t extra_tx) {
  using G = CodeGeom<HD, T>;
  const KernelArgs &a = qa.k;
  const int lane = threadIdx.x & 31;
  const int shift = min(a.ps_shift, G::kShift);  // of a piece's rows
  const int npages = (c.sp.end + a.ps - 1) >> a.ps_shift;
  const bool hm = a.layout == PA_LAYOUT_HEAD_MAJOR;
  const int lp0 = c.tok >> a.ps_shift;
  bt_page(a, w, c.b, lp0, npages);  // the window is over the tile's first page from here on
  const int tok = c.tok + (lane << shift);
  const int at = min((tok >> a.ps_shift) - w.base, 63);
  const int p0 = __shfl_sync(0xffffffffu, w.cur, at & 31);
  const int p1 = __shfl_sync(0xffffffffu, w.nxt, at & 31);
  int page = at < 32 ? p0 : p1;
  const bool needed = lane < T >> shift && tok < c.sp.end && tok + (1 << shift) > c.sp.lo;
  const bool good = needed && page >= 0 && page < a.num_pages;
  if (needed && !good) atomicOr(a.err, PA_DEVERR_PAGE_ID);
  page = good ? page : -1;
  unsigned pieces = __ballot_sync(0xffffffffu, good);
  expect_bytes_warp(bar, (__popc(pieces) << shift) * (HD * 2) + extra_tx);
#pragma unroll 1
  for (; pieces; pieces &= pieces - 1) {
    const int p = __ffs(pieces) - 1;
    const int pg = __shfl_sync(0xffffffffu, page, p);
    const int slot = (c.tok + (p << shift)) & (a.ps - 1);
    const int row = hm ? slot : (pg << a.ps_shift) + slot;
    const int head = hm ? pg * a.kvh + kv : kv;
    const uint32_t dst = stage + (p << shift) * G::kBlock;
    tma_rows_warp(dst, tk, bar, row, head, 0, pol);
    tma_rows_warp(dst + G::kHalfBytes, tv, bar, row, head, 0, pol);
    if constexpr (HD > 128) {
      if (shift < G::kShift) {  // a whole tile's box has both column blocks
        tma_rows_warp(dst + T * G::kBlock, tk, bar, row, head, 1, pol);
        tma_rows_warp(dst + T * G::kBlock + G::kHalfBytes, tv, bar, row, head, 1, pol);
      }
    }
  }
  const int i = (lane & 15) * 8;  // token of the tile
  const int pg = __shfl_sync(0xffffffffu, page, (i >> shift) & 31);
  if (i < T) {
    const bool is_v = lane >= 16;
    const uint8_t *src = (is_v ? qa.v_scale : qa.k_scale) +
                         scale_place(max(pg, 0), kv, (c.tok + i) & (a.ps - 1), a.kvh, a.ps);
    copy8_async(scales + (is_v ? T : 0) + i, src, pg >= 0 ? 8u : 0u);
  }
  arrive_after_copies(bar);
}

// Running state of a unit (as SpanState of decode_scored.cu). Lane l has heads 2 (l % 4) and the next
// in its scores and outputs, and of the queries elements 4 (l % 4) .. + 3 of each 16 of head l / 4.
template <int HD>
struct CodeState {
  float m[2], lsum[2];
  float slope2[2];
  float o[HD / 16][4];  // elements 16 k + l / 4 (two heads), + 8 (two heads)
  uint32_t q[HD / 16][2];
};

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

// Zero V rows [from, to) of a stage: a zero probability must not meet a NaN code.
template <int HD, int T>
__device__ __forceinline__ void zero_code_rows(uint32_t stv, int from, int to) {
  const int lane = threadIdx.x & 31;
  const int n = (to - from) * (HD / 16);
  for (int i = lane; i < n; i += 32)
    sts128(stv + CodeGeom<HD, T>::at(from + i / (HD / 16), i % (HD / 16)), make_uint4(0, 0, 0, 0));
}

// Addresses of a lane's rows in a stage. Tokens are dealt in groups of 16: rows 0..7 of the scores are
// tokens 0..7, rows 8..15 tokens 12..15, 8..11, so that after the transposition lane l has weights of
// tokens 2 c, 2 c + 1 and 8 + (2 c + 4) % 8, + 1 (c = l % 4), and these four are rows 4 c .. 4 c + 3 of
// the values' matrix. (With the second eight in order, eight rows of a load would meet four banks.)
template <int HD, int T>
struct CodeLane {
  uint32_t k[HD < 128 ? 2 : 4];  // 32-element quarter of a column block
  uint32_t v[HD < 128 ? 2 : 4];
  __device__ __forceinline__ void init() {
    using G = CodeGeom<HD, T>;
    const int lane = threadIdx.x & 31;
    const int mi = lane >> 3, rr = lane & 7;
    const int i = lane & 15, c = 2 * (i >> 2) + (i & 1);
#pragma unroll
    for (int d = 0; d < (HD < 128 ? 2 : 4); ++d) {
      // matrices: rows 0..7 and 8..15 of the first 16 elements, then of the second
      k[d] = G::at(mi & 1 ? 8 + ((rr + 4) & 7) : rr, 2 * d + (mi >> 1));
      v[d] = G::kHalfBytes + G::at(i & 2 ? 8 + ((c + 4) & 7) : c, 2 * d + (lane >> 4));
    }
  }
};

// An 8x8 matrix of 16-bit elements, transposed: a lane gives row l / 4, columns 2 (l % 4), + 1.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int HD, int T>
__device__ __forceinline__ void code_tile(CodeState<HD> &st, const CodeLane<HD, T> &ln,
                                          uint32_t stage, uint32_t scales, const SpanCursor &c,
                                          const ScoredArgs &a) {
  using G = CodeGeom<HD, T>;
  constexpr int NG = T / 16;  // groups of 16 tokens
  constexpr int kQuarters = HD < 128 ? 2 : 4;
  const int lane = threadIdx.x & 31;
  // the lane's tokens of a group: 16 g + row[i]
  const int row[2] = {lane >> 2, 8 + (((lane >> 2) + 4) & 7)};
  const int tok0 = c.tok;
  const uint32_t sa = scales + row[0], sb = scales + row[1];

  // x[g][i][j]: token 16 g + row[i], head 2 (lane % 4) + j, in two chains (even and odd steps)
  float x[NG][2][2];
  unrolled<NG>([&](auto g) {
    constexpr int gi = decltype(g)::value;
    float d[2][4];
    unrolled<HD / 32>([&](auto q) {
      constexpr int ks = decltype(q)::value;
      uint32_t w[4];
      ldsm_x4_at<(ks / kQuarters) * (T * 128) + gi * 16 * G::kBlock>(stage + ln.k[ks % kQuarters],
                                                                     w);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint32_t k[4] = {half2_of_low(w[2 * n]), half2_of_low(w[2 * n + 1]),
                               half2_of_high(w[2 * n]), half2_of_high(w[2 * n + 1])};
        mma_halves(d[n], k, st.q[2 * ks + n][0], st.q[2 * ks + n][1], ks == 0);
      }
    });
    // a scale that no written row has belongs to a token that is masked below
    const float f[2] = {__uint_as_float(lds8_at<gi * 16>(sa) << 23),
                        __uint_as_float(lds8_at<gi * 16>(sb) << 23)};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) x[gi][i][j] = (d[0][2 * i + j] + d[1][2 * i + j]) * f[i];
  });

  // the score rule, in base-2 units
  const bool partial = tok0 < c.sp.lo || c.sp.end - tok0 < T;
  auto seen = [&](int g, int i) {
    const int t = tok0 + g * 16 + row[i];
    return t >= c.sp.lo && t < c.sp.end;
  };
  auto each = [&](auto f) {  // f(score, group, i, j)
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) f(x[g][i][j], g, i, j);
  };
  if (a.s.cap_in != 0.f)
    each([&](float &y, int, int, int) { y = a.s.cap_out * tanhf(y * a.s.cap_in); });
  else
    each([&](float &y, int, int, int) { y *= a.k.scale_log2; });
  if (a.s.slopes)
    each([&](float &y, int g, int i, int j) {
      y = fmaf(st.slope2[j], static_cast<float>(tok0 + g * 16 + row[i] - (c.sp.end - 1)), y);
    });
  if (partial) each([&](float &y, int g, int i, int) { y = seen(g, i) ? y : -INFINITY; });
  float top[2] = {-INFINITY, -INFINITY};
  each([&](float &y, int, int, int j) { top[j] = fmaxf(top[j], y); });
#pragma unroll
  for (int o = 4; o < 32; o <<= 1)
#pragma unroll
    for (int j = 0; j < 2; ++j) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
  if (__any_sync(0xffffffffu, top[0] > st.m[0] + (kLift + kRescaleSlack) ||
                                  top[1] > st.m[1] + (kLift + kRescaleSlack))) {
    float alpha[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float mn = fmaxf(st.m[j], top[j] - kLift);
      alpha[j] = mn == -INFINITY ? 1.f : fast_exp2(st.m[j] - mn);
      st.m[j] = mn;
      st.lsum[j] *= alpha[j];
    }
#pragma unroll
    for (int k = 0; k < HD / 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.o[k][i] *= alpha[i & 1];
  }
  float m[2];  // no score above -inf yet: 0
#pragma unroll
  for (int j = 0; j < 2; ++j) m[j] = st.m[j] == -INFINITY ? 0.f : st.m[j];

  // the values' scales, and the tile's largest of a value that is seen
  uint32_t vbyte[NG][2];
  unrolled<NG>([&](auto g) {
    constexpr int gi = decltype(g)::value;
    vbyte[gi][0] = lds8_at<T + gi * 16>(sa);
    vbyte[gi][1] = lds8_at<T + gi * 16>(sb);
  });
  if (partial) {
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < 2; ++i) vbyte[g][i] = seen(g, i) ? vbyte[g][i] : kSmallestByte;
  }
  uint32_t most = 0;
#pragma unroll
  for (int g = 0; g < NG; ++g) most = max(most, max(vbyte[g][0], vbyte[g][1]));
  most = min(__reduce_max_sync(0xffffffffu, most), 254u);
  const float out_scale = __uint_as_float(most << 23);
  // 2^(b - most) as float bits: (b - most + 127) << 23. Bytes of written rows lie within 23 of each
  // other, and a token that is not seen has the smallest, so that its probability of 0 meets a finite
  // number.
  const uint32_t bias = (127u - most) << 23;

  // Weights relative to the tile's scale: at most the probability, so they hold as fp16; the row sum
  // takes the probability.
  uint32_t hi[NG][2], lo[NG][2];
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float f = __uint_as_float((vbyte[g][i] << 23) + bias);
      float p0 = fast_exp2(x[g][i][0] - m[0]);
      float p1 = fast_exp2(x[g][i][1] - m[1]);
      st.lsum[0] += p0;
      st.lsum[1] += p1;
      p0 *= f;
      p1 *= f;
      const uint32_t h = pack_half2(p0, p1);
      const float2 r = half2_bits_to_float2(h);
      hi[g][i] = transposed(h);
      lo[g][i] = transposed(pack_half2(p0 - r.x, p1 - r.y));
    }

  if (partial) {
    const uint32_t stv = stage + G::kHalfBytes;
    if (tok0 < c.sp.lo) zero_code_rows<HD, T>(stv, 0, c.sp.lo - tok0);
    if (c.sp.end - tok0 < T) zero_code_rows<HD, T>(stv, c.sp.end - tok0, T);
    __syncwarp();
  }
  unrolled<HD / 32>([&](auto db) {
    constexpr int D = decltype(db)::value;
    float d[2][4];  // 16 elements each
    unrolled<NG>([&](auto g) {
      constexpr int gi = decltype(g)::value;
      uint32_t w[4];
      ldsm_bytes_trans<(D / kQuarters) * (T * 128) + gi * 16 * G::kBlock>(
          stage + ln.v[D % kQuarters], w);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint32_t v[4] = {half2_of_low(w[2 * n]), half2_of_low(w[2 * n + 1]),
                               half2_of_high(w[2 * n]), half2_of_high(w[2 * n + 1])};
        mma_halves(d[n], v, hi[gi][0], hi[gi][1], gi == 0);
        mma_halves(d[n], v, lo[gi][0], lo[gi][1], false);
      }
    });
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        st.o[2 * D + n][i] = fmaf(d[n][i], out_scale, st.o[2 * D + n][i]);
  });
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
    code_tile<HD, T>(st, lane_addr, wbase + cs * G::kStageBytes, wscales + cs * G::kScaleBytes, c, sa);
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


constexpr int kQuantStages = 2;

int quant_tile(int head_dim) { return head_dim == 64 ? 64 : head_dim == 128 ? 32 : 16; }

int quant_smem(int head_dim, int warps, int stages) {
  const int t = quant_tile(head_dim);
  return kSmemAlign + warps * stages * 2 * t * (head_dim + 1);
}

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
