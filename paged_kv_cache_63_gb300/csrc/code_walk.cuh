// code_walk.cuh -- a warp's walk through tiles of a quantised cache with up to eight query heads:
// loads, products of codes converted as they become operands, softmax. Used by the decode step
// (decode_quant.cu, whose head says why it is laid out like this) and by few new tokens
// (prefill_few_quant.cu).
#pragma once

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
constexpr int kQuantStages = 2;

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

// A tile's weights carry its values' scales, relative to the smallest that is seen, where these lie
// within 2^kScaleSpan: probabilities stay within 2^(kLift + kCodeSlack), weights within 2^15, and a
// weight keeps all bits of its probability. In other tiles the codes take their scales as they become
// operands, at four products of fp16 pairs for two of the tensor cores. 64 sequences of 1500 seen
// tokens, 32 heads of 128 of their own, cap: 134 us, 143 with the codes scaled in every tile; 32
// sequences of up to 4096, 32/8 heads: 32.6 and 34.3. (All weights relative to the tile's largest scale:
// 133 and 31.6, but they lost a bit for each power of two that they lay below it.)
constexpr uint32_t kScaleSpan = 3;
constexpr float kCodeSlack = 8.f - kScaleSpan;

// A tile's outputs, from the weights of its tokens. kScaled: the codes take their scales here, in a
// product that fp16 holds exactly; else the weights have them, relative to out_scale.
template <int HD, int T, bool kScaled>
__device__ __forceinline__ void code_values(CodeState<HD> &st, const CodeLane<HD, T> &ln,
                                            uint32_t stage, uint32_t scales,
                                            const uint32_t (&hi)[T / 16][2],
                                            const uint32_t (&lo)[T / 16][2], float out_scale) {
  using G = CodeGeom<HD, T>;
  constexpr int NG = T / 16, kQuarters = HD < 128 ? 2 : 4;
  uint32_t vs[NG][2];  // scales of the four tokens whose weights the lane has
  if constexpr (kScaled) {
    const int c = 2 * (threadIdx.x & 3);
    unrolled<NG>([&](auto g) {
      constexpr int gi = decltype(g)::value;
      const uint32_t b0 = lds16_at<T + gi * 16>(scales + c);
      const uint32_t b1 = lds16_at<T + gi * 16>(scales + 8 + ((c + 4) & 7));
      vs[gi][0] = half2_of_scales(b0 & 255, b0 >> 8);
      vs[gi][1] = half2_of_scales(b1 & 255, b1 >> 8);
    });
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
        uint32_t v[4] = {half2_of_low(w[2 * n]), half2_of_low(w[2 * n + 1]),
                         half2_of_high(w[2 * n]), half2_of_high(w[2 * n + 1])};
        if constexpr (kScaled) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = mul_half2(v[i], vs[gi][i >> 1]);
        }
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

// One tile: scores, rule, weights, outputs. c.sp is what some head sees; `rows` knows of each of the
// lane's two heads what it sees and where its query is.
template <int HD, int T, class Rows>
__device__ __forceinline__ void code_tile(CodeState<HD> &st, const CodeLane<HD, T> &ln,
                                          uint32_t stage, uint32_t scales, const SpanCursor &c,
                                          const ScoredArgs &a, const Rows &rows) {
  using G = CodeGeom<HD, T>;
  constexpr int NG = T / 16;  // groups of 16 tokens
  constexpr int kQuarters = HD < 128 ? 2 : 4;
  const int lane = threadIdx.x & 31;
  // the lane's tokens of a group: 16 g + row[i]
  const int row[2] = {lane >> 2, 8 + (((lane >> 2) + 4) & 7)};
  const int tok0 = c.tok;
  const uint32_t sa = scales + row[0], sb = scales + row[1];

  // the smallest and the largest scale of the values that are seen
  uint32_t least, most;
  {
    const int t = lane & (T > 32 ? 31 : T - 1);
    least = most = lds8_at<T>(scales + t);
    if (tok0 + t < c.sp.lo || tok0 + t >= c.sp.end) {
      least = 255;
      most = 0;
    }
    if constexpr (T > 32) {
      const uint32_t v = lds8_at<T + 32>(scales + t);
      if (tok0 + t + 32 >= c.sp.lo && tok0 + t + 32 < c.sp.end) {
        least = min(least, v);
        most = max(most, v);
      }
    }
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
  }
  const bool apart = most > least + kScaleSpan;

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
      y = fmaf(st.slope2[j], rows.distance(j, tok0 + g * 16 + row[i]), y);
    });
  if (rows.masks(tok0, tok0 + T))
    each([&](float &y, int g, int i, int j) {
      y = rows.sees(j, tok0 + g * 16 + row[i]) ? y : -INFINITY;
    });
  float top[2] = {-INFINITY, -INFINITY};
  each([&](float &y, int, int, int j) { top[j] = fmaxf(top[j], y); });
#pragma unroll
  for (int o = 4; o < 32; o <<= 1)
#pragma unroll
    for (int j = 0; j < 2; ++j) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
  if (__any_sync(0xffffffffu, top[0] > st.m[0] + (kLift + kCodeSlack) ||
                                  top[1] > st.m[1] + (kLift + kCodeSlack))) {
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

  uint32_t vbyte[NG][2];
  unrolled<NG>([&](auto g) {
    constexpr int gi = decltype(g)::value;
    vbyte[gi][0] = lds8_at<T + gi * 16>(sa);
    vbyte[gi][1] = lds8_at<T + gi * 16>(sb);
  });
  auto each_byte = [&](auto f) {
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < 2; ++i) f(vbyte[g][i], g, i);
  };
  // (a token that is not seen gets a finite factor, which its probability of 0 meets)
  if (partial) each_byte([&](uint32_t &v, int g, int i) { v = seen(g, i) ? v : least; });
  if (apart) {
    each_byte([&](uint32_t &v, int, int) { v = 127u; });
    least = 127u;
  }
  const float out_scale = __uint_as_float(least << 23);
  // 2^(b - least) as float bits: (b - least + 127) << 23
  const uint32_t bias = (127u - least) << 23;

  // Weights relative to the tile's scale: from the probability to 2^kScaleSpan of it, so they hold as
  // fp16 and keep all its bits; the row sum takes the probability.
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
  if (apart)
    code_values<HD, T, true>(st, ln, stage, scales, hi, lo, out_scale);
  else
    code_values<HD, T, false>(st, ln, stage, scales, hi, lo, out_scale);
}

// A decode step's heads: all of one query, which sees [lo, end) from its last token.
struct OneQuery {
  Span sp;
  __device__ __forceinline__ bool masks(int from, int to) const { return from < sp.lo || sp.end < to; }
  __device__ __forceinline__ bool sees(int, int t) const { return t >= sp.lo && t < sp.end; }
  __device__ __forceinline__ float distance(int, int t) const {
    return static_cast<float>(t - (sp.end - 1));
  }
};

// Bytes of shared memory of a CTA of `warps` walks with rings of `stages` tiles.
inline int quant_tile(int head_dim) { return head_dim == 64 ? 64 : head_dim == 128 ? 32 : 16; }

inline int quant_smem(int head_dim, int warps, int stages) {
  const int t = quant_tile(head_dim);
  return kSmemAlign + warps * stages * 2 * t * (head_dim + 1);
}

}  // namespace pa
