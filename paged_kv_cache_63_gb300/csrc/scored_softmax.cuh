// scored_softmax.cuh -- the softmax of one key tile under a score rule, for the multi-token
// kernels: one query row per thread, the tile's raw dot products in registers.
//
// A tile's chain bounds the kernel (scores, weights, the two products, the next scores), in it
// the instructions per score of a warp, and with them their fetching: so a tile is walked twice
// by short loops of 32 columns that hold no more than 32 scores, the first for the maximum, the
// second for the weights, each written to tensor memory as it stands. (One walk with the
// maximum as it was, checked by the sum as in the causal kernels, has to keep a row's weights
// until the check; its code spilled or outgrew the instruction cache: 6900 cycles a tile
// unrolled and 4750 as a loop of 64 columns, on the capped rows of 2048-token prompts.)
//  * tanh is a polynomial on the fp32 pipe in packed pairs wherever a warp's arguments allow:
//    tanh t = t P(t^2) with P of degree 3, fitted to the least relative error for |t| <= 1/2
//    (5.8e-7 evaluated in fp32; weighted least squares on Chebyshev nodes, weights iterated
//    towards the equal-ripple fit), the scale and the cap folded into its coefficients. A score
//    is then off by at most 0.47 cap * 5.8e-7, 1.4e-5 for a cap of 50, against the 2^-11 by
//    which the fp16 probability is rounded. A warp with a larger argument in its tile takes
//    1 - 2 / (1 + e^2t) for it. tanh being monotonic, the first walk needs the extremes of the
//    raw products only.
//  * The bias is linear in the key's column wherever no key of the columns lies past its query.
//  * The mask is compared per score only in tiles where some row of the warp needs it, and a
//    tile that none of the warp's rows sees is not computed at all.
#pragma once

#include <type_traits>

#include "prefill_common.cuh"
#include "score_rule.cuh"

namespace pa {

struct PrefillScoredArgs : PrefillArgs {
  ScoreArgs s;
  uint16_t *out16;  // [total][qh][hd], fp16 bits
};

template <bool kScored>
using PrefillArgsOf = std::conditional_t<kScored, PrefillScoredArgs, PrefillArgs>;

// A row's reference maximum moves only when a score passes it by more than 2^15: weights stay
// below 2^15 until then, which fp16 holds as precisely as any.
constexpr float kScoredSlack = 15.f;  // log2 units

// A query row: its position, the tokens [lo, hi] it sees, its head's slope * log2 e, and the
// softmax so far (reference maximum in base 2, sum).
struct ScoredRow {
  int pos, lo, hi;
  float slope2, m, l;
};

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// cap_out * tanh(v * cap_in); e^2t overflows to infinity and underflows to 0 where tanh is +-1
__device__ __forceinline__ float cap_exact(const ScoreArgs &s, float v) {
  const float e = prefill_exp2(v * (s.cap_in * (2.f * kLog2e)));
  return fmaf(-2.f * s.cap_out, fast_rcp(1.f + e), s.cap_out);
}

__device__ __forceinline__ void cap_scores(float (&v)[32], const ScoreArgs &s, bool poly) {
  if (__builtin_expect(poly, 1)) {
    const float2 c0 = make_float2(s.cap_poly[0], s.cap_poly[0]),
                 c1 = make_float2(s.cap_poly[1], s.cap_poly[1]),
                 c2 = make_float2(s.cap_poly[2], s.cap_poly[2]),
                 c3 = make_float2(s.cap_poly[3], s.cap_poly[3]);
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      const float2 x = make_float2(v[c], v[c + 1]);
      const float2 z = fmul2(x, x);
      float2 p = ffma2(c3, z, c2);
      p = ffma2(p, z, c1);
      p = ffma2(p, z, c0);
      p = fmul2(p, x);
      v[c] = p.x;
      v[c + 1] = p.y;
    }
  } else {
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] = cap_exact(s, v[c]);
  }
}

// v * mult - slope2 * distance for 32 columns of which the first is `rel` past the query; the
// part of the bias that the columns share is returned instead of added. Warp-collective.
__device__ __forceinline__ float bias_scores(float (&v)[32], float slope2, int rel, float mult) {
  if (__builtin_expect(__all_sync(0xffffffffu, rel + 31 <= 0), 1)) {
    // slope * column by steps of two columns, each off by a rounding: a table of columns for
    // the packed pairs would take 32 registers
    const float2 m2 = make_float2(mult, mult), step = make_float2(2.f * slope2, 2.f * slope2);
    float2 bias = make_float2(0.f, slope2);
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      const float2 x = ffma2(make_float2(v[c], v[c + 1]), m2, bias);
      v[c] = x.x;
      v[c + 1] = x.y;
      bias = fadd2(bias, step);
    }
    return slope2 * static_cast<float>(rel);
  }
  // keys on both sides of the query: the distance of each
  const float first = static_cast<float>(rel);
#pragma unroll
  for (int c = 0; c < 32; ++c)
    v[c] = fmaf(-slope2, fabsf(first + static_cast<float>(c)), v[c] * mult);
  return 0.f;
}

// One tile of TN keys from token `base`: raw dot products become weights relative to row.m,
// row.l grows by their sum. Warp-collective. `load(h, v)` reads raw columns 32 h .. 32 h + 31;
// `emit(h, pk)` takes their weights as fp16 pairs (columns are emitted in order, those up to
// 32 h + 31 having been read for the last time); `rescale(f)` multiplies the row's accumulated
// output by f (only called when `later`, a tile after the row's first; false from it: a wait
// gave up). A row that has seen nothing yet has m = -inf.
template <int TN, class Load, class Emit, class Rescale>
__device__ __forceinline__ bool scored_weights(const ScoreArgs &s, float scale_log2,
                                               ScoredRow &row, int base, bool later, Load load,
                                               Emit emit, Rescale rescale) {
  constexpr int H = TN / 32;
  const int lo = row.lo - base, hi = row.hi - base;
  const bool some = hi >= 0 && lo < TN && lo <= hi;
  if (!__any_sync(0xffffffffu, some)) {
    float none[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) none[e] = 0.f;
#pragma unroll
    for (int h = 0; h < H; ++h) emit(h, none);
    return true;
  }
  const bool full = __all_sync(0xffffffffu, lo <= 0 && hi >= TN - 1);
  const bool cap = s.cap_in != 0.f, biased = s.slopes != nullptr;

  // ---- the row's largest score
  float top = -INFINITY, low = INFINITY;  // of the raw products; of the scores where biased
  bool poly = true;
#pragma unroll 1
  for (int h = 0; h < H; ++h) {
    float v[32];
    load(h, v);
    float offset = 0.f;
    if (biased) {
      if (cap) cap_scores(v, s, false);
      offset = bias_scores(v, row.slope2, base + 32 * h - row.pos, cap ? 1.f : scale_log2);
    }
    float mx[2] = {-INFINITY, -INFINITY}, mn[2] = {INFINITY, INFINITY};
    if (full) {
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        mx[(c >> 1) & 1] = max3(mx[(c >> 1) & 1], v[c], v[c + 1]);
        mn[(c >> 1) & 1] = min3(mn[(c >> 1) & 1], v[c], v[c + 1]);
      }
    } else {
      const int l = lo - 32 * h, r = hi - 32 * h;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const bool in = c >= l && c <= r;
        mx[c & 1] = fmaxf(mx[c & 1], in ? v[c] : -INFINITY);
        mn[c & 1] = fminf(mn[c & 1], in ? v[c] : INFINITY);
      }
    }
    top = max3(top, mx[0] + offset, mx[1] + offset);
    low = min3(low, mn[0], mn[1]);
  }
  if (!biased) {
    // scores are monotonic in the raw products: growing with them for a positive scale
    const float ext = scale_log2 >= 0.f ? top : low;
    if (cap) {
      const float far = fmaxf(fabsf(top), fabsf(low));
      poly = __all_sync(0xffffffffu, !some || far * far <= s.cap_poly_max);
      top = some ? cap_exact(s, ext) : -INFINITY;
    } else {
      top = some ? ext * scale_log2 : -INFINITY;
    }
  } else {
    poly = false;
  }
  const bool grow = top > row.m + kScoredSlack;
  if (__any_sync(0xffffffffu, grow)) {
    const float mnew = grow ? top : row.m;
    const float f = mnew == -INFINITY ? 1.f : prefill_exp2(row.m - mnew);
    row.l *= f;
    if (later && !rescale(f)) return false;
    row.m = mnew;
  }

  // ---- the weights
  const float nm = row.m == -INFINITY ? 0.f : -row.m;
  float rp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int h = 0; h < H; ++h) {
    float v[32], mult = scale_log2, offset = nm;
    load(h, v);
    if (cap) {
      cap_scores(v, s, poly);
      mult = 1.f;
    }
    if (biased) {
      offset += bias_scores(v, row.slope2, base + 32 * h - row.pos, mult);
      mult = 1.f;
    }
    if (!full) {
      // the scale is never 0, so that the score of a masked column is -inf
      const float none = mult >= 0.f ? -INFINITY : INFINITY;
      const int l = lo - 32 * h, r = hi - 32 * h;
#pragma unroll
      for (int c = 0; c < 32; ++c) v[c] = c >= l && c <= r ? v[c] : none;
    }
    const float2 m2 = make_float2(mult, mult), n2 = make_float2(offset, offset);
    float pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int c = 2 * e;
      const float2 x = ffma2(make_float2(v[c], v[c + 1]), m2, n2);
      const float2 w = make_float2(prefill_exp2(x.x), prefill_exp2(x.y));
      const float2 acc = fadd2(make_float2(rp[c & 2], rp[(c & 2) + 1]), w);
      rp[c & 2] = acc.x;
      rp[(c & 2) + 1] = acc.y;
      pk[e] = __uint_as_float(pack_half2(w.x, w.y));
    }
    emit(h, pk);
  }
  row.l += (rp[0] + rp[1]) + (rp[2] + rp[3]);
  return true;
}

// The tokens that the new tokens [t0, t1) of sequence b see (t0 < t1; the sequence's query rows
// start at q0, its new tokens at position p0), as the range its key tiles are taken from:
// lowest first token and highest last one. A token that sees nothing counts as seeing itself,
// so that its tile still writes its zero row. Warp-collective; a lane takes every 32nd token.
__device__ __forceinline__ void seen_range(const ScoreArgs &s, int q0, int p0, int t0, int t1,
                                           int prefix, int &lo, int &last) {
  const int p_last = p0 + t1 - 1;
  last = p0 + t0 < prefix ? max(p_last, prefix - 1) : p_last;
  if (!s.first) {
    lo = min(first_seen(s, 0, p0 + t0), p0 + t0);  // the window's start grows with the position
    return;
  }
  int mine = 0x7fffffff;
  for (int t = t0 + (threadIdx.x & 31); t < t1; t += 32)
    mine = min(mine, min(first_seen(s, static_cast<long long>(q0) + t, p0 + t), p0 + t));
  lo = __reduce_min_sync(0xffffffffu, mine);
}

// Length of sequence b's prefix within its context.
__device__ __forceinline__ int prefix_of(const ScoreArgs &s, int b, int ctx) {
  return s.prefix ? min(__ldg(s.prefix + b), ctx) : 0;
}

// The thread's row: new token t of sequence b (position p0 + t).
__device__ __forceinline__ ScoredRow scored_row(const ScoreArgs &s, int q0, int p0, int t, int head,
                                                int prefix) {
  ScoredRow r;
  r.pos = p0 + t;
  r.lo = first_seen(s, static_cast<long long>(q0) + t, r.pos);
  r.hi = r.pos < prefix ? prefix - 1 : r.pos;
  r.slope2 = s.slopes ? __ldg(s.slopes + head) * kLog2e : 0.f;
  r.m = -INFINITY;
  r.l = 0.f;
  return r;
}

// 32 consecutive fp32 outputs of a row, scaled and written as fp16.
__device__ __forceinline__ void store_half32(uint16_t *dst, const float (&o)[32], float inv,
                                             bool v8, uint64_t pol) {
  uint32_t w[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e] = pack_half2(o[2 * e] * inv, o[2 * e + 1] * inv);
  if (v8) {
#pragma unroll
    for (int e = 0; e < 16; e += 8)
      st_global_v8(reinterpret_cast<float *>(dst + 2 * e), __uint_as_float(w[e]),
                   __uint_as_float(w[e + 1]), __uint_as_float(w[e + 2]), __uint_as_float(w[e + 3]),
                   __uint_as_float(w[e + 4]), __uint_as_float(w[e + 5]), __uint_as_float(w[e + 6]),
                   __uint_as_float(w[e + 7]), pol);
  } else {
#pragma unroll
    for (int e = 0; e < 16; e += 4)
      *reinterpret_cast<uint4 *>(dst + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
  }
}

}  // namespace pa
