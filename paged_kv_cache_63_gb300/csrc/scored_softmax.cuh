// scored_softmax.cuh -- the softmax of one key tile under a score rule, for the multi-token
// kernels: one query row per thread, the tile's raw dot products in registers.
//
// A tile's chain bounds the kernel (scores, weights, the two products, the next scores), and in
// it the instructions per score of one warp and their fetching. So a tile is walked twice, first
// for the maximum, then for the weights, each part of them written as it stands, by loops short
// enough for the instruction cache. (One walk with the maximum as it was, checked by the sum as
// in the causal kernels, has to keep a row's weights until the check; its code spilled -- a
// spilled word is an L2 access, the shared memory being full -- or outgrew the cache: 6900
// cycles a tile unrolled, 4750 as a loop of 64 columns, on capped rows in a window.)
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

#include "prefill_kernel.cuh"
#include "score_rule.cuh"

namespace pa {

struct PrefillScoredArgs : PrefillArgs {
  ScoreArgs s;
  uint16_t *out16;  // [total][qh][hd], fp16 bits
};

// Parts of a rule that a kernel is compiled for.
enum : int { kRuleCap = 1, kRuleSlopes = 2, kRuleFirst = 4, kRuleParts = 8 };

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

// v = cap_out * tanh(v * cap_in), by the polynomial where `poly` (warp-uniform) says so.
__device__ __forceinline__ void cap_scores(float (&v)[64], const ScoreArgs &s, bool poly) {
  if (__builtin_expect(poly, 1)) {
    const float2 c0 = make_float2(s.cap_poly[0], s.cap_poly[0]),
                 c1 = make_float2(s.cap_poly[1], s.cap_poly[1]),
                 c2 = make_float2(s.cap_poly[2], s.cap_poly[2]),
                 c3 = make_float2(s.cap_poly[3], s.cap_poly[3]);
#pragma unroll
    for (int c = 0; c < 64; c += 2) {
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
    for (int c = 0; c < 64; ++c) v[c] = cap_exact(s, v[c]);
  }
}

// v = v * mult + slope2 * column, by steps of two columns, each off by a rounding (a table of
// columns for the packed pairs would take a register each).
__device__ __forceinline__ void add_slope(float (&v)[64], float slope2, float mult) {
  const float2 m2 = make_float2(mult, mult), step = make_float2(2.f * slope2, 2.f * slope2);
  float2 bias = make_float2(0.f, slope2);
#pragma unroll
  for (int c = 0; c < 64; c += 2) {
    const float2 x = ffma2(make_float2(v[c], v[c + 1]), m2, bias);
    v[c] = x.x;
    v[c + 1] = x.y;
    bias = fadd2(bias, step);
  }
}

// Extremes of 64 columns.
__device__ __forceinline__ void extremes(const float (&v)[64], float &hi, float &lo) {
  float mx[4] = {v[0], v[0], v[0], v[0]}, mn[4] = {v[0], v[0], v[0], v[0]};
#pragma unroll
  for (int c = 0; c < 64; c += 2) {
    mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], v[c], v[c + 1]);
    mn[(c >> 1) & 3] = min3(mn[(c >> 1) & 3], v[c], v[c + 1]);
  }
  hi = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
  lo = min3(fminf(mn[0], mn[1]), mn[2], mn[3]);
}

// Moves a row's reference to `top`, its largest score in the unit at hand, if that passes it by
// more than the slack; rescale(f) then multiplies the accumulated output by f (where `later`;
// false: a wait gave up). Warp-collective.
template <class Rescale>
__device__ __forceinline__ bool settle_row(ScoredRow &row, float top, bool later,
                                           Rescale rescale) {
  const bool grow = top > row.m + kScoredSlack;
  if (__any_sync(0xffffffffu, grow)) {
    const float mnew = grow ? top : row.m;
    const float f = mnew == -INFINITY ? 1.f : prefill_exp2(row.m - mnew);
    row.l *= f;
    if (later && !rescale(f)) return false;
    row.m = mnew;
  }
  return true;
}

// One unit of 64 keys from token `base`: raw dot products become weights relative to row.m,
// row.l grows by their sum. Warp-collective. `io` gives access to the row: load(v) reads the raw
// columns, settle(row, top, later) brings row.m up to date for a largest score `top` (settle_row;
// `later`: a unit after the row's first), emit(pk) takes the weights as fp16 pairs. False: a wait
// gave up. A row that has seen nothing yet has m = -inf.
template <int kParts, class Io>
__device__ __forceinline__ bool scored_weights(const ScoreArgs &s, float scale_log2,
                                               ScoredRow &row, int base, bool later,
                                               const Io &io) {
  const int lo = row.lo - base, hi = row.hi - base;
  float pk[32];
  if (!__any_sync(0xffffffffu, hi >= 0 && lo < 64 && lo <= hi)) {
    if (!io.settle(row, -INFINITY, later)) return false;
#pragma unroll
    for (int e = 0; e < 32; ++e) pk[e] = 0.f;
    io.emit(pk);
    return true;
  }
  const bool masked = !__all_sync(0xffffffffu, lo <= 0 && hi >= 63);
  float v[64], mult = scale_log2, offset = 0.f, high, low;
  io.load(v);
  float top = -INFINITY;
  bool known = false;  // whether top is the row's largest score already
  if constexpr (kParts & kRuleCap) {
    // columns nobody sees may widen the extremes, and so send the warp to the exact form
    extremes(v, high, low);
    const float far = fmaxf(fabsf(high), fabsf(low));
    const bool poly = __all_sync(0xffffffffu, far * far <= s.cap_poly_max);
    if (!masked && !(kParts & kRuleSlopes)) {
      // capped scores are monotonic in the raw products
      top = cap_exact(s, scale_log2 >= 0.f ? high : low);
      known = true;
    }
    cap_scores(v, s, poly);
    mult = 1.f;
  }
  if constexpr (kParts & kRuleSlopes) {
    const int rel = base - row.pos;
    if (__all_sync(0xffffffffu, rel + 63 <= 0)) {
      add_slope(v, row.slope2, mult);
      offset = row.slope2 * static_cast<float>(rel);
    } else {  // keys on both sides of the query: the distance of each
      const float first = static_cast<float>(rel);
#pragma unroll
      for (int c = 0; c < 64; ++c)
        v[c] = fmaf(-row.slope2, fabsf(first + static_cast<float>(c)), v[c] * mult);
    }
    mult = 1.f;
  }
  if (masked) {
    // the scale is never 0, so that the score of a masked column is -inf
    const float none = mult >= 0.f ? -INFINITY : INFINITY;
#pragma unroll
    for (int c = 0; c < 64; ++c) v[c] = c >= lo && c <= hi ? v[c] : none;
  }
  if (!known) {
    extremes(v, high, low);
    top = fmaf(mult >= 0.f ? high : low, mult, offset);
  }
  if (!io.settle(row, top, later)) return false;
  if (row.m != -INFINITY) offset -= row.m;
  const float2 m2 = make_float2(mult, mult), n2 = make_float2(offset, offset);
  float rp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    const int c = 2 * e;
    const float2 x = ffma2(make_float2(v[c], v[c + 1]), m2, n2);
    const float2 w = make_float2(prefill_exp2(x.x), prefill_exp2(x.y));
    const float2 acc = fadd2(make_float2(rp[c & 2], rp[(c & 2) + 1]), w);
    rp[c & 2] = acc.x;
    rp[(c & 2) + 1] = acc.y;
    pk[e] = __uint_as_float(pack_half2(w.x, w.y));
  }
  row.l += (rp[0] + rp[1]) + (rp[2] + rp[3]);
  io.emit(pk);
  return true;
}

// The range [lo, last] of the tokens that the new tokens [t0, t1) of a sequence see (its query
// rows start at q0, its new tokens at position p0); last = -1 if they see nothing. `holes`
// becomes true where some of them sees nothing: then tokens inside a range that is joined from
// several may be seen by nobody (otherwise each sees itself, and what they see is in one piece).
// Warp-collective; a lane takes every 32nd token.
template <int kParts>
__device__ __forceinline__ void seen_range(const ScoreArgs &s, int q0, int p0, int t0, int t1,
                                           int prefix, int &lo, int &last, bool &holes) {
  if constexpr (!(kParts & kRuleFirst)) {
    lo = first_seen(s, 0, p0 + t0);  // the window's start grows with the position
    last = p0 + t0 < prefix ? max(p0 + t1 - 1, prefix - 1) : p0 + t1 - 1;
    return;
  }
  int first = 0x7fffffff, end = -1;
  bool none = false;
  for (int t = t0 + (threadIdx.x & 31); t < t1; t += 32) {
    const int from = first_seen(s, static_cast<long long>(q0) + t, p0 + t);
    const int to = p0 + t < prefix ? prefix - 1 : p0 + t;
    if (from > to) {
      none = true;
    } else {
      first = min(first, from);
      end = max(end, to);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, first);
  last = __reduce_max_sync(0xffffffffu, end);
  if (__any_sync(0xffffffffu, none)) holes = true;
}

// Bits l .. r of a word; either may lie outside it.
__device__ __forceinline__ unsigned bits_between(int l, int r) {
  l = max(l, 0);
  r = min(r, 31);
  return l <= r ? (0xffffffffu >> (31 - r)) & (0xffffffffu << l) : 0u;
}

// Which of the TN tokens from `base` some of the new tokens [t0, t1) sees: 32 bits in each of the
// warp's first TN / 32 lanes. Only for work items with holes. Warp-collective.
template <int TN>
__device__ __forceinline__ unsigned seen_word(const ScoreArgs &s, int q0, int p0, int t0, int t1,
                                              int prefix, int base) {
  const int lane = threadIdx.x & 31;
  unsigned mine = 0;
#pragma unroll 1
  for (int w = 0; w < TN / 32; ++w, base += 32) {
    unsigned bits = 0;
#pragma unroll 1
    for (int t = t0 + lane; t < t1; t += 32) {
      const int from = first_seen(s, static_cast<long long>(q0) + t, p0 + t);
      bits |= bits_between(from - base, (p0 + t < prefix ? prefix - 1 : p0 + t) - base);
    }
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (lane == w) mine = bits;
  }
  return mine;
}

// Whether one of the n tokens from `at` on (n a power of two, at a multiple of it) has its bit set
// in the lanes' words. Warp-collective, with an n that is the same in all lanes.
__device__ __forceinline__ bool any_seen(unsigned word, int at, int n) {
  const unsigned words = __ballot_sync(0xffffffffu, word != 0);
  const unsigned own = __shfl_sync(0xffffffffu, word, (at >> 5) & 31);
  if (n >= 32) return (words >> ((at >> 5) & 31) & ((1u << (n >> 5)) - 1)) != 0;
  return (own >> (at & 31) & ((1u << n) - 1)) != 0;
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

// A row that sees nothing.
__device__ __forceinline__ void store_zero_row(uint16_t *dst, int n) {
  for (int i = 0; i < n; i += 8) *reinterpret_cast<uint4 *>(dst + i) = make_uint4(0, 0, 0, 0);
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
