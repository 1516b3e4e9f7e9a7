// scored_softmax.cuh -- the softmax of one unit of 64 keys under a score rule, for the multi-token
// kernels: one query row per thread, the unit's raw dot products in registers.
//
// These instructions bound the kernels: two warps a scheduler run them (one at head_dim 256)
// next to the products. 64 scores, loaded once and worked on in place, and the packed weights fit
// the registers but for one to four words of an item's state (4 to 16 bytes a thread at head_dim 64
// and 128, none at 256); of 128 columns the scores themselves spilled, and the shared memory being
// full a spilled word is an L2 access (eight prompts of 2048 in windows of 1024, capped, head_dim
// 128: 968 us so, 265 us with 64). The code has to fit the instruction cache as well: each part of
// the rule is written once, and what only some calls need is compiled into kernels of their own.
//  * tanh is a polynomial on the fp32 pipe in packed pairs wherever a warp's arguments allow:
//    tanh t = t P(t^2) with P of degree 3, fitted to the least relative error for |t| <= 1/2
//    (5.8e-7 evaluated in fp32; weighted least squares on Chebyshev nodes, weights iterated
//    towards the equal-ripple fit), the scale and the cap folded into its coefficients. A score
//    is then off by at most 0.47 cap * 5.8e-7, 1.4e-5 for a cap of 50, against the 2^-11 by
//    which the fp16 probability is rounded. A warp with a larger argument in its unit takes
//    1 - 2 / (1 + e^2t) for it, whose error of up to 3.6e-7 of the cap stays below a fifth of that
//    rounding up to a cap of 256. Larger caps have kernels of their own, in which such a unit goes
//    through tensor memory once more and each score takes the form that is exact for it (eight
//    prompts of 2048 in windows of 1024, head_dim 128: 423 us if every unit does, 348 with the
//    exponential alone, 265 with the polynomial alone; in the same kernels that code cost calls
//    under small caps up to 4 %). tanh being monotonic, the unit's maximum is that of the raw
//    products, capped, where nothing is masked or biased.
//  * The bias is linear in the key's column wherever no key of the columns lies past its query.
//  * The mask is compared per score only in units where some row of the warp needs it, and a
//    unit that none of the warp's rows sees is not computed at all.
#pragma once

#include <type_traits>

#include "prefill_kernel.cuh"
#include "score_rule.cuh"

namespace pa {

struct PrefillScoredArgs : PrefillArgs {
  ScoreArgs s;
  uint16_t *out16;  // [total][qh][hd], fp16 bits
};

// Parts of a rule that a kernel is compiled for; kRuleWide (only with kRuleCap): a cap above 256.
enum : int { kRuleCap = 1, kRuleSlopes = 2, kRuleFirst = 4, kRuleParts = 8, kRuleWide = 8 };

template <bool kScored>
using PrefillArgsOf = std::conditional_t<kScored, PrefillScoredArgs, PrefillArgs>;

// A row's reference maximum moves only when a score passes it by more than 2^15: weights stay
// below 2^15 until then, which fp16 holds as precisely as any.
constexpr float kScoredSlack = 15.f;  // log2 units

// A query row: its position, the tokens [lo, hi] it sees, its head's slope * log2 e, and the
// softmax so far (reference maximum in base 2, sum). `counts` is false for a row of the query tile
// that is no new token's: its scores may be anything.
struct ScoredRow {
  int pos, lo, hi;
  bool counts;
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

// cap_out * tanh(v * cap_in) = cap_out (1 - 2 / (1 + e^2t)); e^2t overflows to infinity and
// underflows to 0 where tanh is +-1. Off by at most 7.2e-7 of the score for |t| >= 1/2, and by
// 3.6e-7 of the cap below, where the difference cancels.
__device__ __forceinline__ float cap_exp(const ScoreArgs &s, float v) {
  const float e = prefill_exp2(v * (s.cap_in * (2.f * kLog2e)));
  return fmaf(-2.f * s.cap_out, fast_rcp(1.f + e), s.cap_out);
}

// The polynomial: cap_out * tanh(v * cap_in) = v * cap_poly(v), two columns at a time.
__device__ __forceinline__ float2 cap_poly(const ScoreArgs &s, float2 v) {
  const float2 z = fmul2(v, v);
  float2 p = ffma2(make_float2(s.cap_poly[3], s.cap_poly[3]), z,
                   make_float2(s.cap_poly[2], s.cap_poly[2]));
  p = ffma2(p, z, make_float2(s.cap_poly[1], s.cap_poly[1]));
  return ffma2(p, z, make_float2(s.cap_poly[0], s.cap_poly[0]));
}

// v = cap_out * tanh(v * cap_in), by the polynomial where `poly` (warp-uniform) says so.
__device__ __forceinline__ void cap_scores(float (&v)[64], const ScoreArgs &s, bool poly) {
  if (__builtin_expect(poly, 1)) {
#pragma unroll
    for (int c = 0; c < 64; c += 2) {
      const float2 x = make_float2(v[c], v[c + 1]);
      const float2 y = fmul2(cap_poly(s, x), x);
      v[c] = y.x;
      v[c + 1] = y.y;
    }
  } else {
#pragma unroll
    for (int c = 0; c < 64; ++c) v[c] = cap_exp(s, v[c]);
  }
}

// The same score by the form that is exact for it: below |t| = 1/2 the polynomial, not folded, so
// that it holds under any cap (the largest make t subnormal, which moves a score by 2^-22).
__device__ __forceinline__ float cap_each(const ScoreArgs &s, float v) {
  constexpr float p0 = kTanhFit[0], p1 = kTanhFit[1], p2 = kTanhFit[2], p3 = kTanhFit[3];
  const float t = v * s.cap_in, z = t * t;
  const float near = s.cap_out * (t * fmaf(fmaf(fmaf(p3, z, p2), z, p1), z, p0));
  return fabsf(t) <= 0.5f ? near : cap_exp(s, v);
}

// Replaces 64 columns of tensor memory by f of each. Warp-collective.
template <class F>
__device__ __forceinline__ void rewrite_columns(uint32_t ts, F f) {
#pragma unroll 1
  for (int c = 0; c < 64; c += 32) {
    float v[32];
    tmem_ld32(ts + c, v);
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = f(v[e]);
    tmem_st32(ts + c, v);
  }
  tmem_wait_st();
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

// Largest absolute value of 64 columns.
__device__ __forceinline__ float farthest(const float (&v)[64]) {
  float mx[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 64; c += 2)
    mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], fabsf(v[c]), fabsf(v[c + 1]));
  return max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
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

// Weights 2^x of 64 columns, arg(c) giving x of columns c and c + 1, as fp16 pairs; row.l grows by
// their sum, taken in fp32 before the rounding. fp16 because the tensor cores multiply the values'
// own type: off by half a step, 2^-11 of a weight, which moves an output by 1.2e-4 to 2.0e-4 of its
// size (rms) next to the 2.1e-4 of its own rounding to fp16. A second fp16 part for the remainder,
// as the decode step has, would double the output product and take the packing twice. Sixteen
// arguments are formed before their exponentials are taken.
template <class Arg>
__device__ __forceinline__ void weigh(ScoredRow &row, float (&pk)[32], Arg arg) {
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int e0 = 0; e0 < 32; e0 += 8) {
    float2 x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = arg(2 * (e0 + e));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 w = make_float2(prefill_exp2(x[e].x), prefill_exp2(x[e].y));
      sum[e & 1] = fadd2(sum[e & 1], w);
      pk[e0 + e] = __uint_as_float(pack_half2(w.x, w.y));
    }
  }
  row.l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// One unit of 64 keys from token `base`: raw dot products become weights relative to row.m,
// row.l grows by their sum. Warp-collective. `io` gives access to the row: load(v) reads the raw
// columns, rewrite(f) replaces each by f of it, settle(row, top, later) brings row.m up to date for
// a largest score `top` (settle_row; `later`: a unit after the row's first), emit(pk) takes the
// weights as fp16 pairs. False: a wait gave up. A row that has seen nothing yet has m = -inf.
//
// The largest score is needed only where it may move the reference, and where nothing is masked or
// biased the farthest raw product bounds it at half the comparisons (|tanh t| <= |t|).
// Io::kCapWithWeights: the cap of such a unit is taken in the loop of its weights (head_dim 128,
// two softmax warps a scheduler: 260 us against 304 for the prompts above; at head_dim 256, one
// warp a scheduler, two capped prompts of 4096 took 364 against 361, so not there).
// Io::kKeysCleared: the scores of tokens that no row sees are 0 (at head_dim 128 the prompts above
// take 266 us with those keys cleared, 275 with the raw products masked here; at 256 masking costs
// nothing).
template <int kParts, class Io>
__device__ __forceinline__ bool scored_weights(const ScoreArgs &s, float scale_log2,
                                               ScoredRow &row, int base, bool later,
                                               const Io &io) {
  const int lo = row.lo - base, hi = row.hi - base;
  float pk[32];
  if (!__any_sync(0xffffffffu, hi >= 0 && lo < 64 && lo <= hi)) {
#pragma unroll
    for (int e = 0; e < 32; ++e) pk[e] = 0.f;
    io.emit(pk);
    return true;
  }
  const bool masked = !__all_sync(0xffffffffu, lo <= 0 && hi >= 63);
  float v[64], mult = scale_log2, offset = 0.f, high, low;
  io.load(v);
  bool settled = false;
  if constexpr (kParts & kRuleCap) {
    constexpr bool kWide = (kParts & kRuleWide) != 0;
    // what no row sees, and rows that do not count, must not choose the warp's form of tanh
    if (masked && !Io::kKeysCleared) {
#pragma unroll
      for (int c = 0; c < 64; ++c) v[c] = c >= lo && c <= hi ? v[c] : 0.f;
    }
    const float far = farthest(v);
    const bool poly = __all_sync(0xffffffffu, !row.counts || far * far <= s.cap_poly_max);
    if (!(kParts & kRuleSlopes) && !masked && poly) {
      // |tanh t| <= |t|: no score is farther from 0 than the uncapped one
      if (__any_sync(0xffffffffu, far * fabsf(scale_log2) > row.m + kScoredSlack)) {
        extremes(v, high, low);  // capped scores are monotonic in the raw products
        const float best = scale_log2 >= 0.f ? high : low;
        // (the exponential form is near enough for a reference, but not at any cap)
        const float top = kWide ? cap_poly(s, make_float2(best, best)).x * best : cap_exp(s, best);
        if (!io.settle(row, top, later)) return false;
      }
      if constexpr (Io::kCapWithWeights) {
        const float2 n2 = make_float2(-row.m, -row.m);
        weigh(row, pk, [&](int c) {
          const float2 x = make_float2(v[c], v[c + 1]);
          return ffma2(cap_poly(s, x), x, n2);
        });
        io.emit(pk);
        return true;
      }
      settled = true;
    }
    if (kWide && !poly) {
      io.rewrite([&](float x) { return cap_each(s, x); });
      io.load(v);
    } else {
      cap_scores(v, s, kWide || poly);
    }
    mult = 1.f;
  } else if (!(kParts & kRuleSlopes) && !masked) {
    settled = !__any_sync(0xffffffffu,
                          farthest(v) * fabsf(scale_log2) > row.m + kScoredSlack);
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
  if (!settled) {
    extremes(v, high, low);
    const float top = fmaf(mult >= 0.f ? high : low, mult, offset);
    if (!io.settle(row, top, later)) return false;
  }
  if (row.m != -INFINITY) offset -= row.m;
  const float2 m2 = make_float2(mult, mult), n2 = make_float2(offset, offset);
  weigh(row, pk, [&](int c) { return ffma2(make_float2(v[c], v[c + 1]), m2, n2); });
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
                                                int prefix, bool counts) {
  ScoredRow r;
  r.counts = counts;
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

// Two outputs as fp16. Weights rounded up carry a mean of values next to fp16's largest past it by
// up to 2^-11 of it, which would round to infinity: it is given as the largest.
__device__ __forceinline__ uint32_t pack_mean2(float x, float y) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}

// 32 consecutive fp32 outputs of a row, scaled and written as fp16.
__device__ __forceinline__ void store_half32(uint16_t *dst, const float (&o)[32], float inv,
                                             bool v8, uint64_t pol) {
  uint32_t w[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e] = pack_mean2(o[2 * e] * inv, o[2 * e + 1] * inv);
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
