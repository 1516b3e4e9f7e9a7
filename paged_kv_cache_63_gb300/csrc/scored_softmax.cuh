// scored_softmax.cuh -- the softmax of one key tile under a score rule, for the multi-token
// kernels: one query row per thread, the tile's raw dot products in registers.
//
// What bounds it is instructions per score (the special-function pipe and the fp32 pipe share
// the softmax warps' issue slots with the tensor-memory traffic), so:
//  * tanh is a polynomial on the fp32 pipe in packed pairs wherever a warp's arguments allow:
//    tanh t = t P(t^2) with P of degree 3, fitted to the least relative error for |t| <= 1/2
//    (5.8e-7 evaluated in fp32; weighted least squares on Chebyshev nodes, weights iterated
//    towards the equal-ripple fit), the scale and the cap folded into its coefficients. A score
//    is then off by at most 0.47 cap * 5.8e-7, 1.4e-5 for a cap of 50, against the 2^-11 by
//    which the fp16 probability is rounded. A warp with a larger argument among its 64 columns
//    takes 1 - 2 / (1 + e^2t) for them.
//  * The bias is linear in the key's column wherever no key of the tile lies past its query:
//    slope * column joins the score in the instruction that scales it, the rest of the bias
//    is one number per row and tile.
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
// below 2^15 until then, which fp16 holds as precisely as any, and a tile's row sum of at most
// 2^15 shows that none passed.
constexpr float kScoredSlack = 15.f;  // log2 units
constexpr float kScoredSlackBound = 32768.f;

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

// v = cap_out * tanh(v * cap_in); reload() puts the raw v back. Warp-collective.
template <class Reload>
__device__ __forceinline__ void cap_scores(float (&v)[64], const ScoreArgs &s, Reload reload) {
  float top[4] = {0.f, 0.f, 0.f, 0.f};
  const float2 c0 = make_float2(s.cap_poly[0], s.cap_poly[0]),
               c1 = make_float2(s.cap_poly[1], s.cap_poly[1]),
               c2 = make_float2(s.cap_poly[2], s.cap_poly[2]),
               c3 = make_float2(s.cap_poly[3], s.cap_poly[3]);
#pragma unroll
  for (int c = 0; c < 64; c += 2) {
    const float2 x = make_float2(v[c], v[c + 1]);
    const float2 z = fmul2(x, x);
    top[(c >> 1) & 3] = max3(top[(c >> 1) & 3], z.x, z.y);
    float2 p = ffma2(c3, z, c2);
    p = ffma2(p, z, c1);
    p = ffma2(p, z, c0);
    p = fmul2(p, x);
    v[c] = p.x;
    v[c + 1] = p.y;
  }
  const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  if (__builtin_expect(__any_sync(0xffffffffu, !(most <= s.cap_poly_max)), 0)) {
    reload();
    // e^2t overflows to infinity and underflows to 0 where tanh is +-1
#pragma unroll
    for (int c = 0; c < 64; ++c) {
      const float e = prefill_exp2(v[c] * (s.cap_in * (2.f * kLog2e)));
      v[c] = fmaf(-2.f * s.cap_out, fast_rcp(1.f + e), s.cap_out);
    }
  }
}

// From raw dot products to base-2 scores: afterwards the score of column c is
// v[c] * mult + offset. `base` is the columns' first token. Warp-collective.
template <class Reload>
__device__ __forceinline__ void rule_scores(float (&v)[64], const ScoreArgs &s, float scale_log2,
                                            const ScoredRow &row, int base, Reload reload,
                                            float &mult, float &offset) {
  mult = scale_log2;
  offset = 0.f;
  if (s.cap_in != 0.f) {
    cap_scores(v, s, reload);
    mult = 1.f;
  }
  if (s.slopes) {
    const int rel = base - row.pos;
    const float2 m2 = make_float2(mult, mult);
    if (__builtin_expect(__all_sync(0xffffffffu, rel + 63 <= 0), 1)) {
      // the empty asm keeps the biases of all columns, the same for every tile, from being
      // kept in registers across tiles
      float sl = row.slope2;
      asm volatile("" : "+f"(sl));
      const float2 slope = make_float2(sl, sl);
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        const float2 bias = fmul2(slope, make_float2(static_cast<float>(c), static_cast<float>(c + 1)));
        const float2 x = ffma2(make_float2(v[c], v[c + 1]), m2, bias);
        v[c] = x.x;
        v[c + 1] = x.y;
      }
      offset = row.slope2 * static_cast<float>(rel);
    } else {
      // keys on both sides of the query: the distance of each
      const float first = static_cast<float>(rel);
#pragma unroll
      for (int c = 0; c < 64; ++c)
        v[c] = fmaf(-row.slope2, fabsf(first + static_cast<float>(c)), v[c] * mult);
    }
    mult = 1.f;
  }
}

// One tile of TN keys from token `base`: raw dot products become weights relative to row.m,
// row.l grows by their sum. Warp-collective. `load(h, v)` reads raw columns 64 h .. 64 h + 63,
// again when asked again; `emit(h, pk)` takes their weights as fp16 pairs once they stand (all
// loads come before the first emit); `rescale(f)` multiplies the row's accumulated output by f
// (only called when `later`, a tile after the row's first; false from it: a wait gave up).
//
// As in the causal kernels a later tile takes its exponents with the maximum as it stands and
// checks them by their sum; a first tile, and one whose check fails in some row of the warp,
// is gone through for its maximum first. A row that has seen nothing yet (m = -inf) takes its
// maximum as soon as a tile holds a token it sees.
//
// The columns are taken 64 at a time by one loop body that serves both walks. Whole rows of 128
// scores beside their weights do not fit a thread's registers (a spilled word is an L2 access
// here, the shared memory being full), and the body unrolled over both parts and both walks
// outgrew the instruction cache: the softmax warps spent most of their time fetching (6900
// cycles a tile against 2500 of the causal form's).
template <int TN, class Load, class Emit, class Rescale>
__device__ __forceinline__ bool scored_weights(const ScoreArgs &s, float scale_log2,
                                               ScoredRow &row, int base, bool later, Load load,
                                               Emit emit, Rescale rescale) {
  constexpr int H = TN / 64;
  const int lo = row.lo - base, hi = row.hi - base;
  const bool some = hi >= 0 && lo < TN && lo <= hi;
  float pk[H][32];
  if (!__any_sync(0xffffffffu, some)) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
#pragma unroll
      for (int e = 0; e < 32; ++e) pk[h][e] = 0.f;
      emit(h, pk[h]);
    }
    return true;
  }
  const bool full = __all_sync(0xffffffffu, lo <= 0 && hi >= TN - 1);
  bool find = !later;  // whether the next walk looks for the maximum
  float sum;
  for (bool last = find;;) {
    const float nm = row.m == -INFINITY ? 0.f : -row.m;
    float mx = -INFINITY;
    float rp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int h = 0; h < H; ++h) {
      float v[64], mult, offset;
      load(h, v);
      rule_scores(v, s, scale_log2, row, base + 64 * h, [&] { load(h, v); }, mult, offset);
      const float sign = mult >= 0.f ? 1.f : -1.f;
      if (!full) {
        const float none = -sign * INFINITY;
        const int l = lo - 64 * h, r = hi - 64 * h;
#pragma unroll
        for (int c = 0; c < 64; ++c) v[c] = c >= l && c <= r ? v[c] : none;
      }
      if (find) {
        // the maximum of the scores is the extreme of v times mult (the maximum for mult >= 0)
        float mp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 64; ++c) mp[c & 3] = fmaxf(mp[c & 3], v[c] * sign);
        const float ext = fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3]));
        if (ext > -INFINITY) mx = fmaxf(mx, fmaf(ext, mult * sign, offset));
      } else {
        if (H > 1 && h > 0) {
#pragma unroll
          for (int e = 0; e < 32; ++e) pk[0][e] = pk[H - 1][e];
        }
        const float2 m2 = make_float2(mult, mult), n2 = make_float2(offset + nm, offset + nm);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int c = 2 * e;
          const float2 x = ffma2(make_float2(v[c], v[c + 1]), m2, n2);
          const float2 w = make_float2(prefill_exp2(x.x), prefill_exp2(x.y));
          const float2 acc = fadd2(make_float2(rp[c & 2], rp[(c & 2) + 1]), w);
          rp[c & 2] = acc.x;
          rp[(c & 2) + 1] = acc.y;
          pk[H - 1][e] = __uint_as_float(pack_half2(w.x, w.y));
        }
      }
    }
    if (find) {
      const bool grow = mx > row.m + kScoredSlack;
      if (__any_sync(0xffffffffu, grow)) {
        const float mnew = grow ? mx : row.m;
        const float f = mnew == -INFINITY ? 1.f : prefill_exp2(row.m - mnew);
        row.l *= f;
        if (later && !rescale(f)) return false;
        row.m = mnew;
      }
      find = false;
      last = true;
      continue;
    }
    sum = (rp[0] + rp[1]) + (rp[2] + rp[3]);
    if (last || __all_sync(0xffffffffu, sum <= kScoredSlackBound &&
                                            !(some && row.m == -INFINITY)))
      break;
    find = true;
  }
  row.l += sum;
#pragma unroll
  for (int h = 0; h < H; ++h) emit(h, pk[h]);
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
