// score_rule.cuh -- what pa_score_t adds to the attention kernels: the cap of a score by a tanh,
// the bias that grows with distance, the range of tokens a query sees, and the output's type.
#pragma once

#include <stdint.h>

#include "device_common.cuh"
#include "internal.h"

namespace pa {

constexpr float kLog2e = 1.4426950408889634f;

// tanh t = t P(t^2) for |t| <= 1/2: the coefficients of P, lowest first (scored_softmax.cuh).
constexpr double kTanhFit[4] = {0.999999463558197, -0.33326318860054016, 0.13190296292304993,
                                -0.04440222680568695};

// pa_score_t as the kernels take it.
struct ScoreArgs {
  const float *slopes;    // [query_heads] or null
  const int32_t *first;   // [query rows] or null
  const int32_t *prefix;  // [batch] or null (multi-token kernels only)
  float cap_in;           // scale / softcap: a raw dot product times this is tanh's argument; 0:
                          // no cap
  float cap_out;          // softcap * log2 e
  float cap_poly[4];      // cap_out tanh(v cap_in) ~ v (poly[0] + poly[1] v^2 + ...) for
  float cap_poly_max;     // v^2 <= cap_poly_max (multi-token kernels)
  int cap_wide;           // an error relative to the cap would show in the weights (likewise)
  int window;             // 0: no limit
  int out_half;           // output in fp16
};

// First token that the query at position pos of row `row` sees (past pos: it sees none).
__device__ __forceinline__ int first_seen(const ScoreArgs &s, long long row, int pos) {
  int lo = s.window > 0 && pos >= s.window ? pos - s.window + 1 : 0;
  if (s.first) lo = max(lo, __ldg(s.first + row));
  return lo;
}

// Elements i and i + 1 (i even) of the output in the caller's type.
__device__ __forceinline__ void store_out2(const ScoreArgs &s, void *out, long long i, float x,
                                           float y) {
  if (s.out_half)
    static_cast<uint32_t *>(out)[i >> 1] = pack_half2(x, y);
  else
    *reinterpret_cast<float2 *>(static_cast<float *>(out) + i) = make_float2(x, y);
}

// Element i of the output.
__device__ __forceinline__ void store_out1(const ScoreArgs &s, void *out, long long i, float x) {
  if (s.out_half)
    static_cast<uint16_t *>(out)[i] = __half_as_ushort(__float2half_rn(x));
  else
    static_cast<float *>(out)[i] = x;
}

// Host: checks `score` (null: none of it) and fills the kernels' form of it (decode_scored.cu).
pa_status_t resolve_score(const pa_score_t *score, float scale, ScoreArgs *s);

}  // namespace pa
