// append_quant.cu -- several new K/V rows per sequence written into quantised paged caches, queries
// and keys normed head by head and rotated by position on the way (pa_append_quant), and rows read
// back from them (pa_read_quant).
//
// Mathematics: a query or key row x becomes x / sqrt(mean(x^2) + eps) * w, its pairs (x, y) then
// (x c - y s, x s + y c); a query is rounded once to fp16, a key or value row to the codes of
// quant.cuh, each the nearest to the exact value. Everything is computed in fp32 with a bound of the
// error; where that leaves a key's code or its row's scale open, the warp computes its keys again in
// pairs of fp32 (a value and its error, 2^-44 or so). Of normal keys one normed or turned element in
// 2^11.5 is left open, so 15 warps of a hundred compute twice; keys that are neither are exact.
// Bound: HBM. A token reads (query_heads + 2 kv_heads) * head_dim fp16 and writes query_heads *
// head_dim fp16 and 2 kv_heads * (head_dim + 1) bytes.
#include <algorithm>
#include <cmath>

#include "early_launch.cuh"
#include "new_rows.cuh"
#include "quant.cuh"

namespace pa {

struct AppendQuantArgs : RopeArgs {
  const float *q_weight, *k_weight;  // either may be null: its rows are not normed
  float eps;
  uint8_t *k_scale, *v_scale;
};

// A sum of two floats: the value and what rounding it left.
struct Pair {
  float h, l;
};

__device__ __forceinline__ Pair product(float a, float b) {
  Pair r;
  r.h = __fmul_rn(a, b);
  r.l = __fmaf_rn(a, b, -r.h);
  return r;
}

__device__ __forceinline__ Pair sum(float a, float b) {
  Pair r;
  r.h = __fadd_rn(a, b);
  const float t = __fsub_rn(r.h, a);
  r.l = __fadd_rn(__fsub_rn(a, __fsub_rn(r.h, t)), __fsub_rn(b, t));
  return r;
}

// The float nearest to odd: of the two floats around h + l the one with an odd last bit, so that
// rounding it again to fewer bits gives what rounding h + l itself would.
__device__ __forceinline__ float to_odd(Pair x) {
  const float h = __fadd_rn(x.h, x.l);
  const float l = __fadd_rn(__fsub_rn(x.h, h), x.l);
  uint32_t b = __float_as_uint(h);
  if (l != 0.f && !(b & 1u)) b += (l > 0.f) == (h > 0.f) ? 1u : 0xffffffffu;
  return __uint_as_float(b);
}

// 1 / sqrt(m): an approximation and one Newton step, whose residual 1 - m r^2 is exact enough to
// leave 2^-44.
__device__ __forceinline__ Pair inverse_root(Pair m) {
  Pair r;
  r.h = rsqrtf(m.h);
  const Pair g = product(r.h, r.h);
  const Pair t = product(m.h, g.h);
  const float rest = __fmaf_rn(m.h, g.l, __fmaf_rn(m.l, g.h, t.l));
  r.l = r.h * (0.5f * (__fsub_rn(1.f, t.h) - rest));
  return r;
}

// a * b for pairs.
__device__ __forceinline__ Pair times(Pair a, Pair b) {
  Pair r = product(a.h, b.h);
  r.l = __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, r.l));
  return r;
}

// a * c - b * s.
__device__ __forceinline__ Pair turned(Pair a, float c, Pair b, float s) {
  const Pair p = product(a.h, c), q = product(b.h, s);
  Pair r = sum(p.h, -q.h);
  r.l += __fmaf_rn(a.l, c, p.l) - __fmaf_rn(b.l, s, q.l);
  return r;
}

// Two floats at a time.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mov.b64 rc, {%6, %7};\n\tfma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Largest magnitude of 16 values.
__device__ __forceinline__ float top16(const float (&v)[16]) {
  float t = max3(fabsf(v[0]), fabsf(v[1]), fabsf(v[2]));
#pragma unroll
  for (int e = 3; e < 15; e += 2) t = max3(t, fabsf(v[e]), fabsf(v[e + 1]));
  return fmaxf(t, fabsf(v[15]));
}

// Places of an item's 16 elements: element e of the first chunk pairs with element e of the second
// (half style), or 2 e with 2 e + 1 of the 16 (interleaved).
template <bool kInterleaved>
__device__ __forceinline__ int first_of_pair(int e) { return kInterleaved ? 2 * e : e; }
template <bool kInterleaved>
__device__ __forceinline__ int second_of_pair(int e) { return kInterleaved ? 2 * e + 1 : e + 8; }

__device__ __forceinline__ void floats16(const uint4 &x, const uint4 &y, float (&v)[16]) {
  const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 p = half2_bits_to_float2(w[e]);
    v[2 * e] = p.x;
    v[2 * e + 1] = p.y;
  }
}

// Turns an item's eight pairs.
template <bool kInterleaved>
__device__ __forceinline__ void turn16(float (&v)[16], const float (&cs)[8], const float (&sn)[8]) {
  if constexpr (kInterleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = v[2 * e], q = v[2 * e + 1];
      v[2 * e] = p * cs[e] - q * sn[e];
      v[2 * e + 1] = p * sn[e] + q * cs[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 p = make_float2(v[e], v[e + 1]), q = make_float2(v[8 + e], v[9 + e]);
      const float2 c = make_float2(cs[e], cs[e + 1]), s = make_float2(sn[e], sn[e + 1]);
      const float2 f = fma2(make_float2(-q.x, -q.y), s, mul2(p, c)), g = fma2(p, s, mul2(q, c));
      v[e] = f.x;
      v[e + 1] = f.y;
      v[8 + e] = g.x;
      v[9 + e] = g.y;
    }
  }
}

// v *= r * w.
__device__ __forceinline__ void scale16(float (&v)[16], float r, const float (&w)[16]) {
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const float2 x = mul2(make_float2(v[e], v[e + 1]),
                          mul2(make_float2(r, r), make_float2(w[e], w[e + 1])));
    v[e] = x.x;
    v[e + 1] = x.y;
  }
}

// 16 norm weights of an item's chunks.
__device__ __forceinline__ void weights16(const float *w, int off_x, int off_y, float (&v)[16]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float4 f = __ldg(reinterpret_cast<const float4 *>(w + (c < 2 ? off_x : off_y)) + (c & 1));
    v[4 * c] = f.x;
    v[4 * c + 1] = f.y;
    v[4 * c + 2] = f.z;
    v[4 * c + 3] = f.w;
  }
}

// Inverse root mean square of a head's row, from the squares of a lane's 16 elements (those of fp16
// numbers are exact in fp32); HD / 16 neighbouring lanes share the row. Warp-collective.
template <int HD>
__device__ __forceinline__ Pair inverse_rms(const float (&v)[16], float eps) {
  Pair s = {0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const Pair t = sum(s.h, v[e] * v[e]);
    s.h = t.h;
    s.l += t.l;
  }
#pragma unroll
  for (int o = 1; o < HD / 16; o <<= 1) {
    const Pair t = sum(s.h, __shfl_xor_sync(0xffffffffu, s.h, o));
    s.l = t.l + (s.l + __shfl_xor_sync(0xffffffffu, s.l, o));
    s.h = t.h;
  }
  Pair m = sum(s.h * (1.f / HD), eps);
  m.l += s.l * (1.f / HD);
  return inverse_root(m);
}

// A lane's 16 elements (x, y) of key rows, normed and turned in pairs of fp32, each rounded to odd:
// rounding them again to codes gives the codes nearest to the exact values; elements of value rows, and
// of keys that are neither normed nor turned here, stay as they are. Gives the codes and the row's exponent. A call of its own: what it needs of registers
// would halve the warps of the kernel, which takes this way for few rows. Warp-collective.
template <int HD, bool kInterleaved, bool kNorm>
__device__ __noinline__ int exact_codes(uint4 x, uint4 y, const float *weight, float eps, bool is_k,
                                        int off_x, int off_y, const float *angles, int sines,
                                        uint32_t *codes) {
  float v[16];
  floats16(x, y, v);
  Pair norm = {1.f, 0.f};
  if constexpr (kNorm) norm = inverse_rms<HD>(v, eps);
  const bool normed = kNorm && weight;
  if (is_k && (normed || angles)) {
    float w[16];
    if (normed) weights16(weight, off_x, off_y, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float &p = v[first_of_pair<kInterleaved>(e)], &q = v[second_of_pair<kInterleaved>(e)];
      Pair u = {p, 0.f}, z = {q, 0.f};
      if (normed) {
        u = product(p, w[first_of_pair<kInterleaved>(e)]);
        z = product(q, w[second_of_pair<kInterleaved>(e)]);
      }
      const float c = angles ? angles[e] : 1.f, s = angles ? angles[sines + e] : 0.f;
      Pair f = turned(u, c, z, s);
      Pair g = turned(u, s, z, -c);
      if (normed) {
        f = times(f, norm);
        g = times(g, norm);
      }
      p = to_odd(f);
      q = to_odd(g);
    }
  }
  float top = top16(v);
#pragma unroll
  for (int o = 1; o < HD / 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int e = row_exponent(top);
  uint32_t c[4];
  codes16(v, e, c);
#pragma unroll
  for (int k = 0; k < 4; ++k) codes[k] = c[k];
  return e;
}

// Inverse root mean square of a head's row in fp32, off by at most 10 * 2^-24 of itself: 13
// additions, halved by the root, two roundings, and the two units of rsqrtf. Warp-collective.
template <int HD>
__device__ __forceinline__ float row_rsqrt(const float (&v)[16], float eps) {
  float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const float2 x = make_float2(v[e], v[e + 1]);
    s2 = fma2(x, x, s2);
  }
  float s = s2.x + s2.y;
#pragma unroll
  for (int o = 1; o < HD / 16; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return rsqrtf(fmaf(s, 1.f / HD, eps));
}

// A query's item: normed and turned in fp32, rounded to fp16. Warp-collective.
template <int HD, bool kInterleaved, bool kNorm>
__device__ __forceinline__ void query_item(uint4 &x, uint4 &y, const float *weight, float eps,
                                           int off_x, int off_y, bool turns, const float (&cs)[8],
                                           const float (&sn)[8]) {
  float v[16];
  floats16(x, y, v);
  if constexpr (kNorm) {
    if (weight) {
      const float r = row_rsqrt<HD>(v, eps);
      float w[16];
      weights16(weight, off_x, off_y, w);
      scale16(v, r, w);
    }
  }
  if (turns) turn16<kInterleaved>(v, cs, sn);
  uint32_t o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = pack_half2(v[2 * e], v[2 * e + 1]);
  x = make_uint4(o[0], o[1], o[2], o[3]);
  y = make_uint4(o[4], o[5], o[6], o[7]);
}

// What a thread knows of its place in a row: its item, the offsets of its two chunks in query and key
// rows, the angles of its pairs, and what a key's error is bounded by: an element of a pair (x, y) is off
// by at most (|x| + |y|) * bound / 2, for 16 roundings of 2^-24 at the most, of products with cosines and
// sines of up to bound / 2^-19. (Elements that are neither normed nor turned have no error.)
struct Item {
  int i, off_x, off_y;
  bool turns, apart;
  float cs[8], sn[8], bound;

  __device__ __forceinline__ Item(const AppendQuantArgs &a, int index, bool interleaved) {
    i = index;
    turns = i < a.rotary >> 4;
    apart = !interleaved && turns;
    off_x = apart ? i * 8 : i * 16;
    off_y = apart ? i * 8 + a.rotary / 2 : i * 16 + 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cs[e] = 1.f;
      sn[e] = 0.f;
    }
  }
  __device__ __forceinline__ void bounds() {
    float steep = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) steep = max3(steep, fabsf(cs[e]), fabsf(sn[e]));
    bound = steep * 0x1p-19f;
  }
};

constexpr int kThreadsPerSm = 768;  // what the kernel's registers leave room for

// Key or value head n (values after all keys; dead where there is none) of the token at (page, slot):
// its codes and its scale. `angles`: the cosines of the thread's pairs, sines rotary / 2 further.
// Warp-collective.
template <int HD, bool kInterleaved, bool kNorm>
__device__ __forceinline__ void write_kv(const AppendQuantArgs &a, const Item &it, uint4 kx, uint4 ky,
                                         int n, bool live, int page, int slot,
                                         const float *angles) {
  constexpr int IPR = HD / 16;
  const int i = it.i, off_x = it.off_x, off_y = it.off_y;
  const bool turns = it.turns, apart = it.apart, is_k = n < a.kvh;
  const bool normed = kNorm && is_k && a.k_weight;
  // fp16 numbers as they came lie between two codes (one in 128) or do not, but are not open: left so,
  // they sent 95 of a hundred warps the careful way, a quarter of heads of 256 turned, none normed
  const float bound = turns || normed ? it.bound : 0.f;
  float v[16], err[8];  // values; their pairs' error bounds
  floats16(kx, ky, v);
  float far = 0.f, top;
  int e;
  uint32_t c[4];
  if (__any_sync(0xffffffffu, is_k)) {
#pragma unroll
    for (int k = 0; k < 8; ++k) err[k] = 0.f;
    float inv = 1.f;
    if constexpr (kNorm) inv = row_rsqrt<HD>(v, a.eps);
    if (is_k) {
      if (normed) {
        float w[16];
        weights16(a.k_weight, off_x, off_y, w);
        scale16(v, inv, w);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        err[k] = fabsf(v[first_of_pair<kInterleaved>(k)]) + fabsf(v[second_of_pair<kInterleaved>(k)]);
        far = fmaxf(far, err[k]);
      }
      if (turns) turn16<kInterleaved>(v, it.cs, it.sn);
    }
    top = top16(v);
#pragma unroll
    for (int o = 1; o < IPR; o <<= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      far = fmaxf(far, __shfl_xor_sync(0xffffffffu, far, o));
    }
    e = row_exponent(top);
    // (the largest exponent, which clamps, is left to the careful way too)
    bool open = row_exponent(fmaf(far, bound, top)) != row_exponent(fmaf(far, -bound, top)) ||
                e == kMaxExp;
    uint32_t low[4];
    float hi[16], lo[16];
    const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23), d = f * bound;
    const float2 f2 = make_float2(f, f);
    if constexpr (kInterleaved) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 x = make_float2(v[2 * k], v[2 * k + 1]);
        const float z = err[k] * d;
        const float2 h = fma2(x, f2, make_float2(z, z)), l = fma2(x, f2, make_float2(-z, -z));
        hi[2 * k] = h.x;
        hi[2 * k + 1] = h.y;
        lo[2 * k] = l.x;
        lo[2 * k + 1] = l.y;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float2 z = mul2(make_float2(err[k], err[k + 1]), make_float2(d, d));
        const float2 m = make_float2(-z.x, -z.y);
#pragma unroll
        for (int half = 0; half < 16; half += 8) {
          const float2 x = make_float2(v[half + k], v[half + k + 1]);
          const float2 h = fma2(x, f2, z), l = fma2(x, f2, m);
          hi[half + k] = h.x;
          hi[half + k + 1] = h.y;
          lo[half + k] = l.x;
          lo[half + k + 1] = l.y;
        }
      }
    }
    pack_codes(hi, c);
    pack_codes(lo, low);
    open = open || ((c[0] ^ low[0]) | (c[1] ^ low[1]) | (c[2] ^ low[2]) | (c[3] ^ low[3])) != 0;
    if (__any_sync(0xffffffffu, open)) {
      uint32_t codes[4];
      e = exact_codes<HD, kInterleaved, kNorm>(kx, ky, a.k_weight, a.eps, is_k, off_x, off_y,
                                               turns ? angles : nullptr, a.rotary / 2, codes);
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = codes[k];
    }
  } else {
    top = top16(v);
#pragma unroll
    for (int o = 1; o < IPR; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    e = row_exponent(top);
    codes16(v, e, c);
  }
  if (live) {
    const int kv = is_k ? n : n - a.kvh;
    const long long at = a.layout == PA_LAYOUT_HEAD_MAJOR
                             ? (static_cast<long long>(page) * a.kvh + kv) * a.ps + slot
                             : (static_cast<long long>(page) * a.ps + slot) * a.kvh + kv;
    uint8_t *dst = static_cast<uint8_t *>(is_k ? a.k_cache : a.v_cache) + at * HD;
    if (is_k && apart) {
      *reinterpret_cast<uint2 *>(dst + off_x) = make_uint2(c[0], c[1]);
      *reinterpret_cast<uint2 *>(dst + off_y) = make_uint2(c[2], c[3]);
    } else {
      *reinterpret_cast<uint4 *>(dst + i * 16) = make_uint4(c[0], c[1], c[2], c[3]);
    }
    if (i == 0)
      (is_k ? a.k_scale : a.v_scale)[scale_place(page, kv, slot, a.kvh, a.ps)] =
          static_cast<uint8_t>(e + kScaleBias);
  }
}

// A CTA takes one row. A head row is HD / 16 items of two 16-byte chunks, paired as in append_rope_kernel;
// a thread keeps its item index and walks query heads, then key and value heads, and asks for the next
// item before it works on one. All warps look up the row's place, and the first query and key or value
// item are asked for before that: no address of them depends on the sequence that the row is of. That
// chain of offsets, length, page and angles is half of a row's time, so the rows in flight count: CTAs of
// 64 threads, twelve a multiprocessor, unless the rows are so few that all of them are in flight as CTAs
// of 256 (launch_append_quant_as). Rows that share a CTA, prefetched through shared memory, saved
// instructions and cost warps: 83.6 us against 78.4 then for eight prompts of 2048 tokens, 32/8 heads of
// 128, now 79.3 to 80. That is 0.69 of the copy bandwidth; the instructions of norm, rotation, error bound and rounding set it.
template <int HD, bool kInterleaved, bool kNorm, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreadsPerSm / kThreads)
    append_quant_kernel(const __grid_constant__ AppendQuantArgs a) {
  constexpr int IPR = HD / 16;
  wait_for_stream();
  const long long row = blockIdx.x;
  Item it(a, threadIdx.x % IPR, kInterleaved);
  const int nq = a.q ? a.qh : 0, nkv = 2 * a.kvh;
  const int step = blockDim.x / IPR, slot0 = threadIdx.x / IPR;
  auto load_q = [&](int h, uint4 &x, uint4 &y) {  // plain: query_out may be the query buffer itself
    if (h >= nq) return;
    const uint16_t *src = a.q + row * a.q_stride + static_cast<long long>(h) * HD;
    x = *reinterpret_cast<const uint4 *>(src + it.off_x);
    y = *reinterpret_cast<const uint4 *>(src + it.off_y);
  };
  auto load_kv = [&](int n, uint4 &x, uint4 &y) {
    if (n >= nkv) return;
    const bool is_k = n < a.kvh;
    const uint16_t *src =
        is_k ? a.k + row * a.k_stride + n * HD : a.v + row * a.v_stride + (n - a.kvh) * HD;
    x = __ldg(reinterpret_cast<const uint4 *>(src + (is_k ? it.off_x : it.i * 16)));
    y = __ldg(reinterpret_cast<const uint4 *>(src + (is_k ? it.off_y : it.i * 16 + 8)));
  };
  uint4 qx = make_uint4(0, 0, 0, 0), qy = qx, kx = qx, ky = qx;
  load_q(slot0, qx, qy);
  load_kv(slot0, kx, ky);

  check_sequences(a);
  const int b = sequence_of_row(a, static_cast<int>(row));
  if (b < 0) return;
  int t, page, pos;
  if (!place_of_row(a, b, static_cast<int>(row), t, page, pos, threadIdx.x == 0)) return;
  if (it.turns) load_angles(a, pos, it.i, it.cs, it.sn);
  it.bounds();

  // a warp's lanes walk together, so that those past the last head take part in the shuffles
  const int first = (threadIdx.x & ~31) / IPR;
#pragma unroll 1
  for (int w0 = first, h = slot0; w0 < nq; w0 += step, h += step) {
    uint4 x = qx, y = qy;
    load_q(h + step, qx, qy);
    query_item<HD, kInterleaved, kNorm>(x, y, a.q_weight, a.eps, it.off_x, it.off_y, it.turns, it.cs,
                                        it.sn);
    if (h < nq) {
      uint16_t *dst = a.q_out + (row * a.qh + h) * HD;
      *reinterpret_cast<uint4 *>(dst + it.off_x) = x;
      *reinterpret_cast<uint4 *>(dst + it.off_y) = y;
    }
  }
  const float *turn = a.table + static_cast<long long>(pos) * a.rotary + it.i * 8;
#pragma unroll 1
  for (int w0 = first, n = slot0; w0 < nkv; w0 += step, n += step) {
    const uint4 x = kx, y = ky;
    load_kv(n + step, kx, ky);
    write_kv<HD, kInterleaved, kNorm>(a, it, x, y, n, n < nkv, page, t & (a.ps - 1), turn);
  }
}

struct ReadQuantArgs : NewRowsArgs {
  const uint8_t *k, *v, *k_scale, *v_scale;
  uint16_t *k_out, *v_out;  // packed rows; either may be null
};

constexpr int kReadRows = 8;  // rows of a CTA: one for each of its warps to place

// A CTA places eight rows, a warp each, and then all its threads stream their heads: an item is 16
// codes and 32 bytes of fp16. Bound: HBM, a byte read for two written: 473 MB of 32 sequences (8 heads of
// 128) in 75.9 us, 0.93 of the copy bandwidth.
template <int HD>
__global__ void __launch_bounds__(kReadRows * 32)
    read_quant_kernel(const __grid_constant__ ReadQuantArgs a) {
  constexpr int IPR = HD / 16;
  __shared__ int s_page[kReadRows], s_slot[kReadRows];
  wait_for_stream();
  check_sequences(a);
  const int warp = threadIdx.x >> 5;
  const long long row0 = static_cast<long long>(blockIdx.x) * kReadRows;
  int page = -1, slot = 0;
  if (row0 + warp < a.total) {
    const int row = static_cast<int>(row0) + warp;
    const int b = sequence_of_row(a, row);
    if (b >= 0) {
      const int t = __ldg(a.ctx + b) - __ldg(a.qs + b + 1) + row;
      page = __ldg(a.bt + static_cast<long long>(b) * a.maxp + (t >> a.ps_shift));
      slot = t & (a.ps - 1);
      if (page < 0 || page >= a.num_pages) {
        if ((threadIdx.x & 31) == 0) atomicOr(a.err, PA_DEVERR_PAGE_ID);
        page = -1;
      }
    }
  }
  if ((threadIdx.x & 31) == 0) {
    s_page[warp] = page;
    s_slot[warp] = slot;
  }
  __syncthreads();
  const int per_row = a.kvh * IPR;  // items of a row of one cache
  const int parts = (a.k_out ? 1 : 0) + (a.v_out ? 1 : 0);
  const int items = kReadRows * per_row * parts;
#pragma unroll 4
  for (int n = threadIdx.x; n < items; n += kReadRows * 32) {
    const int line = n / per_row, item = n - line * per_row;
    const int r = line / parts;
    const bool is_v = !a.k_out || line - r * parts == 1;
    if (s_page[r] < 0) continue;
    const int kv = item / IPR, i = item % IPR;
    const long long at =
        a.layout == PA_LAYOUT_HEAD_MAJOR
            ? (static_cast<long long>(s_page[r]) * a.kvh + kv) * a.ps + s_slot[r]
            : (static_cast<long long>(s_page[r]) * a.ps + s_slot[r]) * a.kvh + kv;
    const uint4 c = __ldg(reinterpret_cast<const uint4 *>((is_v ? a.v : a.k) + at * HD) + i);
    const uint32_t e = __ldg((is_v ? a.v_scale : a.k_scale) +
                             scale_place(s_page[r], kv, s_slot[r], a.kvh, a.ps));
    const uint32_t f = half2_of_scales(e, e);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      o[2 * k] = mul_half2(half2_of_low(w[k]), f);
      o[2 * k + 1] = mul_half2(half2_of_high(w[k]), f);
    }
    uint4 *dst = reinterpret_cast<uint4 *>((is_v ? a.v_out : a.k_out) +
                                           ((row0 + r) * a.kvh + kv) * HD + i * 16);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

namespace {

bool off_by(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

template <int HD, bool kInterleaved, bool kNorm, int kThreads>
cudaError_t launch_append_quant_threads(const AppendQuantArgs &a, cudaStream_t stream) {
  constexpr int IPR = HD / 16;
  const int heads = std::max(a.q ? a.qh : 0, 2 * a.kvh);
  const int threads = std::min(kThreads, (heads * IPR + 31) / 32 * 32);
  return launch_early(append_quant_kernel<HD, kInterleaved, kNorm, kThreads>,
                      dim3(static_cast<unsigned>(a.total)), threads, 0, stream, a);
}

// Captured calls, with CTAs of 256 threads and of 64: 256 rows of 64/8 heads of 128 6.7 and 7.9 us; 456
// rows of 32/8 heads 6.9 and 7.1, 600 (past the rule) 9.5 and 7.5, 1000 12.1 and 9.3; 3300 rows of 24/4
// heads of 256, a quarter turned and nothing normed, 26.7 and 18.5.
template <int HD, bool kInterleaved, bool kNorm>
cudaError_t launch_append_quant_as(const AppendQuantArgs &a, cudaStream_t stream) {
  return a.total <= static_cast<long long>(device_sm_count()) * (kThreadsPerSm / 256)
             ? launch_append_quant_threads<HD, kInterleaved, kNorm, 256>(a, stream)
             : launch_append_quant_threads<HD, kInterleaved, kNorm, 64>(a, stream);
}

template <int HD>
cudaError_t launch_append_quant(const AppendQuantArgs &a, cudaStream_t stream) {
  if (a.q_weight || a.k_weight)
    return a.interleaved ? launch_append_quant_as<HD, true, true>(a, stream)
                         : launch_append_quant_as<HD, false, true>(a, stream);
  return a.interleaved ? launch_append_quant_as<HD, true, false>(a, stream)
                       : launch_append_quant_as<HD, false, false>(a, stream);
}

}  // namespace

pa_status_t check_quant_cache(const pa_quant_cache_t *c) {
  if (!c || !c->key || !c->value || !c->key_scale || !c->value_scale) return PA_ERR_INVALID_ARG;
  if (off_by(c->key, 16) || off_by(c->value, 16) || off_by(c->key_scale, 16) ||
      off_by(c->value_scale, 16))
    return PA_ERR_MISALIGNED;
  return PA_OK;
}

}  // namespace pa

extern "C" pa_status_t pa_append_quant(const pa_problem_t *problem, const pa_norm_t *norm,
                                       const pa_rope_t *rope, const void *query,
                                       int64_t query_stride, const void *new_key,
                                       int64_t key_stride, const void *new_value,
                                       int64_t value_stride, const int32_t *query_start,
                                       int64_t total_tokens, const int32_t *block_tables,
                                       const int32_t *context_lengths, void *query_out,
                                       const pa_quant_cache_t *cache, void *stream) {
  using namespace pa;
  pa_status_t st = check_problem_public(problem);
  if (st != PA_OK) return st;
  st = check_quant_cache(cache);
  if (st != PA_OK) return st;
  AppendQuantArgs a = {};
  if (norm) {
    if (norm->reserved != 0 || !(norm->eps >= 1e-30f && norm->eps <= 1e30f))
      return PA_ERR_INVALID_ARG;
    if (off_by(norm->query_weight, 16) || off_by(norm->key_weight, 16)) return PA_ERR_MISALIGNED;
    a.q_weight = norm->query_weight;
    a.k_weight = norm->key_weight;
    a.eps = norm->eps;
  }
  st = resolve_new_rows(problem, rope, query, query_stride, new_key, key_stride, new_value,
                        value_stride, query_start, total_tokens, block_tables, context_lengths,
                        query_out, cache->key, cache->value, &a);
  if (st != PA_OK || a.total == 0) return st;
  a.k_scale = cache->key_scale;
  a.v_scale = cache->value_scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (problem->head_dim) {
    case 64: e = launch_append_quant<64>(a, s); break;
    case 128: e = launch_append_quant<128>(a, s); break;
    case 256: e = launch_append_quant<256>(a, s); break;
    default: return PA_ERR_UNSUPPORTED;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

extern "C" pa_status_t pa_read_quant(const pa_problem_t *problem, const pa_quant_cache_t *cache,
                                     const int32_t *query_start, int64_t total_tokens,
                                     const int32_t *block_tables, const int32_t *context_lengths,
                                     void *key_out, void *value_out, void *stream) {
  using namespace pa;
  pa_status_t st = check_problem_public(problem);
  if (st != PA_OK) return st;
  st = check_quant_cache(cache);
  if (st != PA_OK) return st;
  if (!query_start || !block_tables || !context_lengths || total_tokens < 0 ||
      total_tokens >= (int64_t(1) << 31) || (total_tokens > 0 && !key_out && !value_out))
    return PA_ERR_INVALID_ARG;
  if (off_by(query_start, 4) || off_by(block_tables, 4) || off_by(context_lengths, 4) ||
      off_by(key_out, 16) || off_by(value_out, 16))
    return PA_ERR_MISALIGNED;
  if (problem->kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  if (problem->batch == 0 || total_tokens == 0) return PA_OK;
  int smem = 0;
  st = current_device_smem(&smem);
  if (st != PA_OK) return st;
  ReadQuantArgs a = {};
  a.qs = query_start;
  a.bt = block_tables;
  a.ctx = context_lengths;
  a.err = device_error_word();
  if (!a.err) return PA_ERR_CUDA;
  a.total = total_tokens;
  a.batch = problem->batch;
  a.kvh = problem->kv_heads;
  a.ps = problem->page_size;
  while ((1 << a.ps_shift) < a.ps) ++a.ps_shift;
  a.maxp = problem->max_pages_per_sequence;
  a.num_pages = problem->num_physical_pages;
  a.layout = problem->cache_layout;
  a.k = static_cast<const uint8_t *>(cache->key);
  a.v = static_cast<const uint8_t *>(cache->value);
  a.k_scale = cache->key_scale;
  a.v_scale = cache->value_scale;
  a.k_out = static_cast<uint16_t *>(key_out);
  a.v_out = static_cast<uint16_t *>(value_out);
  const dim3 grid(static_cast<unsigned>((total_tokens + kReadRows - 1) / kReadRows));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (problem->head_dim) {
    case 64: e = launch_early(read_quant_kernel<64>, grid, kReadRows * 32, 0, s, a); break;
    case 128: e = launch_early(read_quant_kernel<128>, grid, kReadRows * 32, 0, s, a); break;
    case 256: e = launch_early(read_quant_kernel<256>, grid, kReadRows * 32, 0, s, a); break;
    default: return PA_ERR_UNSUPPORTED;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
