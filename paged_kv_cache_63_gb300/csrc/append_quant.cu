// append_quant.cu -- several new K/V rows per sequence written into quantised paged caches, queries
// and keys normed head by head and rotated by position on the way (pa_append_quant), and rows read
// back from them (pa_read_quant).
//
// Mathematics: a query or key row x becomes x / sqrt(mean(x^2) + eps) * w, its pairs (x, y) then
// (x c - y s, x s + y c); a query is rounded once to fp16, a key or value row to the codes of
// quant.cuh. Queries are computed in fp32. Keys are computed in pairs of fp32 (value and error, 2^-44
// or so) and each code is the one nearest to the exact value: in plain fp32 one key element in some
// 2^19 lies near enough to the border of two codes to fall on the wrong side.
// Bound: HBM. A token reads (query_heads + 2 kv_heads) * head_dim fp16 and writes query_heads *
// head_dim fp16 and 2 kv_heads * (head_dim + 1) bytes.
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

// One CTA per row of the packed batch, items and their pairing as in append_rope_kernel: HD / 16
// neighbouring lanes share a head's row, so its mean square and its largest element take two to
// four shuffles.
template <int HD, bool kInterleaved, bool kNorm>
__global__ void __launch_bounds__(256)
    append_quant_kernel(const __grid_constant__ AppendQuantArgs a) {
  constexpr int IPR = HD / 16;  // items per head row
  wait_for_stream();
  check_sequences(a);
  const int row = static_cast<int>(blockIdx.x);
  const int b = sequence_of_row(a, row);
  if (b < 0) return;
  int t, page, pos;
  if (!place_of_row(a, b, row, t, page, pos)) return;
  const int slot = t & (a.ps - 1);
  const int i = threadIdx.x % IPR;
  const bool turns = i < a.rotary >> 4;
  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
  }
  if (turns) load_angles(a, pos, i, cs, sn);
  const int nq = a.q ? a.qh : 0;
  const int heads = nq + 2 * a.kvh;
  const int step = blockDim.x / IPR;
  // a warp's lanes walk together, so that those past the last head take part in the shuffles
  const int first = (threadIdx.x & ~31) / IPR, mine = (threadIdx.x & 31) / IPR;
  for (int h0 = first; h0 < heads; h0 += step) {
    const int h = h0 + mine;
    const bool live = h < heads;
    const bool is_q = h < nq, is_k = !is_q && h < nq + a.kvh;
    const bool apart = !kInterleaved && turns && (is_q || is_k);
    const int off_x = apart ? i * 8 : i * 16;
    const int off_y = apart ? i * 8 + a.rotary / 2 : i * 16 + 8;
    const uint16_t *src;
    if (is_q)
      src = a.q + row * a.q_stride + static_cast<long long>(h) * HD;
    else if (is_k)
      src = a.k + row * a.k_stride + static_cast<long long>(h - nq) * HD;
    else
      src = a.v + row * a.v_stride + static_cast<long long>(h - nq - a.kvh) * HD;
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (live) {  // plain loads: query_out may be the query buffer itself
      x = *reinterpret_cast<const uint4 *>(src + off_x);
      y = *reinterpret_cast<const uint4 *>(src + off_y);
    }
    float v[16];
    floats16(x, y, v);
    const float *weight = kNorm && live ? (is_q ? a.q_weight : is_k ? a.k_weight : nullptr) : nullptr;
    Pair norm = {1.f, 0.f};
    float w[16];
    if constexpr (kNorm) {
      Pair s = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 16; ++e) {  // a square of an fp16 number is exact in fp32
        const Pair t = sum(s.h, v[e] * v[e]);
        s.h = t.h;
        s.l += t.l;
      }
#pragma unroll
      for (int o = 1; o < IPR; o <<= 1) {
        const Pair t = sum(s.h, __shfl_xor_sync(0xffffffffu, s.h, o));
        s.l = t.l + (s.l + __shfl_xor_sync(0xffffffffu, s.l, o));
        s.h = t.h;
      }
      if (weight) {
        weights16(weight, off_x, off_y, w);
        Pair m = sum(s.h * (1.f / HD), a.eps);
        m.l += s.l * (1.f / HD);
        norm = inverse_root(m);
      }
    }
    if (is_q) {
      if (weight) {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] *= norm.h * w[e];
      }
      if (turns) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float &p = v[first_of_pair<kInterleaved>(e)], &q = v[second_of_pair<kInterleaved>(e)];
          const float p0 = p, q0 = q;
          p = p0 * cs[e] - q0 * sn[e];
          q = p0 * sn[e] + q0 * cs[e];
        }
      }
      if (live) {
        uint16_t *dst = a.q_out + (static_cast<long long>(row) * a.qh + h) * HD;
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = pack_half2(v[2 * e], v[2 * e + 1]);
        *reinterpret_cast<uint4 *>(dst + off_x) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(dst + off_y) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
    if (__all_sync(0xffffffffu, is_q)) continue;
    if (is_k) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float &p = v[first_of_pair<kInterleaved>(e)], &q = v[second_of_pair<kInterleaved>(e)];
        Pair u = {p, 0.f}, z = {q, 0.f};
        if (weight) {
          u = product(p, w[first_of_pair<kInterleaved>(e)]);
          z = product(q, w[second_of_pair<kInterleaved>(e)]);
        }
        Pair f = turned(u, cs[e], z, sn[e]);
        Pair g = turned(u, sn[e], z, -cs[e]);
        if (weight) {
          f = times(f, norm);
          g = times(g, norm);
        }
        p = to_odd(f);
        q = to_odd(g);
      }
    }
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(v[e]));
#pragma unroll
    for (int o = 1; o < IPR; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!is_q && live) {
      const int e = row_exponent(top);
      uint32_t c[4];
      codes16(v, e, c);
      const int kv = is_k ? h - nq : h - nq - a.kvh;
      const long long at = a.layout == PA_LAYOUT_HEAD_MAJOR
                               ? (static_cast<long long>(page) * a.kvh + kv) * a.ps + slot
                               : (static_cast<long long>(page) * a.ps + slot) * a.kvh + kv;
      uint8_t *dst = static_cast<uint8_t *>(is_k ? a.k_cache : a.v_cache) + at * HD;
      if (apart) {
        *reinterpret_cast<uint2 *>(dst + off_x) = make_uint2(c[0], c[1]);
        *reinterpret_cast<uint2 *>(dst + off_y) = make_uint2(c[2], c[3]);
      } else {
        *reinterpret_cast<uint4 *>(dst + off_x) = make_uint4(c[0], c[1], c[2], c[3]);
      }
      if (i == 0)
        (is_k ? a.k_scale : a.v_scale)[scale_place(page, kv, slot, a.kvh, a.ps)] =
            static_cast<uint8_t>(e + kScaleBias);
    }
  }
}

struct ReadQuantArgs : NewRowsArgs {
  const uint8_t *k, *v, *k_scale, *v_scale;
  uint16_t *k_out, *v_out;  // packed rows; either may be null
};

constexpr int kReadRows = 8;  // rows of a CTA: one for each of its warps to place

// A CTA places eight rows, a warp each, and then all its threads stream their heads: an item is 16
// codes and 32 bytes of fp16. Bound: HBM, a byte read for two written.
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

template <int HD>
cudaError_t launch_append_quant(const AppendQuantArgs &a, cudaStream_t stream) {
  constexpr int IPR = HD / 16;
  const int heads = (a.q ? a.qh : 0) + 2 * a.kvh;
  const int want = heads * IPR;
  const int threads = want >= 256 ? 256 : (want + 31) / 32 * 32;
  void (*kern)(AppendQuantArgs);
  if (a.q_weight || a.k_weight)
    kern = a.interleaved ? append_quant_kernel<HD, true, true> : append_quant_kernel<HD, false, true>;
  else
    kern =
        a.interleaved ? append_quant_kernel<HD, true, false> : append_quant_kernel<HD, false, false>;
  return launch_early(kern, dim3(static_cast<unsigned>(a.total)), threads, 0, stream, a);
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
