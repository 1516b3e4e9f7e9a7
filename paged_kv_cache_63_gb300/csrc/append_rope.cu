// append_rope.cu -- several new K/V rows per sequence written into the paged caches with the
// position rotation applied to the keys on the way, and the rotated queries packed for the
// attention call that follows.
//
// Mathematics: a pair (x, y) of a row at position p becomes (x c - y s, x s + y c) with
// c, s = table[p][0][i], table[p][1][i], in fp32, rounded once to fp16 (the caches' type).
// Bound: HBM. A token reads and writes (query_heads + 2 kv_heads) * head_dim fp16 and reads one
// table row; there are ~1.5 fp32 operations a byte. Eight prompts of 2048 tokens with 32/8 heads
// of 128 (404 MB) take 61.2 us, 0.97 of the copy bandwidth.
#include "device_common.cuh"
#include "early_launch.cuh"
#include "internal.h"

namespace pa {

struct RopeArgs {
  const uint16_t *q, *k, *v;  // fp16 bits; q may be null
  uint16_t *q_out, *k_cache, *v_cache;
  const float *table;
  const int32_t *positions;  // may be null
  const int32_t *qs, *bt, *ctx;
  unsigned *err;
  long long q_stride, k_stride, v_stride;  // elements
  long long total;
  int batch, qh, kvh, ps, ps_shift, maxp, num_pages, layout;
  int rotary, table_rows;
};

// The sequence that holds row `row`: the largest b in [0, batch) with query_start[b] <= row,
// or -1. One warp, 32 probes a round: two rounds for up to 1024 sequences.
__device__ __forceinline__ int find_sequence(const int32_t *qs, int batch, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;
  if (__ldg(qs) > row) return -1;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int off = lane * step;
    const bool le = off < n && __ldg(qs + lo + off) <= row;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);  // probe 0 holds
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

// Whether sequence b holds row `row` by offsets and a length that make sense.
__device__ __forceinline__ bool holds(const RopeArgs &a, int b, int row) {
  const int q0 = __ldg(a.qs + b), q1 = __ldg(a.qs + b + 1), c = __ldg(a.ctx + b);
  return q0 >= 0 && q0 <= row && row < q1 && q1 <= a.total && c <= (a.maxp << a.ps_shift) &&
         q1 - q0 <= c;
}

// The sequence that holds row `row`, or -1, by a look at every one: one wrong offset sends the
// search by halves astray for rows of other sequences. Warp-collective.
__device__ __forceinline__ int look_for_sequence(const RopeArgs &a, int row) {
#pragma unroll 1
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int b = b0 + (threadIdx.x & 31);
    const unsigned found = __ballot_sync(0xffffffffu, b < a.batch && holds(a, b, row));
    if (found) return b0 + __ffs(found) - 1;
  }
  return -1;
}

// Turns eight pairs: half style pairs element e of `a` with element e of `b`; interleaved
// style pairs elements 2e, 2e + 1 of the 16 consecutive elements a, b.
template <bool kInterleaved>
__device__ __forceinline__ void rotate16(uint4 &a, uint4 &b, const float (&c)[8],
                                         const float (&s)[8]) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if constexpr (kInterleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 p = half2_bits_to_float2(w[e]);
      w[e] = pack_half2(p.x * c[e] - p.y * s[e], p.x * s[e] + p.y * c[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = half2_bits_to_float2(w[e]), y = half2_bits_to_float2(w[4 + e]);
      const float c0 = c[2 * e], c1 = c[2 * e + 1], s0 = s[2 * e], s1 = s[2 * e + 1];
      w[e] = pack_half2(x.x * c0 - y.x * s0, x.y * c1 - y.y * s1);
      w[4 + e] = pack_half2(x.x * s0 + y.x * c0, x.y * s1 + y.y * c1);
    }
  }
  a = make_uint4(w[0], w[1], w[2], w[3]);
  b = make_uint4(w[4], w[5], w[6], w[7]);
}

// One CTA per row of the packed batch. A head row is HD / 16 items of two 16-byte chunks; a
// thread keeps its item index (so the cosines and sines it needs stay in registers) and walks
// the token's query, key and value rows. Half style: item i < rotary / 16 holds chunks i and
// i + rotary / 16 of the head, the items after them neighbouring chunks of the rest.
// Interleaved style and values: neighbouring chunks 2 i, 2 i + 1.
constexpr int kRopeUnroll = 4;

template <int HD, bool kInterleaved>
__global__ void __launch_bounds__(256) append_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int IPR = HD / 16;  // items per head row
  wait_for_stream();
  // every sequence is checked once, whichever rows it holds
  for (long long b = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; b < a.batch;
       b += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int q0 = __ldg(a.qs + b), q1 = __ldg(a.qs + b + 1), c = __ldg(a.ctx + b);
    if (c < 0 || c > (a.maxp << a.ps_shift))
      atomicOr(a.err, PA_DEVERR_CONTEXT);
    else if (q0 < 0 || q1 < q0 || q1 > a.total || q1 - q0 > c)
      atomicOr(a.err, PA_DEVERR_QUERY_START);
  }
  const int row = static_cast<int>(blockIdx.x);
  int b = find_sequence(a.qs, a.batch, row);
  if (b < 0 || !holds(a, b, row)) {
    // rows behind the last sequence, and rows of a sequence flagged above
    if (row >= __ldg(a.qs + a.batch) || (b = look_for_sequence(a, row)) < 0) return;
  }
  const int q1 = __ldg(a.qs + b + 1), c = __ldg(a.ctx + b);
  const int t = c - q1 + row;
  const int page = __ldg(a.bt + static_cast<long long>(b) * a.maxp + (t >> a.ps_shift));
  const int pos = a.rotary == 0 ? 0 : a.positions ? __ldg(a.positions + row) : t;
  const bool bad_page = page < 0 || page >= a.num_pages;
  const bool bad_pos = a.rotary > 0 && (pos < 0 || pos >= a.table_rows);
  if (bad_page || bad_pos) {
    if (threadIdx.x == 0)
      atomicOr(a.err, (bad_page ? PA_DEVERR_PAGE_ID : 0u) | (bad_pos ? PA_DEVERR_POSITION : 0u));
    return;
  }
  const int slot = t & (a.ps - 1);
  const int i = threadIdx.x % IPR;
  const int turned = a.rotary >> 4;  // items that turn
  float cs[8], sn[8];
  if (i < turned) {
    const float *tab = a.table + static_cast<long long>(pos) * a.rotary + i * 8;
    const float4 c0 = __ldg(reinterpret_cast<const float4 *>(tab));
    const float4 c1 = __ldg(reinterpret_cast<const float4 *>(tab) + 1);
    const float4 s0 = __ldg(reinterpret_cast<const float4 *>(tab + a.rotary / 2));
    const float4 s1 = __ldg(reinterpret_cast<const float4 *>(tab + a.rotary / 2) + 1);
    cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w;
    cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
    sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w;
    sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
  }
  const int heads = (a.q ? a.qh : 0) + 2 * a.kvh;
  const int step = blockDim.x / IPR;
  const int nq = a.q ? a.qh : 0;
  for (int h0 = threadIdx.x / IPR; h0 < heads; h0 += kRopeUnroll * step) {
    uint4 x[kRopeUnroll], y[kRopeUnroll];
    int off_x[kRopeUnroll], off_y[kRopeUnroll];  // element offsets of the two chunks in the row
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int h = h0 + u * step;
      if (h >= heads) break;
      const bool turn = i < turned && h < nq + a.kvh;
      const bool apart = !kInterleaved && turn;
      off_x[u] = apart ? i * 8 : i * 16;
      off_y[u] = apart ? i * 8 + a.rotary / 2 : i * 16 + 8;
      const uint16_t *src;
      if (h < nq)
        src = a.q + row * a.q_stride + static_cast<long long>(h) * HD;
      else if (h < nq + a.kvh)
        src = a.k + row * a.k_stride + static_cast<long long>(h - nq) * HD;
      else
        src = a.v + row * a.v_stride + static_cast<long long>(h - nq - a.kvh) * HD;
      // plain loads: query_out may be the query buffer itself
      x[u] = *reinterpret_cast<const uint4 *>(src + off_x[u]);
      y[u] = *reinterpret_cast<const uint4 *>(src + off_y[u]);
    }
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int h = h0 + u * step;
      if (h >= heads) break;
      if (i < turned && h < nq + a.kvh) rotate16<kInterleaved>(x[u], y[u], cs, sn);
      uint16_t *dst;
      if (h < nq) {
        dst = a.q_out + (static_cast<long long>(row) * a.qh + h) * HD;
      } else {
        const int kv = h < nq + a.kvh ? h - nq : h - nq - a.kvh;
        const long long at = a.layout == PA_LAYOUT_HEAD_MAJOR
                                 ? (static_cast<long long>(page) * a.kvh + kv) * a.ps + slot
                                 : (static_cast<long long>(page) * a.ps + slot) * a.kvh + kv;
        dst = (h < nq + a.kvh ? a.k_cache : a.v_cache) + at * HD;
      }
      *reinterpret_cast<uint4 *>(dst + off_x[u]) = x[u];
      *reinterpret_cast<uint4 *>(dst + off_y[u]) = y[u];
    }
  }
}

namespace {

bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

template <int HD>
cudaError_t launch_append_rope(const RopeArgs &a, bool interleaved, cudaStream_t stream) {
  constexpr int IPR = HD / 16;
  const int heads = (a.q ? a.qh : 0) + 2 * a.kvh;
  const int want = (heads * IPR + kRopeUnroll - 1) / kRopeUnroll;  // one walk over the heads
  const int threads = want >= 256 ? 256 : (want + 31) / 32 * 32;
  return launch_early(interleaved ? append_rope_kernel<HD, true> : append_rope_kernel<HD, false>,
                      dim3(static_cast<unsigned>(a.total)), threads, 0, stream, a);
}

}  // namespace

}  // namespace pa

extern "C" pa_status_t pa_append_rope(const pa_problem_t *problem, const pa_rope_t *rope,
                                      const void *query, int64_t query_stride,
                                      const void *new_key, int64_t key_stride,
                                      const void *new_value, int64_t value_stride,
                                      const int32_t *query_start, int64_t total_tokens,
                                      const int32_t *block_tables, const int32_t *context_lengths,
                                      void *query_out, void *key_cache, void *value_cache,
                                      void *stream) {
  using namespace pa;
  pa_status_t st = check_problem_public(problem);
  if (st != PA_OK) return st;
  if (total_tokens == 0) {  // no rows, so no addresses of any (an empty tensor's is null)
    query = new_key = new_value = key_cache;
    query_out = key_cache;
    query_stride = key_stride = value_stride = 0;
  }
  if (!new_key || !new_value || !query_start || !block_tables || !context_lengths || !key_cache ||
      !value_cache || (query == nullptr) != (query_out == nullptr))
    return PA_ERR_INVALID_ARG;
  if (total_tokens < 0 || total_tokens >= (int64_t(1) << 31)) return PA_ERR_INVALID_ARG;
  const int64_t hd = problem->head_dim;
  const int64_t q_row = problem->query_heads * hd, kv_row = problem->kv_heads * hd;
  if (query_stride == 0) query_stride = q_row;
  if (key_stride == 0) key_stride = kv_row;
  if (value_stride == 0) value_stride = kv_row;
  if ((query && query_stride < q_row) || key_stride < kv_row || value_stride < kv_row)
    return PA_ERR_INVALID_ARG;
  if (query && query_out == query && query_stride != q_row) return PA_ERR_INVALID_ARG;
  if (rope && rope->reserved != 0) return PA_ERR_INVALID_ARG;
  const int rotary = rope ? rope->rotary_dim : 0;
  if (rotary != 0) {
    if (rotary < 0 || rotary > hd || rope->style < PA_ROPE_HALF ||
        rope->style > PA_ROPE_INTERLEAVED || rope->table_rows < 1 || !rope->table)
      return PA_ERR_INVALID_ARG;
    if (rotary % 16) return PA_ERR_UNSUPPORTED;
    if (misaligned(rope->table, 16) || misaligned(rope->positions, 4)) return PA_ERR_MISALIGNED;
  }
  if (misaligned(query, 16) || misaligned(new_key, 16) || misaligned(new_value, 16) ||
      misaligned(query_out, 16) || misaligned(key_cache, 16) || misaligned(value_cache, 16) ||
      misaligned(query_start, 4) || misaligned(block_tables, 4) ||
      misaligned(context_lengths, 4) || ((query ? query_stride : 0) & 7) || (key_stride & 7) ||
      (value_stride & 7))
    return PA_ERR_MISALIGNED;
  if (problem->query_heads > 65535 || problem->kv_heads > 65535) return PA_ERR_UNSUPPORTED;
  if (problem->batch == 0 || total_tokens == 0) return PA_OK;
  int smem = 0;
  st = current_device_smem(&smem);
  if (st != PA_OK) return st;

  RopeArgs a = {};
  a.q = static_cast<const uint16_t *>(query);
  a.k = static_cast<const uint16_t *>(new_key);
  a.v = static_cast<const uint16_t *>(new_value);
  a.q_out = static_cast<uint16_t *>(query_out);
  a.k_cache = static_cast<uint16_t *>(key_cache);
  a.v_cache = static_cast<uint16_t *>(value_cache);
  a.table = rotary ? rope->table : nullptr;
  a.positions = rotary ? rope->positions : nullptr;
  a.qs = query_start;
  a.bt = block_tables;
  a.ctx = context_lengths;
  a.err = device_error_word();
  if (!a.err) return PA_ERR_CUDA;
  a.q_stride = query_stride;
  a.k_stride = key_stride;
  a.v_stride = value_stride;
  a.total = total_tokens;
  a.batch = problem->batch;
  a.qh = problem->query_heads;
  a.kvh = problem->kv_heads;
  a.ps = problem->page_size;
  while ((1 << a.ps_shift) < a.ps) ++a.ps_shift;
  a.maxp = problem->max_pages_per_sequence;
  a.num_pages = problem->num_physical_pages;
  a.layout = problem->cache_layout;
  a.rotary = rotary;
  a.table_rows = rotary ? rope->table_rows : 0;
  const bool interleaved = rotary && rope->style == PA_ROPE_INTERLEAVED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (problem->head_dim) {
    case 64: e = launch_append_rope<64>(a, interleaved, s); break;
    case 128: e = launch_append_rope<128>(a, interleaved, s); break;
    case 256: e = launch_append_rope<256>(a, interleaved, s); break;
    default: return PA_ERR_UNSUPPORTED;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
