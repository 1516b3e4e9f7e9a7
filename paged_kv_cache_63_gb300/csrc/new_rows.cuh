// new_rows.cuh -- the new tokens of a batch as packed rows: which sequence a row belongs to, and the
// checks of offsets and lengths that come with it.
#pragma once

#include "device_common.cuh"
#include "internal.h"

namespace pa {

// Sequence b's rows are query_start[b] .. query_start[b + 1] - 1, its last tokens.
struct NewRowsArgs {
  const int32_t *qs, *bt, *ctx;
  unsigned *err;
  long long total;
  int batch, kvh, ps, ps_shift, maxp, num_pages, layout;
};

// Rows of queries, keys and values with their position rotation.
struct RopeArgs : NewRowsArgs {
  const uint16_t *q, *k, *v;  // fp16 bits; q may be null
  uint16_t *q_out;
  void *k_cache, *v_cache;
  const float *table;
  const int32_t *positions;  // may be null
  long long q_stride, k_stride, v_stride;  // elements
  int qh;
  int rotary, table_rows, interleaved;
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
__device__ __forceinline__ bool holds(const NewRowsArgs &a, int b, int row) {
  const int q0 = __ldg(a.qs + b), q1 = __ldg(a.qs + b + 1), c = __ldg(a.ctx + b);
  return q0 >= 0 && q0 <= row && row < q1 && q1 <= a.total && c <= (a.maxp << a.ps_shift) &&
         q1 - q0 <= c;
}

// The sequence that holds row `row`, or -1, by a look at every one: one wrong offset sends the
// search by halves astray for rows of other sequences. Warp-collective.
__device__ __forceinline__ int look_for_sequence(const NewRowsArgs &a, int row) {
#pragma unroll 1
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int b = b0 + (threadIdx.x & 31);
    const unsigned found = __ballot_sync(0xffffffffu, b < a.batch && holds(a, b, row));
    if (found) return b0 + __ffs(found) - 1;
  }
  return -1;
}

// Every sequence is checked once, whichever rows it holds: the threads of the grid share them.
__device__ __forceinline__ void check_sequences(const NewRowsArgs &a) {
  for (long long b = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; b < a.batch;
       b += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int q0 = __ldg(a.qs + b), q1 = __ldg(a.qs + b + 1), c = __ldg(a.ctx + b);
    if (c < 0 || c > (a.maxp << a.ps_shift))
      atomicOr(a.err, PA_DEVERR_CONTEXT);
    else if (q0 < 0 || q1 < q0 || q1 > a.total || q1 - q0 > c)
      atomicOr(a.err, PA_DEVERR_QUERY_START);
  }
}

// The sequence that row `row` is of; -1 for rows behind the last sequence, and for rows of a sequence
// that check_sequences flags. Warp-collective.
__device__ __forceinline__ int sequence_of_row(const NewRowsArgs &a, int row) {
  const int b = find_sequence(a.qs, a.batch, row);
  if (b >= 0 && holds(a, b, row)) return b;
  if (row >= __ldg(a.qs + a.batch)) return -1;
  return look_for_sequence(a, row);
}

// Token index, page and rotation position of row `row` of sequence b; false (flagged by the threads
// that `tells`): nothing of it is to be written.
__device__ __forceinline__ bool place_of_row(const RopeArgs &a, int b, int row, int &t, int &page,
                                             int &pos, bool tells) {
  const int q1 = __ldg(a.qs + b + 1), c = __ldg(a.ctx + b);
  t = c - q1 + row;
  page = __ldg(a.bt + static_cast<long long>(b) * a.maxp + (t >> a.ps_shift));
  pos = a.rotary == 0 ? 0 : a.positions ? __ldg(a.positions + row) : t;
  const bool bad_page = page < 0 || page >= a.num_pages;
  const bool bad_pos = a.rotary > 0 && (pos < 0 || pos >= a.table_rows);
  if (!bad_page && !bad_pos) return true;
  if (tells)
    atomicOr(a.err, (bad_page ? PA_DEVERR_PAGE_ID : 0u) | (bad_pos ? PA_DEVERR_POSITION : 0u));
  return false;
}

// Cosines and sines of pairs 8 i .. 8 i + 7 at position pos.
__device__ __forceinline__ void load_angles(const RopeArgs &a, int pos, int i, float (&cs)[8],
                                            float (&sn)[8]) {
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

// Host: checks the arguments of a call that writes new rows and fills the kernel's; args->total 0:
// there is nothing to do (append_rope.cu). `args` comes in zeroed.
pa_status_t resolve_new_rows(const pa_problem_t *problem, const pa_rope_t *rope, const void *query,
                             int64_t query_stride, const void *new_key, int64_t key_stride,
                             const void *new_value, int64_t value_stride,
                             const int32_t *query_start, int64_t total_tokens,
                             const int32_t *block_tables, const int32_t *context_lengths,
                             void *query_out, void *key_cache, void *value_cache, RopeArgs *args);

}  // namespace pa
