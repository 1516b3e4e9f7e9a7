// span_split.cuh -- how the decode kernels under a score rule lay out their work: the span of tokens
// that a sequence's query sees, the split of all units' tiles into one range per worker, TMA loads
// issued by the converged warp, and the launch of the kernel that joins shared units.
#pragma once

#include "decode_kernel.cuh"
#include "early_launch.cuh"
#include "score_rule.cuh"

namespace pa {

struct ScoredArgs {
  KernelArgs k;  // out, flags, epoch and the fixed-split arrays are unused
  ScoreArgs s;
  void *out;  // [batch][query_heads][head_dim], fp32 or fp16
};

// The tokens [lo, end) that sequence b's query sees.
struct Span {
  int lo, end;
};

__device__ __forceinline__ Span load_span(const ScoredArgs &a, int b) {
  Span sp;
  sp.end = load_ctx(a.k, b);
  sp.lo = sp.end > 0 ? min(first_seen(a.s, b, sp.end - 1), sp.end) : 0;
  return sp;
}

// Tiles start at multiples of T, so that a tile's pieces never cross a page.
__device__ __forceinline__ int span_start(const Span &sp, int T) { return sp.lo & ~(T - 1); }

__device__ __forceinline__ int span_tiles(const Span &sp, int T) {
  return sp.end > sp.lo ? (sp.end - span_start(sp, T) + T - 1) / T : 0;
}

// Position of a worker in its token stream.
struct SpanCursor {
  int b, us;  // sequence, group unit
  int tok;    // first token of the current tile
  Span sp;
  int left;       // tiles still to visit
  long long ug0;  // global index of the unit's first tile
};

__device__ __forceinline__ void advance(const ScoredArgs &a, SpanCursor &c, int T) {
  c.tok += T;
  --c.left;
  if (c.left > 0 && c.tok >= c.sp.end) {
    c.ug0 += span_tiles(c.sp, T);
    if (++c.us == a.k.upg) {
      c.us = 0;
      do {
        ++c.b;
        if (c.b < a.k.batch) c.sp = load_span(a, c.b);
      } while (c.b < a.k.batch && c.sp.end <= c.sp.lo);
    }
    c.tok = span_start(c.sp, T);
  }
}

// Total tiles, the workers that get tiles, and the cursor at this worker's first tile; false
// when it gets none (the split of balanced_start over the spans' tiles).
__device__ inline bool span_balanced_start(const ScoredArgs &a, int worker, int T, SpanCursor &c,
                                           long long &total, long long &nworkers) {
  const int lane = threadIdx.x & 31;
  const int batch = a.k.batch, upg = a.k.upg;
  const int blk = (batch + 31) >> 5;
  const int b0 = min(lane * blk, batch);
  const int b1 = min(b0 + blk, batch);
  long long mine = 0;
#pragma unroll 8
  for (int b = b0; b < b1; ++b) mine += span_tiles(load_span(a, b), T);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  total = __shfl_sync(0xffffffffu, incl, 31) * upg;
  nworkers = total < a.k.workers ? total : a.k.workers;
  if (worker >= nworkers) return false;
  const long long s = worker_start(worker, total, nworkers);
  const long long e = worker_start(worker + 1, total, nworkers);
  const int L = __ffs(__ballot_sync(0xffffffffu, incl * upg > s)) - 1;
  long long run = __shfl_sync(0xffffffffu, incl - mine, L) * upg;
  const int lb0 = min(L * blk, batch);
  const int lb1 = min(lb0 + blk, batch);
  for (int base = lb0; base < lb1; base += 32) {
    const int b = base + lane;
    const long long t =
        b < lb1 ? static_cast<long long>(span_tiles(load_span(a, b), T)) * upg : 0;
    long long in2 = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, in2, o);
      if (lane >= o) in2 += y;
    }
    const long long chunk = __shfl_sync(0xffffffffu, in2, 31);
    if (s < run + chunk) {
      const int M = __ffs(__ballot_sync(0xffffffffu, run + in2 > s)) - 1;
      const long long excl = run + __shfl_sync(0xffffffffu, in2 - t, M);
      c.b = base + M;
      c.sp = load_span(a, c.b);
      const int tb = span_tiles(c.sp, T);
      const long long inner = s - excl;
      c.us = static_cast<int>(inner / tb);
      c.tok = span_start(c.sp, T) + static_cast<int>(inner % tb) * T;
      c.ug0 = excl + static_cast<long long>(c.us) * tb;
      c.left = static_cast<int>(e - s);
      return true;
    }
    run += chunk;
  }
  return false;
}

// One elected lane of the converged warp announces the bytes a barrier waits for, or issues a
// TMA load; the operands are the same in every lane. (In a branch of lane 0 alone the issue of a
// 16-token tile of head_dim 128 took 1030 of the 2970 cycles that a worker spends on the tile.)
__device__ __forceinline__ void expect_bytes_warp(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}

__device__ __forceinline__ void tma_rows_warp(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                              int row, int head, int block, uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(row), "r"(head), "r"(block),
      "l"(policy)
      : "memory");
}

// D(16x8, fp32) = A(16x16, fp16) B(16x8, fp16) + D.
__device__ __forceinline__ void mma_rows16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Probabilities are 2^(x - m): the reference m follows the row's maximum so that it lies kLift below
// it when set, and moves only when a score passes m + kLift + kRescaleSlack. They stay within 2^15
// (fp16 holds them), and a probability 2^-31 of the largest still has a nonzero fp16 value.
constexpr float kLift = 7.f;

// Zero the output rows of a unit that sees nothing.
template <int HD>
__device__ __forceinline__ void zero_rows_out(const ScoredArgs &a, const UnitInfo &u) {
  const int lane = threadIdx.x & 31;
  const long long base = (static_cast<long long>(u.b) * a.k.qh + u.h0) * HD;
  for (int i = lane * 2; i < u.nh * HD; i += 64) store_out2(a.s, a.out, base + i, 0.f, 0.f);
}

// Host: the arguments of a decode call under a plan, but the rule, the rings' size and the test hook
// (decode_scored.cu). `a` comes in zeroed but for its rule.
pa_status_t fill_scored_args(const pa_problem_t *problem, const pa_plan_t &pl, const void *query,
                             const int32_t *block_tables, const int32_t *context_lengths,
                             float scale, void *out, void *workspace, ScoredArgs *a);

// Host: launches the kernel that joins the states of units which several workers share
// (decode_scored.cu); `warps` of combine_warps_per_pair, `tile` the decode launch's tokens per tile.
cudaError_t launch_join_states(const ScoredArgs &a, int units, int heads, int warps, int tile,
                               cudaStream_t stream);

}  // namespace pa
