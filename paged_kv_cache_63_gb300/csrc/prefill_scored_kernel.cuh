// prefill_scored_kernel.cuh -- multi-token attention under a score rule (pa_prefill_scored) for
// head_dim 256: one query tile per work item, CTAs that stay resident and take over work items
// of CTAs that have not started, as in prefill_kernel.cuh (work items, K/V stages, score
// buffers).
//
// What differs, beside the keys that an item sees: Q and the weights are tensor-memory operands
// of the products, which read shared memory for K and V alone. The weights lie over the first 32
// columns of their scores, so none are written to shared memory and no buffer is waited for (two
// 4096-token prompts of 24 / 4 heads with a prefix and a cap: 472 -> 418 us). The softmax warps
// copy Q there at the start of an item (the same prompts: 373 -> 361 us, without the cap 359 ->
// 326, with slopes 368 -> 340). The softmax bounds a capped call, one warp a scheduler; a second
// group of softmax warps taking every other tile gained nothing while Q was in shared memory.
//   TMEM (512 columns): S buffers at 0 and 64, the weights of a tile over the first 32 columns of
//   its scores; Q at 128 (row = lane, two fp16 a column); O at 256.
#pragma once

#include "early_launch.cuh"
#include "scored_softmax.cuh"

namespace pa {

// Barrier slots behind those of the plain kernel.
enum : int {
  kS1QReady = kNumBars,  // the item's Q is in tensor memory, its shared copy free (4 arrivals)
  kNumBarsS1 = kNumBars + 1
};

// Warps: 0 loads K, 2 Q and V; 1 owns TMEM and issues the MMAs; 3 schedules; 4..7 softmax.
constexpr int kScoredThreads = 256;
constexpr int kScoredVWarp = 2;
constexpr int kScoredSchedWarp = 3;
constexpr uint32_t kQCol = 128;  // Q's first tensor-memory column

// An item's keys go from kv_lo, the first token that some row sees, to kv_len, and its key tiles
// are taken last to first (as in prefill2_scored_kernel.cuh): tile j is the one j before last_tile.
// Warp-collective.
struct ScoredItem1 : Item1 {
  int kv_lo, prefix, last_tile;
  int rows, holes;  // as in the two-tile kernel
};

template <int TN, int kParts>
__device__ __forceinline__ ScoredItem1 scored_item1_of(const PrefillScoredArgs &a, int kv, int b,
                                                       int qtile) {
  ScoredItem1 it;
  it.kv = kv;
  it.b = b;
  it.live = it.rows = 0;
  it.stop = 0;
  it.ntiles = 0;
  const int q0 = __ldg(a.qs + b), q1 = __ldg(a.qs + b + 1), ctx = __ldg(a.ctx + b);
  const int n = q1 - q0;
  it.q0 = q0;
  it.n = n;
  unsigned bad = 0;
  if (ctx < 0 || static_cast<long long>(ctx) > static_cast<long long>(a.maxp) << a.ps_shift)
    bad = PA_DEVERR_CONTEXT;
  else if (q0 < 0 || n < 0 || static_cast<long long>(q1) > a.total || n > ctx)
    bad = PA_DEVERR_QUERY_START;
  if (bad) {
    if ((threadIdx.x & 31) == 0) atomicOr(a.err, bad);
    return it;
  }
  it.tok0 = qtile * a.qt;
  if (it.tok0 >= n) return it;
  it.base_pos = ctx - n + it.tok0;
  it.rows = 1;
  it.prefix = prefix_of(a.s, b, ctx);
  bool holes = false;
  seen_range<kParts>(a.s, q0, ctx - n, it.tok0, min(it.tok0 + a.qt, n), it.prefix, it.kv_lo,
                     it.max_pos, holes);
  it.holes = holes;
  if (it.max_pos < 0) return it;
  it.kv_len = it.max_pos + 1;
  it.last_tile = it.max_pos / TN;
  it.ntiles = it.last_tile - it.kv_lo / TN + 1;
  it.live = 1;
  return it;
}

// A thread's row of a tile, for scored_weights: scores at TMEM address ts, accumulated output at
// to, stable once the barrier of the last P.V has completed.
template <int HD>
struct ScoredTile1 {
  uint32_t ts, to, pv_bar, pv_parity;
  volatile int *abort_flag;
  unsigned *err;
  static constexpr bool kCapWithWeights = false, kKeysCleared = false;
  __device__ __forceinline__ void load(float (&c)[64]) const { tmem_ld64(ts, c); }
  template <class F>
  __device__ __forceinline__ void rewrite(F f) const { rewrite_columns(ts, f); }
  __device__ __forceinline__ void emit(const float (&pk)[32]) const { tmem_st32(ts, pk); }
  __device__ __forceinline__ bool settle(ScoredRow &row, float top, bool later) const {
    return settle_row(row, top, later, [&](float f) {
      // O holds the tiles before: wait for the last P.V, then scale this row of O in TMEM
      if (!pipe_wait(pv_bar, pv_parity, abort_flag, err)) return false;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        float v[32];
        tmem_ld32(to + c * 32, v);
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] *= f;
        tmem_st32(to + c * 32, v);
      }
      return true;
    });
  }
};

template <int HD, int kParts>
__global__ void __launch_bounds__(kScoredThreads, 1)
    prefill_scored_kernel(const __grid_constant__ PrefillScoredArgs a,
                          const __grid_constant__ CUtensorMap tq,
                          const __grid_constant__ CUtensorMap tk,
                          const __grid_constant__ CUtensorMap tv) {
  using C = PrefillCfg<HD>;
  using Item = ScoredItem1;
  constexpr bool kFirst = (kParts & kRuleFirst) != 0;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kNumBarsS1];
  __shared__ __align__(16) uint4 clc_answer;
  __shared__ Item items[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int *abort_flag = &abort_word;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q_rows = a.qt * a.g;

  const uint32_t sbase = (smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t *sgen = smem_raw + (sbase - smem_addr(smem_raw));
  const uint32_t sq = sbase + C::kQOff;
  auto k_stage = [&](int s) { return sbase + C::kKOff + s * C::kKVBytes; };
  auto v_stage = [&](int s) { return sbase + C::kVOff + s * C::kKVBytes; };
  auto bar = [&](int i) { return smem_addr(&bars[i]); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBarsS1; ++i) {
      uint32_t count = 1;
      if (i == kBarPFull || i == kBarPFull + 1) count = 128;
      if (i == kBarItemEmpty || i == kBarItemEmpty + 1) count = kItemReaders1;
      if (i == kS1QReady) count = 4;
      mbar_init(bar(i), count);
    }
    abort_word = 0;
    fence_barrier_init();
  }
  // Rows of Q past q_rows are never loaded: zero them once so their (discarded) results stay
  // finite.
  if (q_rows < C::kRows) {
    const int per_block = (C::kRows - q_rows) * 8;  // 16-byte chunks
    for (int i = threadIdx.x; i < C::KB * per_block; i += kScoredThreads) {
      const int kb = i / per_block, c = i % per_block;
      *reinterpret_cast<uint4 *>(sgen + C::kQOff + kb * (C::kRows * 128) + q_rows * 128 + c * 16) =
          make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  wait_for_stream();

  // first token of tile j of an item
  auto tile_token = [](const Item &it, int j) { return (it.last_tile - j) * C::TN; };

  // Reader side of the item ring: item k sits in entry k & 1. Returns false on abort.
  auto take_item = [&](int k, Item &it) {
    if (!pipe_wait(bar(kBarItemFull + (k & 1)), (k >> 1) & 1, abort_flag, a.err)) return false;
    it = items[k & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarItemEmpty + (k & 1)));
    return true;
  };

  // K/V tiles, S and P buffers and their barrier phases are numbered across the work items
  // a CTA runs: tile t (global) uses stage / buffer t & 1 and phase (t >> 1) & 1.
  if (warp == kScoredSchedWarp) {
    // ================= scheduler: one request per item (as in prefill2_kernel) =================
    int kv = blockIdx.x, b = blockIdx.y, z = blockIdx.z;
    bool stop = false;
    const uint32_t answer = smem_addr(&clc_answer);
    for (int k = 0;; ++k) {
      if (k >= 2 && !pipe_wait(bar(kBarItemEmpty + (k & 1)), ((k >> 1) - 1) & 1, abort_flag, a.err))
        break;
      Item it;
      it.stop = 1;
      it.live = it.rows = 0;
      if (!stop)  // longest rows first
        it = scored_item1_of<C::TN, kParts>(a, kv, b, a.n_qtiles - 1 - z);
      if (lane == 0) {
        items[k & 1] = it;
        mbar_arrive(bar(kBarItemFull + (k & 1)));
      }
      __syncwarp();
      if (stop) break;
      if (!pipe_wait(bar(kBarProdStart), k & 1, abort_flag, a.err)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(kBarClc), 16);
        clc_try_cancel(answer, bar(kBarClc));
      }
      __syncwarp();
      if (!pipe_wait(bar(kBarClc), k & 1, abort_flag, a.err)) {
        if (lane == 0) drain_wait(bar(kBarClc), k & 1, a.err);  // the answer's write lands first
        __syncwarp();
        break;
      }
      int x, y, zz;
      // after a failed request (every CTA has started) no other may be made
      stop = !clc_query(answer, x, y, zz) || x >= static_cast<int>(gridDim.x) ||
             y >= static_cast<int>(gridDim.y) || zz >= static_cast<int>(gridDim.z);
      kv = x;
      b = y;
      z = zz;
    }
  } else if (warp == 0 || warp == kScoredVWarp) {
    // ============ producers: warp 0 the K tiles, warp 2 Q and the V tiles ============
    const bool is_v = warp == kScoredVWarp;
    if (lane == 0) {
      prefetch_tensormap(is_v ? &tv : &tk);
      if (is_v) prefetch_tensormap(&tq);
    }
    const CUtensorMap *map = is_v ? &tv : &tk;
    // every query tile of the (sequence, K/V head) reads these K/V tiles: keep them in L2
    const uint64_t pol = l2_evict_last_policy();
    const int full = is_v ? kBarVFull : kBarKFull;
    const int empty = is_v ? kBarVEmpty : kBarKEmpty;
    const uint32_t stage0 = is_v ? v_stage(0) : k_stage(0);
    const int rows_per_box = min(a.ps, C::TN);
    const int boxes = C::TN / rows_per_box;
    const uint32_t box_bytes = rows_per_box * 128;
    int g = 0;  // global index of the next tile
    int q_loads = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      Item it;
      ok = take_item(k, it);
      if (!ok || it.stop) break;
      if (!is_v && lane == 0) mbar_arrive(bar(kBarProdStart));
      if (!it.live) continue;
      if (is_v) {
        // Q of this item, once the previous item's has been copied out
        if (q_loads > 0) ok = pipe_wait(bar(kS1QReady), (q_loads - 1) & 1, abort_flag, a.err);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(kBarQ), C::KB * q_rows * 128);
#pragma unroll
          for (int kb = 0; kb < C::KB; ++kb)
            tma_load_3d(sq + kb * (C::kRows * 128), &tq, bar(kBarQ), kb * 64, it.kv * a.g,
                        it.q0 + it.tok0, l2_evict_first_policy());  // read once
        }
        ++q_loads;
      }
      const int32_t *bt_row = a.bt + static_cast<size_t>(it.b) * a.maxp;
      // whether tile j's box of this lane holds a token between kv_lo and kv_len
      auto needed = [&](int j) {
        const int tok = tile_token(it, j) + lane * rows_per_box;
        return j < it.ntiles && lane < boxes && tok < it.kv_len && tok + rows_per_box > it.kv_lo;
      };
      auto page_of = [&](int j) {
        const int tok = tile_token(it, j) + lane * rows_per_box;
        return needed(j) ? __ldg(bt_row + (tok >> a.ps_shift)) : -1;
      };
      // the block-table read for tile j + 1 is issued before the waits of tile j
      int page_next = page_of(0);
      for (int j = 0; j < it.ntiles && ok; ++j, ++g) {
        const int st = g & 1;
        const int tok = tile_token(it, j) + lane * rows_per_box;
        bool need = needed(j);
        int page = page_next;
        page_next = page_of(j + 1);
        if (kFirst && it.holes) {  // no row may see the box
          const unsigned seen = seen_word<C::TN>(a.s, it.q0, it.base_pos - it.tok0, it.tok0,
                                                 min(it.tok0 + a.qt, it.n), it.prefix,
                                                 tile_token(it, j));
          const bool any = any_seen(seen, lane * rows_per_box, rows_per_box);
          need = need && any;
          if (!need) page = -1;
        }
        if (need && (page < 0 || page >= a.num_pages)) {
          if (!is_v) atomicOr(a.err, PA_DEVERR_PAGE_ID);
          page = -1;
        }
        const uint32_t issue = __ballot_sync(0xffffffffu, page >= 0);
        const int slot = tok & (a.ps - 1);
        int y, z;
        if (a.layout == PA_LAYOUT_HEAD_MAJOR) {
          y = slot;
          z = page * a.kvh + it.kv;
        } else {
          y = it.kv;
          z = (page << a.ps_shift) + slot;
        }
        if (g >= 2) ok = pipe_wait(bar(empty + st), ((g >> 1) - 1) & 1, abort_flag, a.err);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(bar(full + st), __popc(issue) * box_bytes * C::KB);
        __syncwarp();
        if (page >= 0) {
#pragma unroll
          for (int kb = 0; kb < C::KB; ++kb)
            tma_load_3d(stage0 + st * C::kKVBytes + kb * (C::TN * 128) + lane * box_bytes, map,
                        bar(full + st), kb * 64, y, z, pol);
        }
      }
    }
    // drain: the last load issued into each stage, and the last Q, have landed before the CTA
    // exits (older loads of a stage were consumed before it was refilled)
    if (lane == 0) {
      if (is_v && q_loads > 0) drain_wait(bar(kBarQ), (q_loads - 1) & 1, a.err);
      for (int t = max(0, g - 2); t < g; ++t) drain_wait(bar(full + (t & 1)), (t >> 1) & 1, a.err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================= MMA issuer =================
    bool ok = true;
    // PA_TEST_EXPIRE_WAITS: the first wait is on kBarDone, which no one completes before the end
    if (a.expire) ok = pipe_wait(bar(kBarDone), 0, abort_flag, a.err);
    int g = 0, q_waits = 0;
    for (int k = 0; ok; ++k) {
      Item it;
      ok = take_item(k, it);
      if (!ok || it.stop) break;
      if (!it.live) continue;
      ok = pipe_wait(bar(kS1QReady), q_waits & 1, abort_flag, a.err);
      ++q_waits;
      if (!ok) break;
      tc_fence_after();
      for (int j = 0; j <= it.ntiles && ok; ++j) {
        if (j < it.ntiles) {
          const int t = g + j, st = t & 1;
          ok = pipe_wait(bar(kBarKFull + st), (t >> 1) & 1, abort_flag, a.err);
          if (!ok) break;
          tc_fence_after();
          {
            // issued warp-collectively by one elected lane of the converged warp, with
            // descriptors = base descriptor + step offset / 16 (the empty asm keeps the
            // compiler from hoisting every step's descriptor into registers)
            const uint32_t d = tmem + st * C::TN;
            uint64_t kd = smem_desc_sw128(k_stage(st), 16, 1024);
            asm volatile("" : "+l"(kd));
#pragma unroll
            for (int ks = 0; ks < HD / 16; ++ks) {
              const uint64_t bd = kd + (((ks >> 2) * (C::TN * 128) + (ks & 3) * 32) >> 4);
              mma_f16_ts_warp(d, tmem + kQCol + ks * 8, bd, C::kIdescS, ks > 0);
            }
            mma_commit_warp(bar(kBarSFull + st));
            mma_commit_warp(bar(kBarKEmpty + st));
            if (j == it.ntiles - 1) mma_commit_warp(bar(kBarQEmpty));
          }
        }
        if (j >= 1) {
          const int i = j - 1, t = g + i, st = t & 1;
          ok = pipe_wait(bar(kBarPFull + st), (t >> 1) & 1, abort_flag, a.err);
          if (ok) ok = pipe_wait(bar(kBarVFull + st), (t >> 1) & 1, abort_flag, a.err);
          if (!ok) break;
          tc_fence_after();
          // V rows of tokens that no row sees (outside [kv_lo, kv_len), or in holes) may hold
          // anything; P is zero there, but 0 * NaN is not, so clear them
          const int first = i == it.ntiles - 1 ? max(it.kv_lo - tile_token(it, i), 0) : 0;
          const int end = i == 0 ? min(it.kv_len - tile_token(it, i), C::TN) : C::TN;
          if (first > 0 || end < C::TN || (kFirst && it.holes)) {
            unsigned seen = bits_between(first - 32 * lane, end - 1 - 32 * lane);
            if (kFirst && it.holes)
              seen = seen_word<C::TN>(a.s, it.q0, it.base_pos - it.tok0, it.tok0,
                                      min(it.tok0 + a.qt, it.n), it.prefix, tile_token(it, i));
            uint8_t *vg = sgen + C::kVOff + st * C::kKVBytes;
#pragma unroll 1
            for (int c = lane; c < C::TN * 8; c += 32) {  // 16-byte chunks of a column block
              const int r = c >> 3;
              if (kFirst ? any_seen(seen, r, 1) : r >= first && r < end) continue;
#pragma unroll
              for (int kb = 0; kb < C::KB; ++kb)
                *reinterpret_cast<uint4 *>(vg + kb * (C::TN * 128) + c * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async();
            __syncwarp();
          }
          {
            // the item's first P.V overwrites O: the softmax released this P only after it
            // had read the previous item's O
            uint64_t vd = smem_desc_sw128(v_stage(st), C::TN * 128, 1024);
            asm volatile("" : "+l"(vd));
#pragma unroll
            for (int ks = 0; ks < C::TN / 16; ++ks) {
              const uint64_t bd = vd + ((ks * 2048) >> 4);
              mma_f16_ts_warp(tmem + C::kOCol, tmem + st * C::TN + ks * 8, bd, C::kIdescPV,
                              (i > 0 || ks > 0) ? 1u : 0u);
            }
            mma_commit_warp(bar(kBarPV + st));
            mma_commit_warp(bar(kBarVEmpty + st));
          }
        }
      }
      g += it.ntiles;
    }
    // every MMA this warp issued has completed before TMEM is released
    mma_commit_warp(bar(kBarDone));
    if (lane == 0) drain_wait(bar(kBarDone), 0, a.err);
    __syncwarp();
  } else {
    // ================= softmax: one query row per thread =================
    const int rg = warp & 3;
    const int row = rg * 32 + lane;
    const int t = row / a.g, h = row - t * a.g;
    const uint32_t trow = tmem + (static_cast<uint32_t>(rg * 32) << 16);
    int g = 0, live = 0;  // tiles and live items so far
    bool ok = true;
    for (int k = 0; ok; ++k) {
      Item it;
      ok = take_item(k, it);
      if (!ok || it.stop) break;
      if (!it.rows) continue;
      const bool valid = row < q_rows && it.tok0 + t < it.n;
      const size_t out_row =
          (static_cast<size_t>(it.q0 + it.tok0 + t) * a.qh + it.kv * a.g + h) * HD;
      if (kFirst && !it.live) {  // no row sees anything
        if (valid) store_zero_row(a.out16 + out_row, HD);
        continue;
      }
      // Q moves to tensor memory, once the last score MMA of the item before has read the Q there
      ok = pipe_wait(bar(kBarQ), live & 1, abort_flag, a.err);
      if (ok && live > 0) ok = pipe_wait(bar(kBarQEmpty), (live - 1) & 1, abort_flag, a.err);
      if (!ok) break;
      ++live;
      tc_fence_after();
#pragma unroll
      for (int kb = 0; kb < C::KB; ++kb) {
        float q[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 w = lds128(sq + kb * (C::kRows * 128) + row * 128 + ((c ^ (row & 7)) << 4));
          q[4 * c] = __uint_as_float(w.x);
          q[4 * c + 1] = __uint_as_float(w.y);
          q[4 * c + 2] = __uint_as_float(w.z);
          q[4 * c + 3] = __uint_as_float(w.w);
        }
        tmem_st32(trow + kQCol + kb * 32, q);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kS1QReady));
      // rows past the tile's last token repeat it (and are not stored)
      ScoredRow sr = scored_row(a.s, it.q0, it.base_pos - it.tok0,
                                min(it.tok0 + min(t, a.qt - 1), it.n - 1), it.kv * a.g + h,
                                it.prefix, valid);
      for (int j = 0; j < it.ntiles; ++j, ++g) {
        const int st = g & 1;
        ok = pipe_wait(bar(kBarSFull + st), (g >> 1) & 1, abort_flag, a.err);
        if (!ok) break;
        tc_fence_after();
        const ScoredTile1<HD> io = {trow + st * C::TN, trow + C::kOCol, bar(kBarPV + (st ^ 1)),
                                    static_cast<uint32_t>(((g - 1) >> 1) & 1), abort_flag, a.err};
        ok = scored_weights<kParts>(a.s, a.scale_log2, sr, tile_token(it, j), j > 0, io);
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kBarPFull + st));
      }
      if (ok) ok = pipe_wait(bar(kBarPV + ((g - 1) & 1)), ((g - 1) >> 1) & 1, abort_flag, a.err);
      if (!ok) break;
      tc_fence_after();
      // Once these loads have returned, O may be overwritten by the next item's first P.V, which
      // waits for this warp's next P.
      const float inv = sr.l > 0.f ? 1.f / sr.l : 0.f;
      const uint64_t pol = l2_evict_first_policy();
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        float v[32];
        tmem_ld32(trow + C::kOCol + c * 32, v);
        if (valid) store_half32(a.out16 + out_row + c * 32, v, inv, a.out_v8, pol);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

}  // namespace pa
