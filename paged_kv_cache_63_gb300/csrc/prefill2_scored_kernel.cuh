// prefill2_scored_kernel.cuh -- multi-token attention under a score rule (pa_prefill_scored) for
// head_dim 64 and 128: two query tiles per work item that share every K/V tile, CTAs that stay
// resident and take over work items of CTAs that have not started, as in prefill2_kernel.cuh
// (work items, roles of the warps, K/V ring).
//
// What differs, because here the softmax bounds the kernel: the scores of a query tile are
// computed 64 keys at a time into two tensor-memory buffers, so that a tile's next scores are
// already there when its softmax has released its weights. (With one buffer of 128 keys, as in
// the plain kernel, a softmax warp waited 1900 of every 5900 cycles for the product that reads
// its weights and the scores after it.)
//   TMEM (512 columns): S_X buffers at 128 X and 128 X + 64, O_X at 256 + 128 X; the weights of
//   a unit of 64 keys overwrite the first 32 columns of its scores.
// Each query tile has an MMA warp of its own (one for both, taking turns, delayed a tile's next
// scores behind the other tile's weights: 1300 of 2500 cycles a unit). Its order is PV(n),
// S(n + 2): S(n + 2) goes into the buffer that PV(n) reads, so it follows it in issue order. A
// softmax that has to rescale O_X waits for the last PV_X.
// Warps: 0 loads K and V; 1 and 2 issue the MMAs of tile A and B (1 also owns the tensor
// memory); 3 schedules and loads Q; 4..7 are tile A's softmax, 8..11 tile B's.
#pragma once

#include "early_launch.cuh"
#include "prefill2_kernel.cuh"
#include "scored_softmax.cuh"

namespace pa {

// Barrier slots. Units of a query tile X are counted across items; unit n uses buffer n & 1 and
// phase n >> 1 of the barriers of that buffer.
enum : int {
  kS2QFull = 0,       // Q of an item landed
  kS2QEmpty = 1,      // both tiles' last score MMAs of the item completed (2 arrivals)
  kS2SFull = 2,       // + 2 X + buffer
  kS2PFull = 6,       // + 2 X + buffer (128 arrivals)
  kS2PV = 10,         // + 2 X + buffer: the P.V of the unit completed
  kS2Done = 14,       // + X: every MMA of the tile's warp completed
  kS2ItemFull = 16,   // +entry
  kS2ItemEmpty = 18,  // +entry (kItemReaders arrivals)
  kS2ProdStart = 20,  // the producer started an item
  kS2Clc = 21,        // the answer to a cancellation request landed
  kS2Full = 22,       // +slot
  kS2Empty = 30,      // +slot (2 arrivals: both MMA warps are done with it)
  kNumBarsS2 = 38
};

constexpr int kUnit = 64;  // keys of a unit

// Geometry of a work item. Its keys go from kv_lo, the first token that some row of the pair
// sees, to kv_len. Its key tiles are taken last to first, tile j (0 .. nt_max - 1) being the one j
// before the last: a bias by distance and most attention favour near keys, so a row meets its
// largest scores first and rarely moves its reference again (first to last, a steep bias moved
// it, and rescaled O, on every tile: 7250 cycles a tile against 3600). A tile is two units of 64
// keys, taken last to first too, and query tile X takes part in units [from_X, to_X), none if it
// has no rows or they see nothing. `rows` tells that the pair has
// rows, `live` that some of them sees something; `holes` that tokens between kv_lo and kv_len may
// be seen by nobody. Warp-collective.
struct ScoredItem2 : Item2 {
  int kv_lo, prefix, last_tile;  // last_tile: index of the key tile taken first
  int from_a, to_a, from_b, to_b;
  int rows, holes;
};

template <int TN, int kParts>
__device__ __forceinline__ ScoredItem2 scored_item2_of(const PrefillScoredArgs &a, int kv, int b,
                                                       int pair) {
  ScoredItem2 it;
  it.kv = kv;
  it.b = b;
  it.live = it.rows = 0;
  it.stop = 0;
  it.from_a = it.to_a = it.from_b = it.to_b = it.nt_max = 0;
  const int q0 = __ldg(a.qs + b), q1 = __ldg(a.qs + b + 1), ctx = __ldg(a.ctx + b);
  const int n = q1 - q0;
  it.q0 = q0;
  it.n = n;
  it.ctx = ctx;
  unsigned bad = 0;
  if (ctx < 0 || static_cast<long long>(ctx) > static_cast<long long>(a.maxp) << a.ps_shift)
    bad = PA_DEVERR_CONTEXT;
  else if (q0 < 0 || n < 0 || static_cast<long long>(q1) > a.total || n > ctx)
    bad = PA_DEVERR_QUERY_START;
  if (bad) {
    if ((threadIdx.x & 31) == 0) atomicOr(a.err, bad);
    return it;
  }
  it.tok0_a = 2 * pair * a.qt;
  it.tok0_b = it.tok0_a + a.qt;
  if (it.tok0_a >= n) return it;
  it.rows = 1;
  it.prefix = prefix_of(a.s, b, ctx);
  int lo_a, lo_b = 0, last_a, last_b = -1;
  bool holes = false;
  seen_range<kParts>(a.s, q0, ctx - n, it.tok0_a, min(it.tok0_b, n), it.prefix, lo_a, last_a,
                     holes);
  if (it.tok0_b < n)
    seen_range<kParts>(a.s, q0, ctx - n, it.tok0_b, min(it.tok0_b + a.qt, n), it.prefix, lo_b,
                       last_b, holes);
  it.holes = holes;
  const int last = max(last_a, last_b);
  if (last < 0) return it;
  it.kv_lo = last_a < 0 ? lo_b : last_b < 0 ? lo_a : min(lo_a, lo_b);
  it.kv_len = last + 1;
  it.last_tile = last / TN;
  if (last_a >= 0) {
    it.from_a = 2 * it.last_tile + 1 - last_a / kUnit;
    it.to_a = 2 * it.last_tile + 2 - lo_a / kUnit;
  }
  if (last_b >= 0) {
    it.from_b = 2 * it.last_tile + 1 - last_b / kUnit;
    it.to_b = 2 * it.last_tile + 2 - lo_b / kUnit;
  }
  it.nt_max = (max(it.to_a, it.to_b) + 1) / 2;
  it.live = 1;
  return it;
}

// A thread's row of a unit, for scored_weights: scores at TMEM address ts, accumulated output at
// to, stable once the barrier of the last P.V has completed.
template <int HD>
struct ScoredTile2 {
  uint32_t ts, to, pv_bar, pv_parity;
  volatile int *abort_flag;
  unsigned *err;
  static constexpr bool kCapWithWeights = true, kKeysCleared = true;
  __device__ __forceinline__ void load(float (&c)[64]) const { tmem_ld64(ts, c); }
  template <class F>
  __device__ __forceinline__ void rewrite(F f) const { rewrite_columns(ts, f); }
  __device__ __forceinline__ void emit(const float (&pk)[32]) const { tmem_st32(ts, pk); }
  __device__ __forceinline__ bool settle(ScoredRow &row, float top, bool later) const {
    return settle_row(row, top, later, [&](float f) {
      if (!pipe_wait(pv_bar, pv_parity, abort_flag, err)) return false;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        float o[32];
        tmem_ld32(to + c * 32, o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= f;
        tmem_st32(to + c * 32, o);
      }
      return true;
    });
  }
};

template <int HD, int kParts>
__global__ void __launch_bounds__(kPrefill2Threads, 1)
    prefill2_scored_kernel(const __grid_constant__ PrefillScoredArgs a,
                           const __grid_constant__ CUtensorMap tq,
                           const __grid_constant__ CUtensorMap tk,
                           const __grid_constant__ CUtensorMap tv) {
  using C = Prefill2Cfg<HD>;
  using Item = ScoredItem2;
  constexpr bool kFirst = (kParts & kRuleFirst) != 0;
  constexpr uint32_t kIdescS = idesc_f16(C::kRows, 64, 0, 0);
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kNumBarsS2];
  __shared__ __align__(16) uint4 clc_answer;
  __shared__ Item items[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int *abort_flag = &abort_word;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q_rows = a.qt * a.g;

  const uint32_t sbase = (smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t *sgen = smem_raw + (sbase - smem_addr(smem_raw));
  auto q_tile = [&](int x) { return sbase + C::kQOff + x * C::kQBytes; };
  auto slot_addr = [&](int s) { return sbase + C::kRingOff + s * C::kSlotBytes; };
  auto bar = [&](int i) { return smem_addr(&bars[i]); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBarsS2; ++i) {
      uint32_t count = 1;
      if (i >= kS2PFull && i < kS2PFull + 4) count = 128;
      if (i == kS2ItemEmpty || i == kS2ItemEmpty + 1) count = kItemReaders;
      if (i == kS2QEmpty || i >= kS2Empty) count = 2;
      mbar_init(bar(i), count);
    }
    abort_word = 0;
    fence_barrier_init();
  }
  // MMA rows past q_rows (g not dividing 128) are never written by the Q loads: zero once
  if (q_rows < C::kRows) {
    const int per_block = (C::kRows - q_rows) * 8;
    for (int i = threadIdx.x; i < 2 * C::KB * per_block; i += kPrefill2Threads) {
      const int x = i / (C::KB * per_block), r = i % (C::KB * per_block);
      const int kb = r / per_block, c = r % per_block;
      *reinterpret_cast<uint4 *>(sgen + C::kQOff + x * C::kQBytes + kb * (C::kRows * 128) +
                                 q_rows * 128 + c * 16) = make_uint4(0, 0, 0, 0);
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

  // first token of K/V tile j of an item
  auto tile_token = [](const Item &it, int j) { return (it.last_tile - j) * C::TN; };

  // Reader side of the item ring: item k sits in entry k & 1. Returns false on abort.
  auto take_item = [&](int k, Item &it) {
    if (!pipe_wait(bar(kS2ItemFull + (k & 1)), (k >> 1) & 1, abort_flag, a.err)) return false;
    it = items[k & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kS2ItemEmpty + (k & 1)));
    return true;
  };

  // registers: the softmax warpgroups hold a 128-column score row per thread; each role
  // changes its own allocation inside its branch so the compiler sees one limit per region
  if (warp < 4) regs_decrease<kPrefill2SmallRegs>();
  if (warp == 3) {
    // ================= scheduler =================
    int kv = blockIdx.x, b = blockIdx.y, z = blockIdx.z;
    bool stop = false;
    int q_loads = 0;
    const uint64_t pol_q = l2_evict_first_policy();  // each Q tile is read once
    const uint32_t answer = smem_addr(&clc_answer);
    if (lane == 0) prefetch_tensormap(&tq);
    for (int k = 0;; ++k) {
      // publish item k once every reader has taken item k - 2 from the same entry
      if (k >= 2 && !pipe_wait(bar(kS2ItemEmpty + (k & 1)), ((k >> 1) - 1) & 1, abort_flag, a.err))
        break;
      Item it;
      it.stop = 1;
      it.live = it.rows = 0;
      if (!stop)  // grid.z counts pairs
        it = scored_item2_of<C::TN, kParts>(a, kv, b, a.n_qtiles - 1 - z);
      if (lane == 0) {
        items[k & 1] = it;
        mbar_arrive(bar(kS2ItemFull + (k & 1)));
      }
      __syncwarp();
      if (it.live) {
        // both query tiles, once the previous item's last score MMAs have read Q; here rather
        // than by the producer, whose K and V tiles of the item must not wait for that
        if (q_loads > 0 && !pipe_wait(bar(kS2QEmpty), (q_loads - 1) & 1, abort_flag, a.err)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(kS2QFull), 2 * C::KB * q_rows * 128);
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb)
              tma_load_3d(q_tile(x) + kb * (C::kRows * 128), &tq, bar(kS2QFull), kb * 64,
                          it.kv * a.g, it.q0 + (x ? it.tok0_b : it.tok0_a), pol_q);
        }
        ++q_loads;
      }
      __syncwarp();
      if (stop) break;
      // ask for item k + 1 when the K producer starts item k
      if (!pipe_wait(bar(kS2ProdStart), k & 1, abort_flag, a.err)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(kS2Clc), 16);
        clc_try_cancel(answer, bar(kS2Clc));
      }
      __syncwarp();
      if (!pipe_wait(bar(kS2Clc), k & 1, abort_flag, a.err)) {
        if (lane == 0) drain_wait(bar(kS2Clc), k & 1, a.err);  // the answer's write lands first
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
    if (lane == 0 && q_loads > 0) drain_wait(bar(kS2QFull), (q_loads - 1) & 1, a.err);
    __syncwarp();
  } else if (warp == 0) {
    // ================= producer: ring item 2t is K of global tile t, 2t + 1 its V =================
    if (lane == 0) {
      prefetch_tensormap(&tk);
      prefetch_tensormap(&tv);
    }
    // every pair of query tiles of a (sequence, K/V head) reads its K/V tiles: they stay in L2
    const uint64_t pol = l2_evict_last_policy();
    const int rows_per_box = min(a.ps, C::TN);
    const int boxes = C::TN / rows_per_box;
    const uint32_t box_bytes = rows_per_box * 128;
    int next = 0;  // next ring item
    bool ok = true;
    for (int k = 0; ok; ++k) {
      Item it;
      ok = take_item(k, it);
      if (!ok || it.stop) break;
      if (lane == 0) mbar_arrive(bar(kS2ProdStart));
      if (!it.live) continue;
      const int32_t *bt_row = a.bt + static_cast<size_t>(it.b) * a.maxp;
      // whether tile j's box of this lane holds a token between kv_lo and kv_len
      auto needed = [&](int j) {
        const int tok = tile_token(it, j) + lane * rows_per_box;
        return j < it.nt_max && lane < boxes && tok < it.kv_len && tok + rows_per_box > it.kv_lo;
      };
      auto load_tile = [&](const CUtensorMap *map, int tok, int page) {
        const int s = next % C::kSlots;
        const uint32_t issue = __ballot_sync(0xffffffffu, page >= 0);
        const int slot_in_page = tok & (a.ps - 1);
        const bool hm = a.layout == PA_LAYOUT_HEAD_MAJOR;
        const int y = hm ? slot_in_page : it.kv;
        const int z = hm ? page * a.kvh + it.kv : (page << a.ps_shift) + slot_in_page;
        if (next >= C::kSlots)
          ok = pipe_wait(bar(kS2Empty + s), ((next / C::kSlots) - 1) & 1, abort_flag, a.err);
        if (!ok) return;
        if (lane == 0) mbar_arrive_expect_tx(bar(kS2Full + s), __popc(issue) * box_bytes * C::KB);
        __syncwarp();
        if (page >= 0) {
#pragma unroll
          for (int kb = 0; kb < C::KB; ++kb)
            tma_load_3d(slot_addr(s) + kb * (C::TN * 128) + lane * box_bytes, map,
                        bar(kS2Full + s), kb * 64, y, z, pol);
        }
        ++next;
      };
      auto page_of = [&](int j) {
        const int tok = tile_token(it, j) + lane * rows_per_box;
        return needed(j) ? __ldg(bt_row + (tok >> a.ps_shift)) : -1;
      };
      int page_next = page_of(0);
      for (int j = 0; j < it.nt_max && ok; ++j) {
        const int tok = tile_token(it, j) + lane * rows_per_box;
        bool need = needed(j);
        int page = page_next;
        page_next = page_of(j + 1);
        if (kFirst && it.holes) {  // no row may see the box
          const unsigned seen = seen_word<C::TN>(a.s, it.q0, it.ctx - it.n, it.tok0_a,
                                                 min(it.tok0_b + a.qt, it.n), it.prefix,
                                                 tile_token(it, j));
          const bool any = any_seen(seen, lane * rows_per_box, rows_per_box);
          need = need && any;
          if (!need) page = -1;
        }
        if (need && (page < 0 || page >= a.num_pages)) {
          atomicOr(a.err, PA_DEVERR_PAGE_ID);
          page = -1;
        }
        load_tile(&tk, tok, page);
        if (ok) load_tile(&tv, tok, page);
      }
    }
    // drain: the newest item of every slot has landed (older items of a slot were consumed
    // before it was refilled)
    if (lane == 0) {
      for (int r = max(0, next - C::kSlots); r < next; ++r)
        drain_wait(bar(kS2Full + r % C::kSlots), (r / C::kSlots) & 1, a.err);
    }
    __syncwarp();
  } else if (warp < 3) {
    // ================= MMA issuer of query tile x =================
    const int x = warp - 1;
    bool ok = true;
    // PA_TEST_EXPIRE_WAITS: the first wait is on the barrier that completes only at the end
    if (a.expire) ok = pipe_wait(bar(kS2Done + x), 0, abort_flag, a.err);
    const uint32_t sx = tmem + 128u * x, ox = tmem + 256u + 128u * x;
    auto wait_ring = [&](int item) {
      const bool r = pipe_wait(bar(kS2Full + item % C::kSlots), (item / C::kSlots) & 1, abort_flag,
                               a.err);
      tc_fence_after();
      return r;
    };
    auto release = [&](int item) { mma_commit_warp(bar(kS2Empty + item % C::kSlots)); };
    int gt = 0, q_waits = 0;
    int s_n = 0, p_n = 0;  // units whose S, P.V were issued
    for (int k = 0; ok; ++k) {
      Item it;
      ok = take_item(k, it);
      if (!ok || it.stop) break;
      if (!it.live) continue;
      const int from = x ? it.from_b : it.from_a, to = x ? it.to_b : it.to_a;
      // MMAs and commits are issued warp-collectively (one elected lane), with operands every
      // lane computes identically; descriptors of a K step are a base descriptor plus the step's
      // byte offset / 16 (the empty asm keeps all steps' descriptors out of registers).
      // Units of a K/V tile run from its later keys (hh 0: rows 64..127) to its earlier ones.
      auto issue_s = [&](int j, int hh) {  // S = Q K^T over 64 keys of tile j
        uint64_t qd = smem_desc_sw128(q_tile(x), 16, 1024);
        uint64_t kd = smem_desc_sw128(slot_addr((2 * (gt + j)) % C::kSlots) + (1 - hh) * 64 * 128,
                                      16, 1024);
        asm volatile("" : "+l"(qd), "+l"(kd));
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          const uint64_t ad = qd + (((ks >> 2) * (C::kRows * 128) + (ks & 3) * 32) >> 4);
          const uint64_t bd = kd + (((ks >> 2) * (C::TN * 128) + (ks & 3) * 32) >> 4);
          mma_f16_ss_warp(sx + 64u * (s_n & 1), ad, bd, kIdescS, ks > 0);
        }
        mma_commit_warp(bar(kS2SFull + 2 * x + (s_n & 1)));
        ++s_n;
      };
      auto issue_pv = [&](int j, int hh) {  // O += P V over 64 keys, P from TMEM
        uint64_t vd = smem_desc_sw128(slot_addr((2 * (gt + j) + 1) % C::kSlots), C::TN * 128, 1024);
        asm volatile("" : "+l"(vd));
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint64_t bd = vd + ((((1 - hh) * 4 + ks) * 2048) >> 4);
          mma_f16_ts_warp(ox, sx + 64u * (p_n & 1) + ks * 8, bd, C::kIdescPV,
                          (2 * j + hh > from || ks > 0) ? 1u : 0u);
        }
        mma_commit_warp(bar(kS2PV + 2 * x + (p_n & 1)));
        ++p_n;
      };
      // Rows of tokens that no row of the item sees (outside [kv_lo, kv_len), or in holes) may hold
      // anything. Of V: P is zero there, but 0 * NaN is not, so they are cleared before the tile's
      // first P.V. Of K: their scores are masked, but a cap chooses its form by all scores of a
      // warp, so it must not see them either. Both MMA warps clear, with the same zeros.
      auto clear_rows = [&](int j, int item) {
        const int first = j == it.nt_max - 1 ? max(it.kv_lo - tile_token(it, j), 0) : 0;
        const int end = j == 0 ? min(it.kv_len - tile_token(it, j), C::TN) : C::TN;
        if (first == 0 && end == C::TN && !(kFirst && it.holes)) return;
        unsigned seen = bits_between(first - 32 * lane, end - 1 - 32 * lane);
        if (kFirst && it.holes)
          seen = seen_word<C::TN>(a.s, it.q0, it.ctx - it.n, it.tok0_a,
                                  min(it.tok0_b + a.qt, it.n), it.prefix, tile_token(it, j));
        uint8_t *at = sgen + C::kRingOff + (item % C::kSlots) * C::kSlotBytes;
#pragma unroll 1
        for (int c = lane; c < C::TN * 8; c += 32) {  // 16-byte chunks of a column block
          const int r = c >> 3;
          if (kFirst ? any_seen(seen, r, 1) : r >= first && r < end) continue;
#pragma unroll
          for (int kb = 0; kb < C::KB; ++kb)
            *reinterpret_cast<uint4 *>(at + kb * (C::TN * 128) + c * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
        __syncwarp();
      };
      // A tile's K has landed (and is cleared) from here on.
      auto wait_keys = [&](int j) {
        if (!wait_ring(2 * (gt + j))) return false;
        if constexpr ((kParts & kRuleCap) != 0) clear_rows(j, 2 * (gt + j));
        return true;
      };
      // Every ring item is waited for and released by both MMA warps, used or not, so that a
      // slot's phases stay in step with both; a commit after unused items completes at once.
      ok = pipe_wait(bar(kS2QFull), q_waits & 1, abort_flag, a.err);
      ++q_waits;
      tc_fence_after();
      // the first scores overwrite buffers from which the previous item's last P.V read P: those
      // MMAs were issued earlier by this thread and so run first
      if (ok) ok = wait_keys(0);
      if (!ok) break;
      if (from == 0 && to > 0) issue_s(0, 0);
      if (from <= 1 && to > 1) issue_s(0, 1);
      release(2 * gt);
      if (it.nt_max == 1) mma_commit_warp(bar(kS2QEmpty));
      for (int j = 0; j < it.nt_max && ok; ++j) {
        // whether some unit of tile j + 1 is this query tile's
        const bool next = j + 1 < it.nt_max && from < 2 * j + 4 && 2 * j + 2 < to;
        ok = wait_ring(2 * (gt + j) + 1);
        if (!ok) break;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int u = 2 * j + hh;
          if (ok && from <= u && u < to) {
            ok = pipe_wait(bar(kS2PFull + 2 * x + (p_n & 1)), (p_n >> 1) & 1, abort_flag, a.err);
            if (ok) {
              tc_fence_after();
              if (hh == 0 || u == from) clear_rows(j, 2 * (gt + j) + 1);
              issue_pv(j, hh);
            }
          }
          if (ok && next) {
            if (hh == 0) ok = wait_keys(j + 1);
            if (ok && from <= u + 2 && u + 2 < to) issue_s(j + 1, hh);
          }
        }
        if (ok && !next && j + 1 < it.nt_max) ok = wait_ring(2 * (gt + j) + 2);
        if (!ok) break;
        release(2 * (gt + j) + 1);
        if (j + 1 < it.nt_max) {
          release(2 * (gt + j) + 2);
          if (j + 2 == it.nt_max) mma_commit_warp(bar(kS2QEmpty));
        }
      }
      gt += it.nt_max;
    }
    mma_commit_warp(bar(kS2Done + x));
    if (lane == 0) drain_wait(bar(kS2Done + x), 0, a.err);
    __syncwarp();
  } else if (warp >= 4) {
    regs_increase<kPrefill2BigRegs>();
    // ================= softmax: tile x = (warp - 4) / 4, one query row per thread =================
    const int x = (warp - 4) >> 2;
    const int rg = warp & 3;
    const int row = rg * 32 + lane;
    const int t = row / a.g, h = row - t * a.g;
    const uint32_t lane_off = static_cast<uint32_t>(rg * 32) << 16;
    const uint32_t ts = tmem + lane_off + 128u * x;
    const uint32_t to = tmem + lane_off + 256u + 128u * x;
    int n = 0;  // units done
    bool ok = true;
    for (int k = 0; ok; ++k) {
      Item it;
      ok = take_item(k, it);
      if (!ok || it.stop) break;
      const int from = x ? it.from_b : it.from_a, end = x ? it.to_b : it.to_a;
      const int tok0 = x ? it.tok0_b : it.tok0_a;
      if (!it.rows || tok0 >= it.n) continue;
      const bool valid = row < q_rows && tok0 + t < it.n;
      const size_t out_row = (static_cast<size_t>(it.q0 + tok0 + t) * a.qh + it.kv * a.g + h) * HD;
      if (kFirst && end == 0) {  // no row of the tile sees anything
        if (valid) store_zero_row(a.out16 + out_row, HD);
        continue;
      }
      // rows past the tile's last token repeat it (and are not stored)
      ScoredRow sr = scored_row(a.s, it.q0, it.ctx - it.n, min(tok0 + min(t, a.qt - 1), it.n - 1),
                                it.kv * a.g + h, it.prefix, valid);
      int base = (2 * it.last_tile + 1 - from) * kUnit;  // first token of the unit
      for (int u = from; u < end; ++u, ++n, base -= kUnit) {
        ok = pipe_wait(bar(kS2SFull + 2 * x + (n & 1)), (n >> 1) & 1, abort_flag, a.err);
        if (!ok) break;
        tc_fence_after();
        const ScoredTile2<HD> io = {ts + 64u * (n & 1), to,
                                    bar(kS2PV + 2 * x + ((n - 1) & 1)),
                                    static_cast<uint32_t>(((n - 1) >> 1) & 1), abort_flag, a.err};
        ok = scored_weights<kParts>(a.s, a.scale_log2, sr, base, u > from, io);
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kS2PFull + 2 * x + (n & 1)));
      }
      if (!ok) break;
      ok = pipe_wait(bar(kS2PV + 2 * x + ((n - 1) & 1)), ((n - 1) >> 1) & 1, abort_flag, a.err);
      if (!ok) break;
      tc_fence_after();
      // Rows go straight from TMEM in whole 32-byte sectors where the output allows. Once these
      // loads have returned, O_X may be overwritten by the next item's first P.V, which waits
      // for this warp's next P. The output is read by no kernel here: it leaves L2 first.
      const float inv = sr.l > 0.f ? 1.f / sr.l : 0.f;
      const uint64_t pol = l2_evict_first_policy();
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        float o[32];
        tmem_ld32(to + c * 32, o);
        if (valid) store_half32(a.out16 + out_row + c * 32, o, inv, a.out_v8, pol);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

}  // namespace pa
