// prefill_common.cuh -- what the multi-token kernels share: arguments, bounded pipeline waits,
// L2 policies, packed fp32 arithmetic, sector stores and cluster launch control.
#pragma once

#include "device_common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace pa {

struct PrefillArgs {
  const int32_t *qs;   // [batch + 1] first query row of each sequence
  const int32_t *bt;   // [batch][maxp]
  const int32_t *ctx;  // [batch] tokens in the cache, the new ones included
  float *out;          // [total][qh][hd]
  unsigned *err;
  long long total;  // rows of query and out
  int batch, qh, kvh, ps, ps_shift, maxp, num_pages, layout;
  int g;         // query heads per K/V head
  int qt;        // new tokens per query tile (128 / g)
  int n_qtiles;  // grid.z
  float scale_log2;
  int expire;  // PA_TEST_EXPIRE_WAITS: the MMA warp's first wait is on a barrier that
               // completes only at the end, so it runs out
  int out_v8;  // out is 32-byte aligned: the two-tile kernel writes rows in 32-byte stores
};

// O is rescaled only when a row's running maximum grows by more than 2^kPrefillSlackLog2;
// until then every exponent term is at most kPrefillSlackBound, which a tile's row sum may
// therefore be checked against.
constexpr int kPrefillSlackLog2 = 8;
constexpr float kPrefillRescaleSlack = static_cast<float>(kPrefillSlackLog2);  // log2 units
constexpr float kPrefillSlackBound = static_cast<float>(1 << kPrefillSlackLog2);

// L2 policy for bytes that other CTAs read again soon: keep them ahead of streamed data.
__device__ __forceinline__ uint64_t l2_evict_last_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

__device__ __forceinline__ float prefill_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Packed fp32 pairs (sm_100 family): one instruction does two FMAs or two adds.
__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mov.b64 rc, {%6, %7};\n\tfma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// 32-byte store (one full sector) of 8 floats with an L2 eviction-priority policy.
__device__ __forceinline__ void st_global_v8(float *p, float v0, float v1, float v2, float v3,
                                             float v4, float v5, float v6, float v7, uint64_t pol) {
  asm volatile(
      "st.global.L2::cache_hint.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8}, %9;" ::"l"(p),
      "f"(v0), "f"(v1), "f"(v2), "f"(v3), "f"(v4), "f"(v5), "f"(v6), "f"(v7), "l"(pol)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Warp-collective bounded wait that also gives up when another role has aborted.
__device__ __forceinline__ bool pipe_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                          unsigned *err) {
  bool ok = mbar_try_wait(bar, parity);
  bool expired = false;
  if (!ok) {
    const uint64_t t0 = global_ns();
    for (uint32_t i = 1;; ++i) {
      if (mbar_try_wait(bar, parity)) {
        ok = true;
        break;
      }
      if ((i & 31u) == 0) {
        if (*abort_flag) break;
        if (global_ns() - t0 > kWaitLimitNs) {
          expired = true;
          break;
        }
      }
    }
  }
  ok = __all_sync(0xffffffffu, ok);
  expired = __any_sync(0xffffffffu, expired);
  if (!ok && (threadIdx.x & 31) == 0) {
    if (expired) atomicOr(err, PA_DEVERR_TIMEOUT);
    *abort_flag = 1;
  }
  return ok;
}

// Bounded wait used while draining (ignores the abort flag).
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, unsigned *err) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = global_ns();
    for (uint32_t i = 1;; ++i) {
      if (mbar_try_wait(bar, parity)) {
        ok = true;
        break;
      }
      if ((i & 31u) == 0 && global_ns() - t0 > kWaitLimitNs) break;
    }
  }
  if (!ok) atomicOr(err, PA_DEVERR_TIMEOUT);
}

// ---- cluster launch control -------------------------------------------------------------
// Ask for one CTA of this grid that has not started to be cancelled so that the caller runs
// its work; the 16-byte answer is written to shared memory and completes `bar` with 16 bytes
// of transaction count.
__device__ __forceinline__ void clc_try_cancel(uint32_t answer, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128"
      " [%0], [%1];" ::"r"(answer), "r"(bar)
      : "memory");
}

// Read an answer: true and the cancelled CTA's index if a CTA was cancelled, false when
// every CTA of the grid has started (no work is left to take).
__device__ __forceinline__ bool clc_query(uint32_t answer, int &x, int &y, int &z) {
  uint32_t ok, cx = 0, cy = 0, cz = 0;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\tld.shared.b128 r, [%4];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %3, 1, 0, p;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, %1, %2, _}, r;\n\t}"
      : "+r"(cx), "+r"(cy), "+r"(cz), "=r"(ok)
      : "r"(answer)
      : "memory");
  x = static_cast<int>(cx);
  y = static_cast<int>(cy);
  z = static_cast<int>(cz);
  return ok != 0;
}

}  // namespace pa
