// code_tiles.cuh -- tiles of a quantised cache on their way to the tensor cores of the multi-token
// kernels: the loads of codes and scales, and the conversion to fp16 operands.
//
// A K or V tile lands as codes in the slot that its fp16 form fills, so the ring is no larger than one
// of fp16 tiles, and converting warps rewrite it in place. A block of 128 columns lies where its upper
// 64 go in fp16: a row's codes are then overwritten by that row alone, which all lanes of a warp have
// read before one writes it, and blocks and rows are independent. At head_dim 64, where rows of codes
// are packed more densely than rows of fp16, the codes fill the slot's upper half; a row's fp16 never
// reaches codes of later rows, so one warp converts in ascending order. Each element is one exact
// conversion and one exact product with the row's power of two.
#pragma once

#include "prefill_kernel.cuh"
#include "quant.cuh"

namespace pa {

// Bytes of a code row of one column block, and where a tile's codes start in its slot.
template <int HD, int TN>
struct CodeTile {
  static constexpr int kBlock = HD < 128 ? HD : 128;
  static constexpr int kBlocks = HD / kBlock;
  static constexpr int kOff = HD < 128 ? TN * HD : TN * 128;  // of the first block
  static constexpr int kStep = 2 * TN * 128;                  // from block to block
};

// The scales of a tile's TN tokens from token `tok` on, eight to a lane, into shared memory at `dst`.
// `page` is the page of the lane's box of `rows_per_box` tokens (negative: not loaded, zeroes). Every
// lane arrives on `bar` once its copies have landed. Warp-collective.
template <int TN>
__device__ __forceinline__ void load_scales(uint32_t dst, const uint8_t *scales, int tok, int page,
                                            int rows_per_box, int kv, int kvh, int ps,
                                            uint32_t bar) {
  const int i = (threadIdx.x & 31) * 8;
  const int pg = __shfl_sync(0xffffffffu, page, (i / rows_per_box) & 31);
  if (i < TN) {
    const uint8_t *src =
        scales + scale_place(max(pg, 0), kv, (tok + i) & (ps - 1), kvh, ps);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst + i), "l"(src),
                 "r"(pg >= 0 ? 8u : 0u)
                 : "memory");
  }
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Rewrites rows [row0, row0 + kRows) of a column block from codes to fp16, K-major in blocks of 64,
// 128-byte swizzled; `at` is the slot, plus the block's number times CodeTile::kStep. A lane takes 16
// codes at a time; the lanes of a quarter warp take even chunks of one row and odd places of the
// next, so that no load or store meets a bank twice. The integer pipe, half rate, takes most of it (a
// conversion 2.2 cycles of a scheduler, one of a word's upper half 3.8), and the loop is kept short
// for the instruction cache, which it shares with the softmax: 512 new tokens of 16 contexts at
// head_dim 128 took 428 us with the waits of all roles written out at each place, 355 with short
// ones (prefill_kernel.cuh, pipe_wait). Warp-collective.
template <int HD, int TN, int kRows>
__device__ __forceinline__ void convert_rows(uint32_t at, uint32_t scales, int row0) {
  using C = CodeTile<HD, TN>;
  constexpr int kAtOnce = HD == 64 ? 8 : 4;  // rows that a warp's lanes cover
  // Two steps to a turn, but one at head_dim 256, where the instruction cache misses most (572 us
  // against 597 for two capped prompts of 4096; at 128 two take 357 us, one 361, for the chunks above)
  constexpr bool kTwo = HD < 256;
  constexpr int kSteps = kRows / (kTwo ? 2 * kAtOnce : kAtOnce);
  const int lane = threadIdx.x & 31;
  const int i = lane & 7, q = lane >> 3;
  int r, c;  // row within the first kAtOnce, chunk of 16 codes within the column block
  uint32_t from;
  if constexpr (HD == 64) {
    r = 2 * q + (i >> 2);
    c = i & 3;
    from = at + C::kOff + (row0 + r) * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  } else {
    r = 2 * (q >> 1) + (i >> 2);
    c = (i & 3) + 4 * ((i >> 2) ^ (q & 1));
    from = at + C::kOff + (row0 + r) * 128 + ((c ^ r) << 4);
  }
  // two chunks of fp16, side by side before the swizzle; the second four rows of eight have the
  // swizzle's bit 2 the other way
  constexpr uint32_t kFlip = HD == 64 ? 0 : 64;
  uint32_t to = at + (c >> 2) * (TN * 128) + (row0 + r) * 128 + (((2 * (c & 3)) ^ (r & 7)) << 4);
  uint32_t scale = scales + row0 + r;
  uint4 w0, w1 = {};
  uint32_t e0, e1 = 0;
  auto load = [&]() {
    w0 = lds128_at<0>(from);
    if constexpr (kTwo) w1 = lds128_at<kAtOnce * C::kBlock>(from ^ kFlip);
    e0 = lds8_at<0>(scale);
    if constexpr (kTwo) e1 = lds8_at<kAtOnce>(scale);
  };
  auto store = [&](auto off, const uint4 &w, uint32_t e, uint32_t flip) {
    const uint32_t f = half2_of_scale(e);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[8];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      o[2 * n] = mul_half2(half2_of_low(v[n]), f);
      o[2 * n + 1] = mul_half2(half2_of_high(v[n]), f);
    }
    sts128_at<decltype(off)::value>(to ^ flip, make_uint4(o[0], o[1], o[2], o[3]));
    sts128_at<decltype(off)::value>(to ^ (flip + 16), make_uint4(o[4], o[5], o[6], o[7]));
  };
  load();
#pragma unroll 1
  for (int m = 0; m < kSteps; ++m) {
    const uint4 v0 = w0, v1 = w1;
    const uint32_t f0 = e0, f1 = e1;
    if constexpr (kTwo) {
      from += 2 * kAtOnce * C::kBlock;
      scale += 2 * kAtOnce;
    } else {
      from = (from ^ kFlip) + kAtOnce * C::kBlock;
      scale += kAtOnce;
    }
    if (m + 1 < kSteps) load();  // rows that nothing has overwritten yet
    __syncwarp();
    store(Const<0>{}, v0, f0, 0);
    if constexpr (kTwo) {
      store(Const<kAtOnce * 128>{}, v1, f1, kFlip);
      to += 2 * kAtOnce * 128;
    } else {
      to = (to ^ kFlip) + kAtOnce * 128;
    }
  }
  // the tensor cores read the slot through the asynchronous proxy
  fence_proxy_async();
  __syncwarp();
}

}  // namespace pa
