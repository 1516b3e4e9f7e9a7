// code_tiles.cuh -- tiles of a quantised cache on their way to the tensor cores of the multi-token
// kernels: the loads of codes and scales, and the conversion to fp16 operands.
//
// A K or V tile lands as codes in the upper half of the slot that its fp16 form fills, so the ring is
// no larger than one of fp16 tiles. A converting warp rewrites it in place: for head_dim 128 and 256
// a row's codes lie where the same row's upper columns go, and all lanes of a warp have read a row
// before one writes it; for head_dim 64 (where codes are packed more densely than rows of fp16) a
// row's fp16 never reaches codes of later rows, so one warp converts in ascending order. Each element
// is one exact conversion and one exact product with the row's power of two.
#pragma once

#include "prefill_kernel.cuh"
#include "quant.cuh"

namespace pa {

// Bytes of a code row of one column block, and where a tile's codes start in its slot.
template <int HD, int TN>
struct CodeTile {
  static constexpr int kBlock = HD < 128 ? HD : 128;
  static constexpr int kBlocks = HD / kBlock;
  static constexpr int kOff = TN * HD;
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

// Rewrites rows [row0, row0 + kRows) of a tile from codes to fp16, K-major in column blocks of 64,
// 128-byte swizzled. A lane takes 16 codes at a time; the lanes of a quarter warp take even chunks of
// one row and odd places of the next, so that no load or store meets a bank twice. Warp-collective.
template <int HD, int TN, int kRows>
__device__ __forceinline__ void convert_rows(uint32_t slot, uint32_t scales, int row0) {
  using C = CodeTile<HD, TN>;
  constexpr int kAtOnce = HD == 64 ? 8 : 4;  // rows of an iteration
  constexpr int U = 4;                       // iterations whose loads are issued together
  static_assert(kRows % (kAtOnce * U) == 0, "rows of a converter");
  const int lane = threadIdx.x & 31;
  const int i = lane & 7, q = lane >> 3;
  int r, c;  // row within the iteration, chunk of 16 codes within the column block
  if constexpr (HD == 64) {
    r = 2 * q + (i >> 2);
    c = i & 3;
  } else {
    r = 2 * (q >> 1) + (i >> 2);
    c = (i & 3) + 4 * ((i >> 2) ^ (q & 1));
  }
#pragma unroll 1
  for (int base = row0; base < row0 + kRows; base += kAtOnce * U) {
#pragma unroll
    for (int blk = 0; blk < C::kBlocks; ++blk) {
      uint4 w[U];
      uint32_t f[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int row = base + u * kAtOnce + r;
        const uint32_t at = HD == 64 ? row * 64 + ((c ^ ((row >> 1) & 3)) << 4)
                                     : blk * (TN * 128) + row * 128 + ((c ^ (row & 7)) << 4);
        w[u] = lds128(slot + C::kOff + at);
        uint16_t e;
        asm volatile("ld.shared.u8 %0, [%1];" : "=h"(e) : "r"(scales + row));
        f[u] = half2_of_scales(e, e);
      }
      __syncwarp();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int row = base + u * kAtOnce + r;
        const uint32_t v[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          o[2 * k] = mul_half2(half2_of_low(v[k]), f[u]);
          o[2 * k + 1] = mul_half2(half2_of_high(v[k]), f[u]);
        }
        const uint32_t to = slot + (2 * blk + (c >> 2)) * (TN * 128) + row * 128;
        const int ch = 2 * (c & 3);
        sts128(to + ((ch ^ (row & 7)) << 4), make_uint4(o[0], o[1], o[2], o[3]));
        sts128(to + (((ch + 1) ^ (row & 7)) << 4), make_uint4(o[4], o[5], o[6], o[7]));
      }
      __syncwarp();
    }
  }
  // the tensor cores read the slot through the asynchronous proxy
  fence_proxy_async();
  __syncwarp();
}

}  // namespace pa
