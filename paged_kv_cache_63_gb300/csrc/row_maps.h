// row_maps.h -- tensor maps; 4-D ones over a paged cache: (64 columns, rows, heads, column blocks).
#pragma once

#include <cuda.h>

#include "pagedattn.h"

namespace pa {

// Elements and swizzle of a map: fp16, or bytes in blocks of 128 or of 64, swizzled over a block.
enum class MapKind { kHalf, kBytes128, kBytes64 };

// A tensor map with `rank` (3 or 4) dimensions and a byte stride for each but the first. Works in a
// thread that has made no CUDA call yet.
pa_status_t encode_map(CUtensorMap *map, int rank, const void *base, const cuuint64_t *dims,
                       const cuuint64_t *strides, const cuuint32_t *box,
                       MapKind kind = MapKind::kHalf);

// A box is rows_per_box rows of one head times blocks_per_box blocks of 64 columns and lands as
// [blocks][rows][128 bytes], 128-byte swizzled. Coordinates are (0, row, head, block): token-major
// caches have row = page * page_size + slot and the K/V head, head-major ones row = slot and
// head = page * kv_heads + K/V head.
pa_status_t encode_row_map(CUtensorMap *map, const void *cache, const pa_problem_t *p,
                           int rows_per_box, int blocks_per_box);

// The same over a cache of one-byte codes: blocks of 128 columns (of 64, with a 64-byte swizzle, at
// head_dim 64), a box landing as [blocks][rows][128 or 64 bytes].
pa_status_t encode_code_map(CUtensorMap *map, const void *codes, const pa_problem_t *p,
                            int rows_per_box, int blocks_per_box);

}  // namespace pa
