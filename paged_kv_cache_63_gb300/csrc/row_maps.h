// row_maps.h -- tensor maps; 4-D ones over a paged cache: (64 columns, rows, heads, column blocks).
#pragma once

#include <cuda.h>

#include "pagedattn.h"

namespace pa {

// A tensor map over fp16 with 128-byte swizzle, `rank` (3 or 4) dimensions and a byte stride for
// each but the first. Works in a thread that has made no CUDA call yet.
pa_status_t encode_map(CUtensorMap *map, int rank, const void *base, const cuuint64_t *dims,
                       const cuuint64_t *strides, const cuuint32_t *box);

// A box is rows_per_box rows of one head times blocks_per_box blocks of 64 columns and lands as
// [blocks][rows][128 bytes], 128-byte swizzled. Coordinates are (0, row, head, block): token-major
// caches have row = page * page_size + slot and the K/V head, head-major ones row = slot and
// head = page * kv_heads + K/V head.
pa_status_t encode_row_map(CUtensorMap *map, const void *cache, const pa_problem_t *p,
                           int rows_per_box, int blocks_per_box);

}  // namespace pa
