// row_maps.cpp -- the library's tensor maps: rows of heads in 64-column blocks.
#include "row_maps.h"

#include <cuda_runtime.h>

#include <atomic>

namespace pa {

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
  static std::atomic<EncodeTiledFn> known{nullptr};
  EncodeTiledFn fn = known.load(std::memory_order_acquire);
  if (!fn) {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    fn = reinterpret_cast<EncodeTiledFn>(p);
    known.store(fn, std::memory_order_release);
  }
  return fn;
}

}  // namespace

pa_status_t encode_map(CUtensorMap *map, int rank, const void *base, const cuuint64_t *dims,
                       const cuuint64_t *strides, const cuuint32_t *box) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return PA_ERR_CUDA;
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  auto encode = [&] {
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, static_cast<cuuint32_t>(rank),
              const_cast<void *>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult rc = encode();
  if (rc == CUDA_ERROR_INVALID_CONTEXT) {
    // a thread has a context only once a call of the runtime has needed one: this may be its first
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return PA_ERR_CUDA;
    rc = encode();
  }
  return rc == CUDA_SUCCESS ? PA_OK : PA_ERR_CUDA;
}

pa_status_t encode_row_map(CUtensorMap *map, const void *cache, const pa_problem_t *p,
                           int rows_per_box, int blocks_per_box) {
  const bool hm = p->cache_layout == PA_LAYOUT_HEAD_MAJOR;
  const cuuint64_t row = static_cast<cuuint64_t>(p->head_dim) * 2;  // bytes of a head's row
  const cuuint64_t pages = p->num_physical_pages, ps = p->page_size, heads = p->kv_heads;
  const cuuint64_t dims[4] = {64, hm ? ps : pages * ps, hm ? pages * heads : heads,
                              static_cast<cuuint64_t>(p->head_dim / 64)};
  const cuuint64_t strides[3] = {hm ? row : heads * row, hm ? ps * row : row, 128};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows_per_box), 1,
                             static_cast<cuuint32_t>(blocks_per_box)};
  return encode_map(map, 4, cache, dims, strides, box);
}

}  // namespace pa
