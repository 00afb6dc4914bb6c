// cp_host.h -- host helpers of the C-ABI layer: the checks of a layer
// description, the views built from it, and tensor maps.
#pragma once

#include <cmath>
#include <cstdint>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "cp_internal.h"

namespace cp {

inline int esize_of(int dtype) { return dtype == CP_F32 ? 4 : 2; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int check_desc(const cp_layer_desc* d, bool need_batch) {
  if (d == nullptr) return CP_ERR_INVALID_ARG;
  if (d->dtype != CP_F32 && d->dtype != CP_BF16 && d->dtype != CP_F16) return CP_ERR_INVALID_ARG;
  if (need_batch && d->batch <= 0) return CP_ERR_INVALID_ARG;
  if (d->num_q_heads <= 0 || d->num_kv_heads <= 0) return CP_ERR_INVALID_ARG;
  if (d->num_q_heads % d->num_kv_heads != 0) return CP_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return CP_ERR_UNSUPPORTED;
  if (!(d->scale >= 0.f) || std::isinf(d->scale)) return CP_ERR_INVALID_ARG;
  switch (d->kind) {
    case CP_CACHE_CONTIG:
    case CP_CACHE_ROLLING:
      if (d->capacity <= 0) return CP_ERR_INVALID_ARG;
      break;
    case CP_CACHE_PAGED:
      if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128)
        return CP_ERR_UNSUPPORTED;
      if (d->num_pages <= 0 || d->max_blocks <= 0) return CP_ERR_INVALID_ARG;
      break;
    default:
      return CP_ERR_INVALID_ARG;
  }
  return CP_OK;
}

// Upper bound of positions a sequence may reach in this layout.
inline int64_t layout_limit(const cp_layer_desc* d) {
  if (d->kind == CP_CACHE_CONTIG) return d->capacity;
  if (d->kind == CP_CACHE_PAGED) return (int64_t)d->max_blocks * d->page_size;
  return INT32_MAX;  // rolling: positions grow without bound, slots wrap
}

inline CacheView make_cache(const cp_layer_desc* d, const int32_t* block_table) {
  CacheView c;
  c.kind = d->kind;
  c.capacity = d->capacity;
  c.page_size = d->page_size;
  c.num_pages = d->num_pages;
  c.max_blocks = d->max_blocks;
  c.block_table = block_table;
  return c;
}

inline float scale_log2(const cp_layer_desc* d) {
  const double sc = d->scale > 0.f ? (double)d->scale : 1.0 / std::sqrt((double)d->head_dim);
  return (float)(sc * 1.4426950408889634);  // log2(e)
}

// ---- tensor maps (driver entry point fetched through the runtime)

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 3-D tensor of 16-bit elements: dims {d0 (contiguous), d1, d2}, 128-byte
// swizzled boxes; out-of-range box elements read as zero.
inline bool encode_3d(CUtensorMap* m, int dtype, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
               uint32_t b0, uint32_t b1, uint32_t b2) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {d0 * 2, d0 * d1 * 2};
  const cuuint32_t box[3] = {b0, b1, b2};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType ty =
      dtype == CP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return fn(m, ty, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int launch_result(cudaError_t e) { return e == cudaSuccess ? CP_OK : CP_ERR_CUDA; }

}  // namespace cp
