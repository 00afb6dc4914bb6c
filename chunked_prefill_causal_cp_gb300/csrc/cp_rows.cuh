// cp_rows.cuh -- which sequence a row belongs to, where its position lives in
// the cache, and conversions between a layer's type and fp32.  Shared by the
// kernels around 4-bit caches, latent caches and drafted trees.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cp_internal.h"

namespace cp {

// The sequence of a row: the last s with cu_rows[s] <= row.
__device__ __forceinline__ int row_seq(const SeqRows& r, int row) {
  if (r.rows_uniform > 0) return row / r.rows_uniform;
  int lo = 0, hi = r.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (r.cu_rows[mid] <= row) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Place of a row within its sequence s, or -1 when it belongs to none (rows
// before the first offset or from the last one on: a padded batch).
__device__ __forceinline__ int row_place(const SeqRows& r, int s, int row) {
  const int i = row - seq_row0(r, s);
  return i < seq_rows(r, s) ? i : -1;
}

// A sequence within a call's bounds: its rows, positions before them, first row.  Calls skip the others.
__device__ __forceinline__ bool seq_bounds(const SeqRows& rows, const int* past, int total_rows, int max_ctx, int s, int& r,
                                           int& p, int& row0) {
  r = seq_rows(rows, s);
  if (r < 1) return false;
  p = past[s];
  row0 = seq_row0(rows, s);
  return p >= 0 && (long long)p + r <= max_ctx && row0 >= 0 && row0 <= total_rows - r;
}

// Index of the (position, KV head) row of sequence s in a cache array, in rows,
// or -1 when the host bound or the layout does not allow the position.
__device__ __forceinline__ long long cache_row(const CacheView& c, int hkv, int s, int g, long long pos, int max_ctx) {
  if (pos < 0 || pos >= max_ctx) return -1;
  const int p = (int)pos;  // below max_ctx
  if (c.kind == CP_CACHE_PAGED) {
    const int lps = 31 - __clz(c.page_size);  // a power of two
    const int blk = p >> lps;
    if (blk >= c.max_blocks) return -1;
    const int page = c.block_table[(long long)s * c.max_blocks + blk];
    if (page < 0 || page >= c.num_pages) return -1;
    return (((long long)page * hkv + g) << lps) + (p & (c.page_size - 1));
  }
  if (c.kind == CP_CACHE_CONTIG && p >= c.capacity) return -1;
  return ((long long)s * hkv + g) * c.capacity + (c.kind == CP_CACHE_ROLLING ? p % c.capacity : p);
}

// A 32-bit word of two 16-bit elements, or one fp32, as floats and back.
template <typename T>
struct Pack;
template <>
struct Pack<float> {
  static constexpr int kPerWord = 1;
  static __device__ __forceinline__ void load(uint32_t w, float* x) { x[0] = __uint_as_float(w); }
  static __device__ __forceinline__ uint32_t store(const float* x) { return __float_as_uint(x[0]); }
};
template <>
struct Pack<__nv_bfloat16> {
  static constexpr int kPerWord = 2;
  static __device__ __forceinline__ void load(uint32_t w, float* x) {
    x[0] = __uint_as_float(w << 16);
    x[1] = __uint_as_float(w & 0xffff0000u);
  }
  static __device__ __forceinline__ uint32_t store(const float* x) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[0], x[1]);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
template <>
struct Pack<__half> {
  static constexpr int kPerWord = 2;
  static __device__ __forceinline__ void load(uint32_t w, float* x) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
    x[0] = v.x;
    x[1] = v.y;
  }
  static __device__ __forceinline__ uint32_t store(const float* x) {
    const __half2 v = __floats2half2_rn(x[0], x[1]);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

// 16 bytes as floats and back.
template <typename T>
__device__ __forceinline__ void unpack16(const uint4& v, float* x) {
  constexpr int P = Pack<T>::kPerWord;
  Pack<T>::load(v.x, x);
  Pack<T>::load(v.y, x + P);
  Pack<T>::load(v.z, x + 2 * P);
  Pack<T>::load(v.w, x + 3 * P);
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const float* x) {
  constexpr int P = Pack<T>::kPerWord;
  return make_uint4(Pack<T>::store(x), Pack<T>::store(x + P), Pack<T>::store(x + 2 * P), Pack<T>::store(x + 3 * P));
}

// Two fp32 operations in one instruction, each rounded as alone.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

}  // namespace cp
