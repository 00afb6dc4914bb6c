// cp_q4.cuh -- device side of the 4-bit cache format: codes to 16-bit values.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace cp {

// Two 16-bit elements in a word, by layer type.
template <typename T>
struct Two;
template <>
struct Two<__nv_bfloat16> {
  typedef __nv_bfloat162 type;
  static constexpr uint32_t kExponent = 0x7f80u;
  static constexpr uint32_t kMagic = 0x43004300u;  // 128: a code in the low mantissa bits is 128 + code
};
template <>
struct Two<__half> {
  typedef __half2 type;
  static constexpr uint32_t kExponent = 0x7c00u;
  static constexpr uint32_t kMagic = 0x64006400u;  // 1024
};

// The offset in a register that the compiler does not know to be constant: with
// two constants the and-or below came out as two instructions.
template <typename T>
__device__ __forceinline__ uint32_t q4_magic() {
  return Two<T>::kMagic + (blockDim.x >> 16);
}

// Codes in bits [0, 4) and [16, 20) of `w` (other bits may be set) -> m + c * s
// for both, rounded once: the code goes under an exponent whose last place is
// one, the offset is subtracted exactly, and one fused multiply-add follows.
template <typename T>
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, uint32_t s2, uint32_t m2, uint32_t magic) {
  typedef typename Two<T>::type V;
  uint32_t x;
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(x) : "r"(w), "r"(magic));  // (w & mask) | magic
  const V c = __hsub2(*reinterpret_cast<V*>(&x), *reinterpret_cast<V*>(&magic));
  const V r = __hfma2(c, *reinterpret_cast<V*>(&s2), *reinterpret_cast<V*>(&m2));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// (s, m) of one group -> the pairs (s, s) and (m, m).
__device__ __forceinline__ uint32_t q4_scale2(uint32_t params) { return __byte_perm(params, params, 0x1010); }
__device__ __forceinline__ uint32_t q4_low2(uint32_t params) { return __byte_perm(params, params, 0x3232); }

// Whether a group's scale or smallest value is a NaN or an infinity.
template <typename T>
__device__ __forceinline__ bool q4_nonfinite(uint32_t params) {
  constexpr uint32_t kExp = Two<T>::kExponent;
  return (params & kExp) == kExp || ((params >> 16) & kExp) == kExp;
}

}  // namespace cp
