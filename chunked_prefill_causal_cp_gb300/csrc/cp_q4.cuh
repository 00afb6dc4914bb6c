// cp_q4.cuh -- device side of the 4-bit cache format: codes to 16-bit values.
#pragma once

#include <cstdint>
#include <type_traits>

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

template <typename T>
__device__ __forceinline__ uint32_t add2_16(uint32_t a, uint32_t b) {
  typedef typename Two<T>::type V;
  const V r = __hadd2(*reinterpret_cast<V*>(&a), *reinterpret_cast<V*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t mul2_16(uint32_t a, uint32_t b) {
  typedef typename Two<T>::type V;
  const V r = __hmul2(*reinterpret_cast<V*>(&a), *reinterpret_cast<V*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t fma2_16(uint32_t a, uint32_t b, uint32_t c) {
  typedef typename Two<T>::type V;
  const V r = __hfma2(*reinterpret_cast<V*>(&a), *reinterpret_cast<V*>(&b), *reinterpret_cast<V*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A group's parameters ready for q4_four: (s, s), (m, m), and for bf16 (4 s, 4 s)
// -- or of two groups side by side, one per half.
struct Q4Scale {
  uint32_t s, m, s4;
};
template <typename T>
__device__ __forceinline__ Q4Scale q4_scale(uint32_t s2, uint32_t m2) {
  return Q4Scale{s2, m2, std::is_same<T, __nv_bfloat16>::value ? mul2_16<T>(s2, 0x40804080u) : 0u};
}

// The codes of nibbles 0 .. 3 of both halves of `w` -> m + c * s in the layer's
// type, r[i] for nibble i of the low and the high half, each rounded once.
// Nibbles 0 and 2 go under an exponent whose last place is one, the offset is
// subtracted exactly, and one fused multiply-add follows.  Nibbles 1 and 3 need no
// shift of their own: in fp16 they stand under the same exponent times 16, and a
// multiply-add takes the code out exactly; in bf16 the bits [4, 8) alone are the
// number 16 c 2^-133 (below the smallest normal exponent and in the first above it
// the bits count evenly), and 2^127 makes it c / 4 exactly (4 s is finite: s is at
// most a 15th of the largest value).
template <typename T>
__device__ __forceinline__ void q4_four(uint32_t w, const Q4Scale& p, uint32_t magic, uint32_t (&r)[4]) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t x = i == 0 ? w : w >> 8;
    uint32_t lo, hi;
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(lo) : "r"(x), "r"(magic));  // (x & mask) | magic
    r[i] = fma2_16<T>(add2_16<T>(lo, Two<T>::kMagic | 0x80008000u), p.s, p.m);
    if constexpr (kBf16) {
      hi = x & 0x00f000f0u;
      r[i + 1] = fma2_16<T>(mul2_16<T>(hi, 0x7f007f00u), p.s4, p.m);
    } else {
      asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(hi) : "r"(x), "r"(magic));
      r[i + 1] = fma2_16<T>(fma2_16<T>(hi, 0x2c002c00u, 0xd400d400u), p.s, p.m);  // / 16 - 64
    }
  }
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
