// cp_rope.cuh -- sines and cosines of rotary positions, shared by the kernels that rotate.
//
// Angles: inv_freq is turned into a 64-bit fixed-point fraction of a turn per
// position (integer product of its significand with 2^66 / 2 pi), so
// position * step mod 2^64 is the angle mod one turn for any int32 position,
// with no reduction error to speak of.  The nearest quarter turn comes off in whole
// numbers too, and the top 32 bits of the rest, at most an eighth of a turn, go to
// sincospif as a float: the angle's error is below 2^-25 (half a unit of that float,
// 2^-25.4, and the cut bits), whatever the position.  (With the whole turn as one float it
// was 2^-23.3, and 8192 rows took 29.9 instead of 30.1 us.)
#pragma once

#include <cstdint>

namespace cp {

// Turns per position, as a 64-bit fraction (mod one turn), of |f| radians per
// position: f = m 2^e, and m * (2^66 / 2 pi) fits 88 bits.
__device__ __forceinline__ uint64_t turn_step(float f) {
  constexpr uint64_t kTurns66 = 11743562013128004906ull;  // 2^66 / (2 pi)
  const uint32_t b = __float_as_uint(f);
  const int ex = (b >> 23) & 255;
  const uint64_t m = (b & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int shift = 152 - (ex ? ex : 1);  // right shift of m * kTurns66: 2 - e
  const uint64_t hi = __umul64hi(m, kTurns66), lo = m * kTurns66;
  uint64_t r;
  if (shift >= 128) r = 0;
  else if (shift >= 64) r = hi >> (shift - 64);
  else if (shift > 0) r = (hi << (64 - shift)) | (lo >> shift);
  else r = shift > -64 ? lo << -shift : 0;
  return (b >> 31) ? 0 - r : r;
}

// Sine and cosine of a fraction of a turn.
__device__ __forceinline__ void sincos_turns(uint64_t turns, float* sn, float* cs) {
  float s, c;
  sincospif((float)(int)(turns >> 30) * 0x1p-33f, &s, &c);  // the rest: bits 30 to 61, signed
  const uint32_t q = (uint32_t)((turns + (1ull << 61)) >> 62);
  const float a = q & 1 ? c : s, b = q & 1 ? s : c;  // of q quarter turns more
  *sn = q & 2 ? -a : a;
  *cs = (q + 1) & 2 ? -b : b;
}

}  // namespace cp
