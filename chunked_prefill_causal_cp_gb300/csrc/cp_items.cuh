// cp_items.cuh -- what the persistent attention kernels of latent caches and drafted
// trees share: the order in which a CTA takes its items, and bits of masks and values.
#pragma once

#include <cstdint>
#include <type_traits>

#include "cp_internal.h"
#include "cp_rows.cuh"

namespace cp {

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const float x[2] = {lo, hi};
  return Pack<T>::store(x);
}

// Whether one of the eight 16-bit values is not finite.
template <typename T>
__device__ __forceinline__ bool nonfinite8(const uint4& v) {
  constexpr uint32_t kExp = std::is_same<T, __nv_bfloat16>::value ? 0x7f807f80u : 0x7c007c00u;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t e = w[i] & kExp;
    bad = bad || (e & 0xffffu) == (kExp & 0xffffu) || (e >> 16) == (kExp >> 16);
  }
  return bad;
}

// 64 bits from bit `from` of a 128-bit number on (bits outside it are 0).
__device__ __forceinline__ uint64_t bits_from(uint64_t lo, uint64_t hi, int from) {
  if (from <= -64 || from >= 128) return 0;
  if (from < 0) return lo << -from;
  if (from == 0) return lo;
  if (from < 64) return (lo >> from) | (hi << (64 - from));
  return hi >> (from - 64);
}

// The even bits of a word.
__device__ __forceinline__ uint32_t even_bits(uint32_t x) {
  x &= 0x55555555u;
  x = (x | x >> 1) & 0x33333333u;
  x = (x | x >> 2) & 0x0f0f0f0fu;
  x = (x | x >> 4) & 0x00ff00ffu;
  return (x | x >> 8) & 0xffffu;
}

// This CTA's items, in order: of all items, numbered over the sequences, those at
// blockIdx.x, then back and forth in rounds of gridDim.x, so that a CTA with a heavy item
// in one round has a light one in the next.  A whole warp asks.
template <typename Work>
struct ItemCursor {
  long long base = 0;      // items of the chunks of 32 sequences before
  int q0 = 0, round = 0;
  long long weight, upto;  // of this lane's sequence; items of the chunk up to and including it
  __device__ __forceinline__ explicit ItemCursor(const Work& wk) { load(wk); }
  __device__ __forceinline__ void load(const Work& wk) {
    const int lane = threadIdx.x & 31;
    weight = q0 + lane < wk.rows.num_seqs ? wk.weight(q0 + lane, blockIdx.x == 0) : 0;
    upto = weight;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
  }
  template <typename Item>
  __device__ __forceinline__ bool next(const Work& wk, Item& x) {
    for (;;) {
      const long long r = (long long)round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      long long total;
      while (r - base >= (total = __shfl_sync(0xffffffffu, upto, 31))) {
        base += total;
        q0 += 32;
        if (q0 >= wk.rows.num_seqs) return false;
        load(wk);
      }
      const int L = __ffs(__ballot_sync(0xffffffffu, upto > r - base)) - 1;
      ++round;
      if (wk.make(q0 + L, r - base - __shfl_sync(0xffffffffu, upto - weight, L), r, x)) return true;
    }
  }
};

}  // namespace cp
