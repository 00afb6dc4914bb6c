// cp_items.cuh -- what the persistent attention kernels of latent caches and drafted
// trees share: the order in which a CTA takes its items, and bits of masks and values.
#pragma once

#include <cstdint>
#include <type_traits>

#include "cp_latent.h"
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

// ---- which items a persistent CTA takes.  A whole warp asks; a lane has the numbers of one of
// 32 sequences at a time.

// An inclusive prefix sum over the lanes of a warp.
__device__ __forceinline__ long long warp_prefix(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Items by their numbers over the sequences, weight(s) of sequence s (0: it is skipped), of
// which make(s, i, x) describes the i-th: those at blockIdx.x, then back and forth in
// rounds of gridDim.x, so that a CTA with a heavy item in one round has a light one in
// the next.
template <typename Work>
struct TurnCursor {
  long long base = 0;      // items of the chunks of 32 sequences before
  int q0 = 0, round = 0;
  long long weight, upto;  // of this lane's sequence; items of the chunk up to and including it
  __device__ __forceinline__ explicit TurnCursor(const Work& wk) { load(wk); }
  __device__ __forceinline__ void load(const Work& wk) {
    const int s = q0 + (threadIdx.x & 31);
    weight = s < wk.rows.num_seqs ? wk.weight(s, blockIdx.x == 0) : 0;
    upto = warp_prefix(weight);
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
      const int at = __ffs(__ballot_sync(0xffffffffu, upto > r - base)) - 1;
      ++round;
      if (wk.make(q0 + at, r - base - __shfl_sync(0xffffffffu, upto - weight, at), x)) return true;
    }
  }
};

// A call's tiles of keys, kStart a unit among them: of sequence s, with units(s) units (0: it is skipped) of key_tiles(s);
// of all.
template <typename Work>
__device__ __forceinline__ int slots_of(const Work& wk, int s, bool report, int& units) {
  units = s < wk.rows.num_seqs ? wk.units(s, report) : 0;
  return units > 0 ? kStart + wk.key_tiles(s) : 1;
}
template <typename Work>
__device__ __forceinline__ long long all_tiles(const Work& wk, bool report) {
  long long all = 0;
  for (int s = threadIdx.x & 31; s < wk.rows.num_seqs; s += 32) {
    int units;
    const int each = slots_of(wk, s, report, units);
    all += (long long)units * each;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  return all;
}

// This CTA's share of the call's tiles of keys (see cp_latent.h), unit by unit: sequence s has
// units(s) (0: it is skipped) of key_tiles(s) tiles each; make(s, unit, k0, n, x) describes n
// tiles of one from tile k0 on.
template <typename Work>
struct ShareCursor {
  long long base = 0;         // of the chunks of 32 sequences before; counted in tiles, kStart a unit among them
  long long at, end;          // next, the share's end
  int q0 = 0;
  long long sum;              // of this lane's sequence: the chunk's up to and including it,
  int each;                   // of a unit,
  long long mine;             // of the sequence
  __device__ __forceinline__ explicit ShareCursor(const Work& wk) {
    long long all;
    if (wk.rows.num_seqs <= 32) {
      load(wk, blockIdx.x == 0);
      all = __shfl_sync(0xffffffffu, sum, 31);
    } else {
      all = all_tiles(wk, blockIdx.x == 0);
      load(wk, false);
    }
    const Shares shares(all, wk.ctas);  // as the merge has them: the grid is wk.ctas
    const int c = min((int)blockIdx.x, shares.ctas);
    at = shares.begin(c);
    end = shares.begin(min(c + 1, shares.ctas));
  }
  __device__ __forceinline__ void load(const Work& wk, bool report) {
    int units;
    each = slots_of(wk, q0 + (threadIdx.x & 31), report, units);
    mine = (long long)units * each;
    sum = warp_prefix(mine);
  }
  template <typename Item>
  __device__ __forceinline__ bool next(const Work& wk, Item& x) {
    while (at < end) {
      const uint32_t some = __ballot_sync(0xffffffffu, base + sum > at);
      if (!some) {
        base += __shfl_sync(0xffffffffu, sum, 31);
        q0 += 32;
        if (q0 >= wk.rows.num_seqs) return false;
        load(wk, false);
        continue;
      }
      const int lane = __ffs(some) - 1, n = __shfl_sync(0xffffffffu, each, lane);
      const long long off = at - base - __shfl_sync(0xffffffffu, sum - mine, lane), unit = Shares::quotient(off, n);
      const int o = (int)(off - unit * n), len = (int)min((long long)(n - o), end - at);
      const int k0 = max(o - kStart, 0), k1 = max(o + len - kStart, 0);
      x.whole = k0 == 0 && k1 == n - kStart;
      x.part = 2 * blockIdx.x + (k0 == 0);
      at += len;
      if (k1 > k0 && wk.make(q0 + lane, (int)unit, k0, k1 - k0, x)) return true;
    }
    return false;
  }
};

// What a CTA of a merging kernel does: unit `nth` of the call, or (by_share, where units are more than shares) the one
// that share nth leaves to the next.
template <typename Work>
struct MergedUnit {
  int s = -1, unit;      // sequence (-1: none), unit of it
  int n;                 // its tiles
  long long all, first;  // tiles of the call; of them, the first of the unit's
  __device__ __forceinline__ MergedUnit(const Work& wk, int nth, bool by_share, int grid) {
    int q0 = 0, units, each;
    long long mine, sum, base = 0;
    auto load = [&]() {
      each = slots_of(wk, q0 + (threadIdx.x & 31), false, units);
      mine = (long long)units * each;
      sum = warp_prefix(mine);
    };
    load();
    all = max(wk.rows.num_seqs <= 32 ? __shfl_sync(0xffffffffu, sum, 31) : all_tiles(wk, false), 1ll);
    long long at = nth;
    if (by_share) {
      const Shares shares(all, grid);
      if (nth + 1 >= shares.ctas) return;
      at = shares.begin(nth + 1);
    }
    for (;;) {
      const long long key = by_share ? mine : units, upto = by_share ? sum : warp_prefix(key);
      const long long total = __shfl_sync(0xffffffffu, upto, 31);
      if (at < total) {
        const int lane = __ffs(__ballot_sync(0xffffffffu, upto > at)) - 1;
        const int slots = __shfl_sync(0xffffffffu, each, lane);
        at -= __shfl_sync(0xffffffffu, upto - key, lane);
        s = q0 + lane;
        unit = (int)(by_share ? Shares::quotient(at, slots) : at);
        n = slots - kStart;
        first = base + __shfl_sync(0xffffffffu, sum - mine, lane) + (long long)unit * slots + kStart;
        return;
      }
      at -= total;
      base += __shfl_sync(0xffffffffu, sum, 31);
      q0 += 32;
      if (q0 >= wk.rows.num_seqs) return;
      load();
    }
  }
};

// The CTAs that have a unit's n tiles, from `first` of the call on, of which the first `seen` are computed: those that
// left parts are [from, to], unless one has them all.
struct UnitShares {
  int from, to;
  bool whole;
  __device__ __forceinline__ UnitShares(long long all, long long first, int n, int seen, int grid) {
    const Shares shares(all, grid);
    from = shares.of(first);
    to = shares.of(first + seen - 1);
    whole = shares.of(first + n - 1) == from;
  }
  __device__ __forceinline__ int part(int c) const { return 2 * c + (c == from); }
};

// A sequence's parents of up to CP_TREE_MAX rows, as bytes: one out of range counts as -1 and sets CP_DEV_BOUNDS.
__device__ __forceinline__ void load_parents(const int* parents, int rows, int* status, int8_t* to) {
  for (int m = threadIdx.x & 31; m < rows; m += 32) {
    int up = parents[m];
    if (up < -1 || up >= m) {
      up = -1;
      if (status) atomicOr(status, CP_DEV_BOUNDS);
    }
    to[m] = (int8_t)up;
  }
}
// The rows that row i sees, 128 bits: its ancestors and itself.
__device__ __forceinline__ void ancestors(const int8_t* parents, int i, uint64_t& lo, uint64_t& hi) {
  for (int j = i; j >= 0; j = parents[j]) {
    if (j < 64) lo |= 1ull << j;
    else hi |= 1ull << (j - 64);
  }
}

}  // namespace cp
