// attn_pairs.cuh -- attention of up to 256 query rows at a time over 128-key
// tiles on the sm_103a tensor cores (TMA, tcgen05, TMEM): drafted trees over a K/V
// cache (attn_tree.cu) and chunks over expanded keys and values
// (attn_expanded.cu).
//
// An item is a pair of 128-row Q tiles (each whole tokens of G heads) of one
// sequence and KV head, over a range of its keys; every K/V tile that a CTA loads
// serves both Q tiles.  One persistent CTA an SM, 384 threads:
//   warps 0, 3  TMA producers: an item's Q tiles and the K of each 128-key tile, and its V,
//               in units of 64 channels (16 KB) through a ring of as many units as fit;
//               a tile's K, and its V, land and are given back as one
//   warp 1      MMA issue:  S_w = Q_w K^T, O_w += P_w V for Q tile w = 0, 1
//   warp 2      scheduling: finds this CTA's items, two ahead of the others
//   warps 4-7, 8-11  softmax of Q tile 0 and 1, a thread a row
// TMEM: Q tile w has [256w, 256w + 128) for S and, over it, P in 16 bits;
// [256w + 128, + channels) for O.  S_w(i + 1) is issued after O_w += P_w(i) V(i), and
// tcgen05 operations of one thread complete in order, so S_w(i + 1) complete means
// that P_w(i) may be overwritten and O_w rescaled -- which happens only when a row's
// maximum has grown by more than 2^8.
//
// A lone Q tile (Work::kLone) has both warpgroups, which take its tiles of keys in turn,
// S_w(i) = Q K^T and O_w += P_w(i) V with w = i mod 2: the tensor cores compute one's
// products during the other's softmax, as with a pair.  Their outputs, maxima and sums
// are joined at the end.
//
// What a row does not see: its scores become -inf by a mask of the tile's columns (a
// tree's row: its ancestors, 128 bits found by walking the parents once).  Its weight
// 0 must not meet a NaN or an infinity in V: in tiles with keys that some row of
// the item does not see, V rows past the sequence, and those that hold a non-finite
// value, are overwritten with zeros in shared memory; the rows that see such a key
// become NaN by their sum.
//
// Weights are rounded to the layer's type for O_w += P_w V, and nothing else is before the output (the sums are of the
// weights before their rounding): both operands of that MMA are of one type, and V is multiplied as it lies.  Weights in
// two 16-bit halves would cost a second product, of a path that the tensor cores bound.  What the rounding costs in
// accuracy: see attn_latent.cu.
//
// Measured: see attn_tree.cu and attn_expanded.cu.  With all in place a pair's tile of keys
// takes about 3000 clocks: softmax 1400, then P V and the next Q K^T of its Q tile 1000 to
// 1300, and two hand-overs of 200 to 300, during which the other Q tile has the tensor cores (2050
// clocks of the 3000 at 128 channels, 2560 of 3300 at 192 + 128).  TMEM has no room for a
// second S beside two O of 128 channels.  Slower were P handed over in two halves and exponentials
// by a polynomial beside the unit's; K and V of a tile by one warp cost a sixth on pages of 16
// keys (a box a page and 64 channels).
#pragma once

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <type_traits>

#include "cp_host.h"
#include "cp_items.cuh"
#include "cp_latent.h"
#include "cp_ptx.cuh"
#include "cp_rows.cuh"

namespace cp {
namespace pairs {

constexpr int kThreads = 384;
constexpr int kKeys = 128;                // keys of a tile
constexpr uint32_t kUnit = 128 * 128;     // bytes of 128 rows x 64 channels
constexpr int kMaxUnits = 12;
constexpr int kMaxTiles = 8;              // that have barriers
constexpr uint32_t kSmem = 232448;        // of a CTA, at most
constexpr float kRescaleLog2 = 8.0f;
// Register split: compiled at kRegsLaunch a thread (the most 384 threads may have); the
// control warpgroup drops to kRegsControl and hands the rest to the softmax warpgroups.
constexpr int kRegsLaunch = 168;
constexpr int kRegsControl = 72;
constexpr int kRegsSoftmax = 216;
static_assert(128 * kRegsControl + 256 * kRegsSoftmax == kThreads * kRegsLaunch, "the split must add up");

// What the scheduling warp hands to the others.
struct Item {
  int ntiles;               // tiles of keys; 0: rows that see none; -1: no more items
  int s, g;                 // sequence, KV head
  int row0, key0;           // the sequence's first row and (expanded) first key
  int rows, past;           // its rows, keys before its first row (negative: the first rows see none)
  int t0;                   // the item's first token
  int j_begin;              // its first key
  int all;                  // keys that every row of the item sees: [0, all)
  int q1;                   // with a second Q tile
  int whole;                // not split: finished here
  int part;                 // else: its part
};

struct __align__(16) Shared {
  uint64_t item_full[2], item_empty[2], q_full[2], q_empty, k_full[kMaxTiles], v_full[kMaxTiles], k_empty[kMaxTiles],
      v_empty[kMaxTiles], s_full[2], p_ready[2], o_done[2], o_free[2], guarded[2], joined, all_done;
  uint32_t tmem_base;
  int abort;
  Item item[2];
  int8_t parent[2][CP_TREE_MAX];            // a tree's, beside its item
  // Keys of a tile with a non-finite value, 16 each: of tiles that one Q tile looks through, that two do (of a lone
  // one's: that each warpgroup does).
  __align__(16) uint16_t bad[2][2][8];
};

template <int NQB, bool kLone>
struct Layout {
  static constexpr uint32_t q_bytes = (kLone ? 1u : 2u) * NQB * kUnit;
  // A lone Q tile's rows: maximum and sum in each warpgroup's keys, of two items in turn.
  static constexpr uint32_t ml_bytes = kLone ? 2 * 2 * 128 * sizeof(float2) : 0;
  static constexpr int fit = (int)((kSmem - q_bytes - ml_bytes - sizeof(Shared)) / kUnit);
  static constexpr int units = fit < kMaxUnits ? fit : kMaxUnits;
  static constexpr uint32_t ctl_off = q_bytes + units * kUnit;
  static constexpr uint32_t ml_off = ctl_off + (uint32_t)sizeof(Shared), alloc = ml_off + ml_bytes;
};

struct Maps {
  CUtensorMap q, k, kr, v;
};

// What a call is about: TreeWork (attn_tree.cu) and ExpandedWork (attn_expanded.cu) add
// kPaged, kExpanded, kLone, and their Cursor with what it asks.
struct WorkBase {
  int hq, hkv, group;
  int tok_tile;            // tokens of a Q tile
  float scale_log2;
  SeqRows rows;
  int total_rows;
  void* out;               // [total_rows, hq, channels]
  int* status;
  float* part_o;           // [parts][channels / 4][256 rows][4]
  float* part_ml;          // [parts][256 rows][2]: maximum (log2 domain), sum
  int page_size, num_pages, max_blocks, dn;
  const int* block_table;
  const int* parents;

  __device__ void report_empty(int lane) const {
    if (status && rows.rows_uniform <= 0)
      for (int s = lane; s < rows.num_seqs; s += 32)
        if (seq_rows(rows, s) < 1) atomicOr(status, CP_DEV_BOUNDS);
  }
};

template <typename T, int NQB, int NVB, typename Work>
__global__ void __launch_bounds__(kThreads, 1) pairs_kernel(const __grid_constant__ Maps tm, const Work wk) {
  using L = Layout<NQB, Work::kLone>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kIdescQK = make_idesc_f16(kBf16, 128, kKeys, false);
  constexpr uint32_t kIdescPV = make_idesc_f16(kBf16, 128, NVB * 64, true);
  // Tile t's barriers are t mod kTiles, and none may be a phase ahead of those who wait for it: t's K and V must not be
  // loaded before the product with V of tile t - kTiles.  They are loaded when units of tile t - kRing / kTile, or a later
  // one, are given back, of its K at the earliest; its scores were issued after the product of the tile before, or (a lone
  // Q tile) the one before that.
  constexpr int kRing = L::units, kTile = NQB + NVB, kTiles = kRing / kTile + (Work::kLone ? 2 : 1);
  static_assert(kTiles <= kMaxTiles, "barriers");
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sRing = smem + L::q_bytes;
  Shared* sh = reinterpret_cast<Shared*>(smem + L::ctl_off);

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  // ---- set-up that reads no global memory: it may overlap the previous kernel
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->item_full[i], 1);
      mbar_init(&sh->item_empty[i], 11);  // warps 0, 1, 3 and the eight of softmax
      mbar_init(&sh->q_full[i], 1);
      mbar_init(&sh->s_full[i], 1);
      mbar_init(&sh->p_ready[i], 128);
      mbar_init(&sh->o_done[i], 1);
      mbar_init(&sh->o_free[i], Work::kLone ? 256 : 128);
    }
    mbar_init(&sh->q_empty, 1);
    mbar_init(&sh->guarded[0], 128);
    mbar_init(&sh->guarded[1], Work::kLone ? 128 : 256);
    mbar_init(&sh->joined, 256);
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(&sh->k_full[i], 1);
      mbar_init(&sh->v_full[i], 1);
      mbar_init(&sh->k_empty[i], 1);
      mbar_init(&sh->v_empty[i], 1);
    }
    mbar_init(&sh->all_done, 1);
    sh->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm.q);
    tma_prefetch_desc(&tm.k);
    tma_prefetch_desc(&tm.v);
    if (Work::kExpanded) tma_prefetch_desc(&tm.kr);
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  volatile int* abort_flag = &sh->abort;
  auto wait = [&](uint64_t* b, uint32_t parity) { return warp_wait(b, parity, abort_flag, wk.status); };
  // Item k of this CTA, as every role takes it: false when there are no more.
  auto give = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->item_empty[k & 1]);
  };
  auto take = [&](int k, Item& x) {
    if (!wait(&sh->item_full[k & 1], (k >> 1) & 1)) return false;
    x = sh->item[k & 1];
    return x.ntiles >= 0;
  };
  pdl_wait_and_launch_dependents();  // everything below, and the combine kernel's lookups, read what earlier kernels wrote

  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
  if (warp == 2) {
    // ================================================================ scheduling
    typename Work::Cursor cur(wk);
    int k = 0;
    bool ok = true;
    Item x;
    while (ok) {
      const bool more = cur.next(wk, x);
      if (k >= 2) ok = wait(&sh->item_empty[k & 1], ((k >> 1) & 1) ^ 1);
      if (!ok) break;
      if (!Work::kExpanded && more) {
        load_parents(wk.parents + x.row0, x.rows, wk.status, sh->parent[k & 1]);
        __syncwarp();
      }
      if (lane == 0) {
        if (!more) x.ntiles = -1;
        sh->item[k & 1] = x;
        mbar_arrive(&sh->item_full[k & 1]);
      }
      if (!more) break;
      ++k;
    }
    __syncwarp();
    if (blockIdx.x == 0) wk.report_empty(lane);
  } else if (warp != 1) {
    // ================================================================ producers: warp 0 of Q and K, warp 3 of V
    const bool of_v = warp == 3;
    const int n = of_v ? NVB : NQB;
    const int ps = Work::kPaged ? wk.page_size : kKeys, lps = 31 - __clz(ps);
    const int npg = kKeys / ps;  // boxes of a unit
    int t = 0;                   // tiles issued so far
    int queries = 0;             // items whose queries were loaded
    uint32_t last_q1 = 0;        // loads of Q tile 1
    bool ok = true;
    Item x;
    for (int k = 0; ok && take(k, x); ++k) {
      give(k);
      if (x.ntiles == 0) continue;
      if (!of_v) {
        if (queries > 0) ok = wait(&sh->q_empty, (queries - 1) & 1);
        if (!ok) break;
        const bool q1 = x.q1;
        if (lane == 0)
          for (int w = 0; w < (q1 ? 2 : 1); ++w) {
            mbar_arrive_expect_tx(&sh->q_full[w], NQB * wk.tok_tile * wk.group * 128);
            for (int b = 0; b < NQB; ++b)
              tma_load_3d(smem + (w * NQB + b) * kUnit, &tm.q, &sh->q_full[w], b * 64, x.g * wk.group,
                          x.row0 + x.t0 + w * wk.tok_tile);
          }
        __syncwarp();
        ++queries;
        last_q1 += q1;
      }
      for (int i = 0; ok && i < x.ntiles; ++i) {
        const int j0 = x.j_begin + i * kKeys;
        int plane = x.s * wk.hkv + x.g, off = j0;
        if (Work::kPaged) {
          const int key = j0 + (lane % npg) * ps, blk = key >> lps;
          plane = wk.num_pages * wk.hkv;  // out of range: zeros
          if (key < x.past + x.rows) {
            const int page = blk < wk.max_blocks ? wk.block_table[(long long)x.s * wk.max_blocks + blk] : -1;
            if (page >= 0 && page < wk.num_pages) plane = page * wk.hkv + x.g;
            else if (wk.status && lane < npg) atomicOr(wk.status, CP_DEV_BOUNDS);
          }
          off = 0;
        }
        // The units before them in the ring, the last of which is given back last (but for a lone Q tile: K before the V of
        // the tile before it).
        const int u = t * kTile + (of_v ? NQB : 0), old = u + n - 1 - kRing;
        if (old >= 0) {
          const int to = old / kTile;
          ok = wait(old % kTile < NQB ? &sh->k_empty[to % kTiles] : &sh->v_empty[to % kTiles], (to / kTiles) & 1);
          if (Work::kLone && ok && to > 0 && old % kTile < n - 1 && old % kTile < NQB)
            ok = wait(&sh->v_empty[(to - 1) % kTiles], ((to - 1) / kTiles) & 1);
          if (!ok) break;
        }
        uint64_t* bar = of_v ? &sh->v_full[t % kTiles] : &sh->k_full[t % kTiles];
        ++t;
        if (lane == 0) mbar_arrive_expect_tx(bar, n * kUnit);
        __syncwarp();
        for (int idx = lane; idx < npg * n; idx += 32) {  // npg divides 32: the page stays the lane's
          const int e = idx / npg;
          uint8_t* dst = sRing + (u + e) % kRing * kUnit + (idx % npg) * ps * 128;
          if (!Work::kExpanded) tma_load_3d(dst, of_v ? &tm.v : &tm.k, bar, e * 64, off, plane);
          else if (of_v) tma_load_3d(dst, &tm.v, bar, e * 64, x.g, x.key0 + j0);
          else if (e * 64 < wk.dn) tma_load_3d(dst, &tm.k, bar, e * 64, x.g, x.key0 + j0);
          else tma_load_3d(dst, &tm.kr, bar, 0, x.key0 + j0, 0);
        }
      }
    }
    // Every copy has landed before shared memory is released, also after an abort.
    volatile int zero = 0;
    if (queries > 0) mbar_wait(&sh->q_full[0], (queries - 1) & 1, &zero, wk.status);
    if (last_q1 > 0) mbar_wait(&sh->q_full[1], (last_q1 - 1) & 1, &zero, wk.status);
    for (int i = max(0, t - kTiles); i < t; ++i)
      mbar_wait(of_v ? &sh->v_full[i % kTiles] : &sh->k_full[i % kTiles], (i / kTiles) & 1, &zero, wk.status);
    __syncwarp();
  } else {
    // ================================================================ MMA issuer
    // The whole warp runs the loop, converged; one elected lane issues.  What addresses come from is broadcast.
    auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    const uint32_t tm0 = (uint32_t)uniform((int)tmem);
    constexpr uint32_t kStep = kUnit >> 4;  // of a descriptor: 16 bytes
    const uint64_t q_desc = make_sdesc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t v_desc = make_sdesc_sw128(smem_u32(sRing), kUnit, 1024);
    const uint32_t q_lo = (uint32_t)q_desc, k_hi = (uint32_t)(q_desc >> 32);  // Q and K differ in their addresses only
    const uint32_t k_lo = (uint32_t)make_sdesc_sw128(smem_u32(sRing), 16, 1024);
    const uint32_t v_lo = (uint32_t)v_desc, v_hi = (uint32_t)(v_desc >> 32);
    auto wrap = [](int slot) { return slot >= kRing ? slot - kRing : slot; };
    // Of the tile whose K, whose V comes next: its barriers, their parity; the ring's slot of its first unit.
    int kt = 0, vt = 0, k_slot = 0, v_slot = NQB % kRing;
    uint32_t k_turn = 0, v_turn = 0;
    uint32_t pq = 0, pp = 0, po = 0, begun = 0;  // bit w: parity of the Q tiles and P tiles taken, of the outputs begun; any begun
    bool ok = true;
    auto scores = [&](int w) {  // S_w = Q_w K^T
      const uint32_t d = tm0 + 256u * w, q = q_lo + (Work::kLone ? 0u : (uint32_t)w * (NQB * kStep));
#pragma unroll
      for (int b = 0; b < NQB; ++b) {
        const uint32_t kd = k_lo + (uint32_t)wrap(k_slot + b) * kStep;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_ss_lo(d, q + b * kStep + 2 * kk, k_hi, kd + 2 * kk, k_hi, kIdescQK, b | kk);
      }
      mma_commit_elect(&sh->s_full[w]);
    };
    auto output = [&](int w, uint32_t acc) {  // O_w += P_w V
      const uint32_t s = tm0 + 256u * w, o = s + 128u;
      if (NVB == 1 || v_slot + 1 < kRing) {
        const uint32_t v = v_lo + (uint32_t)v_slot * kStep;
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk) mma_ts_lo(o, s + kk * 8, v + 128 * kk, v_hi, kIdescPV, kk ? 1u : acc);
      } else {  // the ring's end lies between V's units: 64 channels at a time
        constexpr uint32_t kIdescHalf = make_idesc_f16(kBf16, 128, 64, true);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          mma_ts_lo(o, s + kk * 8, v_lo + (uint32_t)v_slot * kStep + 128 * kk, v_hi, kIdescHalf, kk ? 1u : acc);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk) mma_ts_lo(o + 64u, s + kk * 8, v_lo + 128 * kk, v_hi, kIdescHalf, kk ? 1u : acc);
      }
    };
    auto k_done = [&] {
      mma_commit_elect(&sh->k_empty[kt]);
      k_slot = wrap(k_slot + kTile);
      if (++kt == kTiles) {
        kt = 0;
        k_turn ^= 1u;
      }
    };
    auto v_done = [&] {
      mma_commit_elect(&sh->v_empty[vt]);
      v_slot = wrap(v_slot + kTile);
      if (++vt == kTiles) {
        vt = 0;
        v_turn ^= 1u;
      }
    };
    // A lone Q tile: tile i of keys is warpgroup i mod 2's.
    auto next_scores = [&](int w) {
      if (!wait(&sh->k_full[kt], k_turn)) return false;
      tc_fence_after();
      scores(w);
      k_done();
      return true;
    };
    for (int k = 0; Work::kLone && ok; ++k) {
      if (!wait(&sh->item_full[k & 1], (k >> 1) & 1)) break;
      const int ntiles = uniform(sh->item[k & 1].ntiles);
      give(k);
      if (ntiles < 0) break;
      if (ntiles == 0) continue;
      ok = wait(&sh->q_full[0], pq);
      pq ^= 1u;
      for (int i = 0; ok && i < 2 && i < ntiles; ++i) ok = next_scores(i);
      if (ntiles <= 2) mma_commit_elect(&sh->q_empty);
      for (int i = 0; ok && i < ntiles; ++i) {
        const int w = i & 1;
        ok = wait(&sh->v_full[vt], v_turn);
        if (ok && i < 2 && ((begun >> w) & 1)) ok = wait(&sh->o_free[w], ((po >> w) & 1) ^ 1);
        ok = ok && wait(&sh->p_ready[w], (pp >> w) & 1);
        if (!ok) break;
        pp ^= 1u << w;
        tc_fence_after();
        output(w, i >= 2);
        if (i + 2 >= ntiles) mma_commit_elect(&sh->o_done[w]);
        v_done();
        if (i < 2) {
          po ^= 1u << w;
          begun |= 1u << w;
        }
        if (i + 2 < ntiles) ok = next_scores(w);
        if (i + 3 == ntiles) mma_commit_elect(&sh->q_empty);  // the item's last scores are issued
      }
    }
    for (int k = 0; !Work::kLone && ok; ++k) {
      if (!wait(&sh->item_full[k & 1], (k >> 1) & 1)) break;
      const int ntiles = uniform(sh->item[k & 1].ntiles);
      const int nw = uniform(sh->item[k & 1].q1) + 1;
      give(k);
      if (ntiles < 0) break;
      if (ntiles == 0) continue;
      for (int w = 0; ok && w < nw; ++w) {
        ok = wait(&sh->q_full[w], (pq >> w) & 1);
        pq ^= 1u << w;
        if (ok && w == 0) ok = wait(&sh->k_full[kt], k_turn);
        if (!ok) break;
        tc_fence_after();
        scores(w);
      }
      if (!ok) break;
      k_done();
      if (ntiles == 1) mma_commit_elect(&sh->q_empty);
      for (int i = 0; ok && i < ntiles; ++i) {
        const bool more = i + 1 < ntiles;
        for (int w = 0; w < nw; ++w) {
          // P last: it comes last, and what follows it is what the softmax waits for.
          if (w == 0) ok = wait(&sh->v_full[vt], v_turn);
          if (ok && i == 0 && ((begun >> w) & 1)) ok = wait(&sh->o_free[w], ((po >> w) & 1) ^ 1);  // the output before has left TMEM
          ok = ok && wait(&sh->p_ready[w], (pp >> w) & 1);
          pp ^= 1u << w;
          if (!ok) break;
          tc_fence_after();
          output(w, i > 0);
          if (!more) mma_commit_elect(&sh->o_done[w]);
          if (w == nw - 1) v_done();
          if (more) {
            if (w == 0) {
              ok = wait(&sh->k_full[kt], k_turn);
              if (!ok) break;
              tc_fence_after();
            }
            scores(w);
          }
          if (i == 0) {
            po ^= 1u << w;
            begun |= 1u << w;
          }
        }
        if (!ok) break;
        if (more) k_done();
        if (i + 2 == ntiles) mma_commit_elect(&sh->q_empty);  // the item's last scores are issued
      }
    }
    mma_commit_elect(&sh->all_done);
    volatile int zero = 0;  // wait even after an abort: MMAs may still be in flight
    mbar_wait(&sh->all_done, 0, &zero, wk.status);
    __syncwarp();
  }
  } else {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
  // ================================================================ softmax, output
  const int w = (warp - 4) >> 2;            // Q tile of this warpgroup
  const int quarter = warp & 3;             // TMEM lanes [32 * quarter, + 32)
  const int m = quarter * 32 + lane;        // this thread's row of its Q tile
  const uint32_t s_col = tmem + ((uint32_t)(quarter * 32) << 16) + 256u * w, o_col = s_col + 128u;
  const int mtok = m / wk.group, mhead = m % wk.group;
  int t = 0;            // the CTA's tiles so far
  int ns = 0;           // score tiles of this warpgroup so far
  int no[2] = {0, 0};   // items with an output w so far
  Item x;
  int guards[2] = {0, 0};  // tiles looked through for hidden values so far, by one Q tile, by two
  for (int k = 0;; ++k) {
    // After a wait that gave up, an item's walk goes on without waiting, and its output is not written.
    bool alive = take(k, x) && !*abort_flag;
    if (!__all_sync(0xffffffffu, alive)) break;
    const bool q1 = x.q1;
    const int tok = x.t0 + (Work::kLone ? 0 : w * wk.tok_tile) + mtok;  // this row's token
    const bool row_ok = mtok < wk.tok_tile && tok < x.rows;
    const int n = x.past + x.rows;
    uint64_t see_lo = 0, see_hi = 0;  // a tree's row: the call's rows that it sees
    if (!Work::kExpanded) ancestors(sh->parent[k & 1], row_ok ? tok : -1, see_lo, see_hi);
    give(k);
    if (!Work::kLone && w == 1 && !q1) {
      t += x.ntiles;
      continue;
    }
    const int seen = Work::kExpanded ? x.past + tok + 1 : x.past;  // keys [0, seen) are seen, and in a tree the row's ancestors
    float m_run = -INFINITY, l_run = 0.f;
    constexpr int kTurns = Work::kLone ? 2 : 1;
    for (int i = Work::kLone ? w : 0; i < x.ntiles; i += kTurns, ++ns) {
      alive = alive && wait(&sh->s_full[w], ns & 1);
      tc_fence_after();
      uint32_t sv[128];
      tmem_ld32(s_col + 0, &sv[0]);
      tmem_ld32(s_col + 32, &sv[32]);
      tmem_ld32(s_col + 64, &sv[64]);
      tmem_ld32(s_col + 96, &sv[96]);
      tmem_wait_ld();
      const int j0 = x.j_begin + i * kKeys;
      const bool guard = j0 + kKeys > x.all;  // keys that some row of the item does not see
      uint64_t vis[2] = {~0ull, ~0ull};
      if (guard) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = seen - j0 - 64 * h;  // columns [0, c) of this half are seen
          vis[h] = !row_ok ? 0 : c >= 64 ? ~0ull : c > 0 ? (1ull << c) - 1 : 0;
          if (!Work::kExpanded && row_ok && c < 64) vis[h] |= bits_from(see_lo, see_hi, -c);
        }
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (!((vis[c >> 6] >> (c & 63)) & 1)) sv[c] = __float_as_uint(-INFINITY);
      }
      float mx;
      {
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
          m4[0] = fmax3(m4[0], __uint_as_float(sv[c + 0]), __uint_as_float(sv[c + 1]));
          m4[1] = fmax3(m4[1], __uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3]));
          m4[2] = fmax3(m4[2], __uint_as_float(sv[c + 4]), __uint_as_float(sv[c + 5]));
          m4[3] = fmax3(m4[3], __uint_as_float(sv[c + 6]), __uint_as_float(sv[c + 7]));
        }
        mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
      }
      const float mx2 = mx * wk.scale_log2;  // scale > 0, so the max commutes with it
      const bool grow = mx2 > m_run + kRescaleLog2 || (m_run == -INFINITY && mx2 != -INFINITY);
      const float m_new = grow ? mx2 : m_run;
      const float alpha = grow ? (m_run == -INFINITY ? 0.f : ex2_approx(m_run - m_new)) : 1.f;
      const float neg_m = m_new == -INFINITY ? 0.f : -m_new;
      float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 64; ++c) {
        float x0 = __uint_as_float(sv[2 * c]), x1 = __uint_as_float(sv[2 * c + 1]);
        ffma2(x0, x1, wk.scale_log2, neg_m);
        x0 = ex2_approx(x0);
        x1 = ex2_approx(x1);
        fadd2(ps[2 * (c & 1)], ps[2 * (c & 1) + 1], x0, x1);
        sv[c] = pack2<T>(x0, x1);  // V's type: see above
      }
      l_run = l_run * alpha + ((ps[0] + ps[1]) + (ps[2] + ps[3]));
      m_run = m_new;
      tmem_st32(s_col + 0, &sv[0]);
      tmem_st32(s_col + 32, &sv[32]);
      // O holds P V of the earlier tiles (complete: see the ordering note above).
      if (i >= kTurns && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
        for (int c = 0; c < 2 * NVB; ++c) {
          uint32_t ov[32];
          tmem_ld32(o_col + 32 * c, ov);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
          tmem_st32(o_col + 32 * c, ov);
        }
      }
      if (guard) {
        // ---- values that must not meet a weight of 0: the threads of the item's Q tiles share the tile's keys
        const int tile = t + i;
        alive = alive && wait(&sh->v_full[tile % kTiles], (tile / kTiles) & 1);
        const int v_unit = tile * kTile + NQB;
        const int per = !Work::kLone && q1 ? 2 : 1, me = (Work::kLone ? 0 : w * 128) + m;   // threads of a key; this one
        const int key = me / per, part = me % per;
        const bool gone = j0 + key >= n;
        bool bad = gone;
        constexpr int kChunks = NVB * 8;  // 16-byte chunks of a key
        auto chunk = [&](int c) {         // in an order that spreads the threads over the banks
          c = (c + key) % kChunks;
          return reinterpret_cast<uint4*>(sRing + ((v_unit + c / 8) % kRing) * kUnit + key * 128 + (c & 7) * 16);
        };
        if (!bad && j0 + key >= x.all)
          for (int c = part; c < kChunks; c += per) bad = bad || nonfinite8<T>(*chunk(c));
        if (per == 2) bad = __shfl_xor_sync(0xffffffffu, bad, 1) || bad;
        if (bad)
          for (int c = part; c < kChunks; c += per) *chunk(c) = make_uint4(0, 0, 0, 0);
        const int by = Work::kLone ? w : (int)q1, turn = by ? guards[1]++ : guards[0]++;
        uint16_t* found = sh->bad[by][turn & 1];
        const uint32_t bits = __ballot_sync(0xffffffffu, bad && !gone);
        if (lane == 0) {
          if (per == 2) {
            found[me / 32] = (uint16_t)even_bits(bits);
          } else {
            found[2 * quarter] = (uint16_t)bits;
            found[2 * quarter + 1] = (uint16_t)(bits >> 16);
          }
        }
        fence_proxy_async_smem();  // the tensor cores read V through the async proxy
        mbar_arrive(&sh->guarded[by]);
        alive = alive && wait(&sh->guarded[by], turn & 1);
        const uint4 y = *reinterpret_cast<const uint4*>(found);
        if ((vis[0] & (y.x | (uint64_t)y.y << 32)) | (vis[1] & (y.z | (uint64_t)y.w << 32))) l_run = __int_as_float(0x7fffffff);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sh->p_ready[w]);
    }

    t += x.ntiles;

    // ---- output
    if constexpr (Work::kLone) {
      // The two warpgroups' parts, of even and odd tiles, are joined: each writes half of the channels.
      float k0 = 0.f, k1 = 0.f;  // factors of the parts
      if (x.ntiles > 0) {
        for (int v = 0; v < 2 && v < x.ntiles; ++v) alive = alive && wait(&sh->o_done[v], (v ? no[1] : no[0]) & 1);
        float2* ml = reinterpret_cast<float2*>(smem + L::ml_off) + (no[0] & 1) * 256 + m;
        ml[w * 128] = make_float2(m_run, l_run);
        mbar_arrive(&sh->joined);
        alive = alive && wait(&sh->joined, no[0] & 1);
        tc_fence_after();
        const float2 a = ml[0], b = ml[128];
        const float top = fmaxf(a.x, b.x), z = top == -INFINITY ? 0.f : top;
        k0 = ex2_approx(a.x - z);
        k1 = ex2_approx(b.x - z);
        const float l = a.y * k0 + b.y * k1;
        if (x.whole) {
          const float inv = l == 0.f ? 0.f : 1.f / l;  // a NaN stays
          k0 *= inv;
          k1 *= inv;
        } else if (w == 0 && row_ok && alive) {
          *reinterpret_cast<float2*>(wk.part_ml + ((long long)x.part * 256 + m) * 2) = make_float2(top, l);
        }
      }
      const uint32_t o0 = o_col - 256u * w;
      const long long row = (long long)(x.row0 + tok) * wk.hq + x.g * wk.group + mhead;
      uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(wk.out) + row * (NVB * 64));
      float4* part = reinterpret_cast<float4*>(wk.part_o) + ((long long)x.part * (NVB * 16)) * 256 + m;
#pragma unroll
      for (int j = 0; j < NVB; ++j) {
        const int c = w * NVB + j;
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0.f;
        if (x.ntiles > 0) {
          uint32_t ov[32];
          tmem_ld32(o0 + 32 * c, ov);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(ov[e]) * k0;
          if (x.ntiles > 1) {
            tmem_ld32(o0 + 256 + 32 * c, ov);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = fmaf(__uint_as_float(ov[e]), k1, o[e]);
          }
        }
        if (!Work::kExpanded && !x.whole) {
          if (row_ok && alive) {
#pragma unroll
            for (int e = 0; e < 8; ++e) part[(8 * c + e) * 256] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        } else if (row_ok && alive) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            out[4 * c + e] = make_uint4(pack2<T>(o[8 * e], o[8 * e + 1]), pack2<T>(o[8 * e + 2], o[8 * e + 3]),
                                        pack2<T>(o[8 * e + 4], o[8 * e + 5]), pack2<T>(o[8 * e + 6], o[8 * e + 7]));
        }
      }
      tc_fence_before();
      for (int v = 0; v < 2 && v < x.ntiles; ++v) {
        ++no[v];
        mbar_arrive(&sh->o_free[v]);
      }
      if (!alive) *abort_flag = 1;
      continue;
    }
    if (x.ntiles > 0) alive = alive && wait(&sh->o_done[w], no[0] & 1);
    tc_fence_after();
    const bool write = row_ok && alive;
    const long long row = (long long)(x.row0 + tok) * wk.hq + x.g * wk.group + mhead;
    if (x.whole) {
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;  // a NaN stays
      uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(wk.out) + row * (NVB * 64));
#pragma unroll
      for (int c = 0; c < 2 * NVB; ++c) {
        uint32_t ov[32];
        if (x.ntiles > 0) {
          tmem_ld32(o_col + 32 * c, ov);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = 0;
        }
        if (write) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t y[4];
#pragma unroll
            for (int f = 0; f < 4; ++f)
              y[f] = pack2<T>(__uint_as_float(ov[8 * e + 2 * f]) * inv, __uint_as_float(ov[8 * e + 2 * f + 1]) * inv);
            out[4 * c + e] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
      }
    } else {
      // [16-byte piece][256 rows]: a warp's stores are 512 bytes in a row.
      if (write) *reinterpret_cast<float2*>(wk.part_ml + ((long long)x.part * 256 + w * 128 + m) * 2) = make_float2(m_run, l_run);
      float4* part = reinterpret_cast<float4*>(wk.part_o) + ((long long)x.part * (NVB * 16)) * 256 + w * 128 + m;
#pragma unroll
      for (int c = 0; c < 2 * NVB; ++c) {
        uint32_t ov[32];
        tmem_ld32(o_col + 32 * c, ov);
        tmem_wait_ld();
        if (write) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            part[(8 * c + e) * 256] = make_float4(__uint_as_float(ov[4 * e]), __uint_as_float(ov[4 * e + 1]),
                                                  __uint_as_float(ov[4 * e + 2]), __uint_as_float(ov[4 * e + 3]));
        }
      }
    }
    if (x.ntiles > 0) {
      ++no[0];
      tc_fence_before();
      mbar_arrive(&sh->o_free[w]);
    }
    if (!alive) *abort_flag = 1;
  }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int NQB, int NVB, typename Work>
cudaError_t launch(const Maps& tm, const Work& wk, int ctas, cudaStream_t st) {
  using L = Layout<NQB, Work::kLone>;
  static_assert(L::units >= NQB + NVB + (Work::kLone ? NQB : 0), "a tile fits the ring; of a lone Q tile's, the next one's K too");
  const auto kernel = pairs_kernel<T, NQB, NVB, Work>;
  // Raise the dynamic shared-memory limit once per device, so later calls --
  // including ones being captured into a CUDA graph -- only launch.
  static std::atomic<uint64_t> ready_mask{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  constexpr uint32_t smem = L::alloc > 120u * 1024u ? L::alloc : 120u * 1024u;  // one CTA an SM: each takes all of TMEM
  if (!(ready_mask.load(std::memory_order_acquire) & bit)) {
    // The register split is only sound at the per-thread count it was sized
    // for: refuse to launch a build that came out at another count.
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kRegsLaunch || fa.sharedSizeBytes != 0) return cudaErrorInvalidDeviceFunction;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    ready_mask.fetch_or(bit, std::memory_order_release);
  }
  return launch_pdl(kernel, dim3(ctas), dim3(kThreads), smem, st, tm, wk);
}

}  // namespace pairs
}  // namespace cp
