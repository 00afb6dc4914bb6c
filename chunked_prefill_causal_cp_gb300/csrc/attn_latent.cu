// attn_latent.cu -- attention over a latent cache in the absorbed form, on the sm_103a
// tensor cores (TMA, tcgen05, TMEM), the keys shared out over the SMs.
//
// A position's row of up to 512 + 64 channels is the key and, without its last
// channels, the value of every head: it is read once for a tile of 64 (row, head)
// pairs, and the path is bound by the cache's bytes until the pairs are many.  64 keys
// are 72 KB, of which shared memory holds two beside 64 pairs' queries (two and a half
// beside 32 pairs', of which it keeps no more than there are), and an output of
// 512 channels leaves TMEM room for 64 pairs only if the channels lie over its lanes.
// Hence
//   S[64 pairs x 64 keys] = Q K^T  A = Q, B = K, both K-major, an M of 64, whose rows lie
//                                  in the lower 16 lanes of each quarter of TMEM
//   P -> shared memory             [pair][64 keys] in 16 bits, one swizzled 128-byte row
//   O^T[128 channels x pairs] += V^T P^T   A = V as it lies (MN-major), B = P (K-major),
//                                  a block of TMEM columns for each 128 channels
// An MMA takes as long as its operands take out of shared memory (128 bytes a clock: 32
// clocks of the first kind, 48 of the second with 64 pairs), 1920 clocks a tile of 512 +
// 64 channels, beside 576 for the copies into it.
// Four threads share a pair's scores of a tile, 16 keys each.  A raised maximum scales a
// column of O^T, which all lanes hold: the threads vote each tile (a barrier that ORs),
// and only when some score passes its pair's maximum by more than 2^8 do they exchange
// maxima, leave the factors in shared memory and pass over O.
//
// One persistent CTA an SM, 384 threads: warps 0 and 3 TMA producers, warp 1 TMEM and MMA
// issue, warp 2 scheduling (finds the CTA's items, two ahead), warps 4-11 softmax and output.
// A tile's blocks of 64 channels land, and are given back, in two groups -- the first
// 256 channels and the rotated part, and the next 256 -- through a ring of slots of a
// group each.  The first half of a tile's scores fills the wait for the softmax of the one
// before, and the first half of its values is refilled while the second is still
// multiplied.  Which comes first goes by what is there: a product whose weights are ready
// before the next keys (it frees the slots that these wait for: decode 189 -> 173 us), the
// next tile's scores between the halves of a product (the softmax waits for them: chunk
// 247 -> 235 us).
//
// What a row does not see: its scores become -inf by a 64-bit mask of the tile's
// columns (a tree's row: its ancestors, 128 bits found by walking the parents once).
// Its weight 0 must not meet a NaN or an infinity in V: slots past the sequence are
// overwritten with zeros in shared memory, and so are rows of the call's own
// positions that hold a non-finite value; the pairs that see such a one become NaN by
// their sum.
//
// Weights are rounded to the layer's type for O^T += V^T P^T (nothing else is, before the output: scores, maxima, sums,
// O and parts are fp32, and the sums are of the weights before their rounding).  Both operands of that MMA are of one
// type, and V is multiplied as it lies in the cache: weights in 32 bits would want V widened in shared memory, twice the
// bytes of what bounds a tile, and weights in two 16-bit halves a second product with V.  What it costs against 64
// bits, relative, root mean square, with the output's own rounding (alone 1.7e-3 in bf16, 2.1e-4 in fp16): 1.8e-3 to
// 2.4e-3 and 2.5e-4.  (Weights of one size have errors of the output's own, independent ones: a factor of up to sqrt(2).)
// A weight below fp16's normal range is off by up to 2^-25 of the largest.
//
// The CTAs share the tiles of keys of all tiles of pairs out evenly (cp_latent.h); a tile of
// pairs that several of them have leaves unnormalised fp32 parts and (maximum, sum) in
// the workspace, which the combine kernel merges in order.
//
// Measured (bf16, 512 + 64 channels): 32 rows of 32 heads over 12000 to 40000 keys 165 us,
// 5.8 TB/s, 0.85 of a copy's rate, bound by the cache's bytes; 2 x 45 rows of 64 heads over
// 8000 to 16000 keys 199 us, 760 TFLOP/s, bound by the chain of a tile -- softmax 1200
// clocks, half of V's product 400, half of the next scores 600, 100 to 300 from each to the
// next -- of which the tensor cores work two thirds; one row of 32 heads over 1025 keys 11
// us, latency.  Slower were exponentials by a polynomial beside the unit's (and they lose a NaN),
// and weights handed over in two halves.
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
namespace {

constexpr int kThreads = 384;
constexpr int kTile = 64;                 // keys of a tile
constexpr uint32_t kBlock = kTile * 128;  // bytes of 64 keys x 64 channels
constexpr int kMaxSlots = 8;
constexpr int kPairs = 64;                // (row, head) pairs of a tile
constexpr uint32_t kSmem = 232448;        // of a CTA, at most
constexpr float kRescaleLog2 = 8.0f;
constexpr int kCombineThreads = 1024 * kSms;

// A (tile of pairs, split) of the call: what the scheduling warp hands to the others.
struct Item {
  int ntiles;               // tiles of keys; -1: no more items
  int s;                    // sequence
  int row0, rows, past;     // its first row, rows, positions before them
  int first, pairs;         // first (row, head) pair of the sequence, pairs of the tile
  int j_begin, j_end;       // keys
  int whole;                // not split: finished here
  int part;                 // else: its part
};

struct __align__(16) Shared {
  uint64_t item_full[2], item_empty[2], q_full, q_empty, full[kMaxSlots], empty[kMaxSlots], s_full[2],
      p_ready, pv_done, o_free, all_done;
  uint32_t tmem_base;
  int abort;
  Item item[2];
  uint32_t bad[2][8];         // keys of the tile with a non-finite value, 8 a warp
  int8_t parent[2][CP_TREE_MAX];  // a tree's, beside its item
  union __align__(16) {
    struct {                  // during an item's walk
      float alpha[kPairs];    // the factor of a pair's column for its raised maximum
      float top[4][kPairs];   // maximum of a pair's 16 scores of this tile, by part
    };
    struct {                  // after it
      float inv[kPairs];      // 1 / sum of a pair
      float sum[4][kPairs];   // of a pair's weights, by part
    };
  };
};
static_assert(offsetof(Shared, alpha) % 16 == 0, "the factors are read four at a time");

// Shared memory: Q, slots of a group of blocks each, slots of a tile's rotated part, P, Shared.
struct Layout {
  uint32_t q_block, slot_bytes, slots_off, rot_off, p_off, ctl_off, alloc;
  int nqb, nvb;             // blocks of 64 channels: of a row, of its value
  int ngroups, slots, rot_slots;
};

Layout layout_of(int dqk, int dv, int q_rows) {
  Layout l;
  l.nqb = (dqk + 63) / 64;
  l.nvb = dv / 64;
  l.ngroups = (l.nvb + 3) / 4;
  // Rows of Q and P: those that the MMAs' N has.  An MMA's 64 rows of Q go on into what lies
  // behind them, of no pair.
  const uint32_t rows = (uint32_t)(q_rows + 15) / 16 * 16;
  l.q_block = rows * 128;
  l.slot_bytes = (uint32_t)std::min(l.nvb, 4) * kBlock;
  l.slots_off = l.nqb * l.q_block;
  // A group's slot is free again after the output of the tile that had it, and with it the
  // rotated parts of all tiles before: as many as begin in the other slots.
  for (l.slots = kMaxSlots;; --l.slots) {
    l.rot_slots = l.nqb > l.nvb ? (l.slots + l.ngroups - 1) / l.ngroups : 0;
    l.rot_off = l.slots_off + l.slots * l.slot_bytes;
    l.p_off = l.rot_off + l.rot_slots * kBlock;
    l.ctl_off = l.p_off + l.q_block;
    l.alloc = l.ctl_off + (uint32_t)sizeof(Shared);
    if (l.alloc <= kSmem) return l;
  }
}

// The call's units: tiles of pairs of each sequence.
struct Work : RowsAttnArgs {
  // A sequence within the call's bounds: its rows, positions before them, first row.
  __device__ __forceinline__ bool bounds(int s, int& r, int& p, int& row0) const {
    return seq_bounds(rows, past, total_rows, max_ctx, s, r, p, row0) && !(parents && r > CP_TREE_MAX);
  }
  __device__ __forceinline__ int pair_tiles(int r) const { return (r * hq - 1) / kPairs + 1; }
  __device__ __forceinline__ int units(int s, bool report) const {
    int r, p, row0;
    if (bounds(s, r, p, row0)) return pair_tiles(r);
    if (report && status && r >= 1) atomicOr(status, CP_DEV_BOUNDS);
    return 0;
  }
  __device__ __forceinline__ int key_tiles(int s) const { return (past[s] + seq_rows(rows, s) - 1) / kTile + 1; }
  __device__ __forceinline__ bool make(int s, int u, int k0, int n, Item& x) const {
    if (!bounds(s, x.rows, x.past, x.row0)) return false;
    x.s = s;
    x.first = u * kPairs;
    x.pairs = min(kPairs, x.rows * hq - x.first);
    x.j_begin = k0 * kTile;
    const int seen = x.past + (x.first + x.pairs - 1) / hq + 1;  // by the tile's last row
    x.ntiles = seen > x.j_begin ? min((seen - x.j_begin - 1) / kTile + 1, n) : 0;
    x.j_end = min(seen, x.j_begin + x.ntiles * kTile);
    return x.ntiles > 0;
  }
};

// A place in the ring of slots, and how often it came round (divisions by the number of slots, made where the MMAs
// are issued, took longer than the MMAs).
struct Ring {
  int slot = 0;
  uint32_t turn = 0;  // parity
  __device__ __forceinline__ void advance(int slots) {
    if (++slot == slots) {
      slot = 0;
      turn ^= 1u;
    }
  }
};

// Barriers of the eight softmax warps, one of which also ORs a predicate.
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool softmax_any(bool x) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r)
               : "r"((uint32_t)x)
               : "memory");
  return r != 0;
}

template <typename T, bool kPaged>
__global__ void __launch_bounds__(kThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const Work a, const Layout L) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sSlot = smem + L.slots_off;
  uint8_t* sP = smem + L.p_off;
  Shared* sh = reinterpret_cast<Shared*>(smem + L.ctl_off);

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  // ---- set-up that reads no global memory: it may overlap the previous kernel
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->item_full[i], 1);
      mbar_init(&sh->item_empty[i], 11);  // warps 0, 1, 3 and the eight of softmax
      mbar_init(&sh->s_full[i], 1);
    }
    mbar_init(&sh->q_full, 1);
    mbar_init(&sh->q_empty, 1);
    for (int i = 0; i < L.slots; ++i) {
      mbar_init(&sh->full[i], 2);  // both producers
      mbar_init(&sh->empty[i], 1);
    }
    mbar_init(&sh->p_ready, 256);
    mbar_init(&sh->pv_done, 1);
    mbar_init(&sh->o_free, 256);
    mbar_init(&sh->all_done, 1);
    sh->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
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
  auto wait = [&](uint64_t* b, uint32_t parity) { return warp_wait(b, parity, abort_flag, a.status); };
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

  if (warp == 2) {
    // ================================================================ scheduling
    ShareCursor<Work> cur(a);
    Item x;
    for (int k = 0;; ++k) {
      const bool more = cur.next(a, x);
      if (k >= 2 && !wait(&sh->item_empty[k & 1], ((k >> 1) & 1) ^ 1)) break;
      if (a.parents && more) {
        load_parents(a.parents + x.row0, x.rows, a.status, sh->parent[k & 1]);
        __syncwarp();
      }
      if (lane == 0) {
        if (!more) x.ntiles = -1;
        sh->item[k & 1] = x;
        mbar_arrive(&sh->item_full[k & 1]);
      }
      if (!more) break;
    }
    __syncwarp();
    if (blockIdx.x == 0 && a.status && a.rows.rows_uniform <= 0)
      for (int s = lane; s < a.rows.num_seqs; s += 32)
        if (seq_rows(a.rows, s) < 1) atomicOr(a.status, CP_DEV_BOUNDS);
  } else if (warp != 1 && warp < 4) {
    // ================================================================ producers: each of every other block
    const int odd = warp == 3;
    const int ps = kPaged ? min(a.cache.page_size, kTile) : kTile, lps = kPaged ? 31 - __clz(a.cache.page_size) : 0;
    const int npg = kTile / ps;  // boxes of a block
    Ring ring, rot;
    int groups = 0, queries = 0;    // groups, items' queries issued so far
    uint32_t begun = 0, phase = 0;  // bit of a slot: any copy begun, parity of their number
    bool ok = true;
    Item x;
    for (int k = 0; ok && take(k, x); ++k) {
      give(k);
      if (k > 0 && !odd) ok = wait(&sh->q_empty, (k - 1) & 1);
      if (!ok) break;
      if (lane == 0 && !odd) {
        mbar_arrive_expect_tx(&sh->q_full, L.nqb * a.q_rows * 128);
        for (int b = 0; b < L.nqb; ++b) tma_load_3d(smem + b * L.q_block, &tm_q, &sh->q_full, b * 64, x.row0 * a.hq + x.first, 0);
      }
      __syncwarp();
      queries = odd ? 0 : k + 1;
      for (int i = 0; ok && i < x.ntiles; ++i, rot.advance(L.rot_slots)) {
        const int j0 = x.j_begin + i * kTile;
        // This lane's boxes: idx = lane, lane + 32, ...: page idx % npg of block idx / npg.
        int plane = x.s, off = j0;
        if (kPaged) {
          const int key = j0 + (lane % npg) * ps, blk = key >> lps;
          plane = a.cache.num_pages;  // out of range: zeros
          if (key < x.j_end) {
            const int page = blk < a.cache.max_blocks ? a.cache.block_table[(long long)x.s * a.cache.max_blocks + blk] : -1;
            if (page >= 0 && page < a.cache.num_pages) plane = page;
            else if (a.status && lane < npg) atomicOr(a.status, CP_DEV_BOUNDS);
          }
          off = key & (a.cache.page_size - 1);
        }
        for (int j = 0; ok && j < L.ngroups; ++j, ++groups, ring.advance(L.slots)) {
          const int st = ring.slot, nv = min(4, L.nvb - 4 * j);
          if (groups >= L.slots) ok = wait(&sh->empty[st], ring.turn ^ 1);
          if (!ok) break;
          // The first group also has the rotated part, behind its values.
          const int nb = (nv + (j == 0 ? L.nqb - L.nvb : 0) + 1 - odd) / 2;  // this warp's blocks
          begun |= 1u << st;
          phase ^= 1u << st;
          if (lane == 0) mbar_arrive_expect_tx(&sh->full[st], nb * kBlock);
          __syncwarp();
          for (int idx = lane; idx < npg * nb; idx += 32) {  // npg divides 32: the page stays the lane's
            const int e = 2 * (idx / npg) + odd;
            uint8_t* to = e < nv ? sSlot + st * L.slot_bytes + e * kBlock : smem + L.rot_off + rot.slot * kBlock;
            tma_load_3d(to + (idx % npg) * ps * 128, &tm_k, &sh->full[st], (e < nv ? 4 * j + e : L.nvb) * 64, off, plane);
          }
        }
      }
    }
    // Every copy has landed before shared memory is released, also after an abort.
    volatile int zero = 0;
    if (queries > 0) mbar_wait(&sh->q_full, (queries - 1) & 1, &zero, a.status);
    for (int i = 0; i < kMaxSlots; ++i)
      if ((begun >> i) & 1) mbar_wait(&sh->full[i], ((phase >> i) & 1) ^ 1, &zero, a.status);
    __syncwarp();
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    // The whole warp runs the loop, converged; one elected lane issues.  What addresses come from is broadcast.
    auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    const uint32_t tm = (uint32_t)uniform((int)tmem);
    constexpr uint32_t kKStep = kBlock >> 4;  // of a descriptor: 16 bytes
    const uint32_t q_step = L.q_block >> 4;
    constexpr uint32_t kIdescQK = make_idesc_f16(kBf16, 64, kTile, false);
    const uint64_t q_desc = make_sdesc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t v_desc = make_sdesc_sw128(smem_u32(sSlot), kBlock, 1024);
    const uint32_t q_lo = (uint32_t)q_desc, k_hi = (uint32_t)(q_desc >> 32);  // Q, K and P differ in their addresses only
    const uint32_t k_lo = (uint32_t)make_sdesc_sw128(smem_u32(sSlot), 16, 1024);
    const uint32_t r_lo = (uint32_t)make_sdesc_sw128(smem_u32(smem) + L.rot_off, 16, 1024);
    const uint32_t p_lo = (uint32_t)make_sdesc_sw128(smem_u32(sP), 16, 1024);
    const uint32_t v_lo = (uint32_t)v_desc, v_hi = (uint32_t)(v_desc >> 32), slot_step = L.slot_bytes >> 4;
    const int nvb = L.nvb;
    const bool rotated = L.nqb > nvb;
    // Scores over n blocks from Q at q, K at kd on; `acc`: added to what is there.
    auto scores = [&](int n, uint32_t d, uint32_t q, uint32_t kd, uint32_t acc) {
#pragma unroll 1
      for (int b = 0; b < n; ++b, q += q_step, kd += kKStep, acc = 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) mma_ss_lo(d, q + 2 * e, k_hi, kd + 2 * e, k_hi, kIdescQK, e ? 1u : acc);
    };
    // Output of n x 128 channels from V at vd on into the columns at d.
    auto output = [&](int n, uint32_t d, uint32_t vd, uint32_t idesc, uint32_t acc) {
#pragma unroll 1
      for (int b = 0; b < n; ++b, d += kPairs, vd += 2 * kKStep)
#pragma unroll
        for (int e = 0; e < 4; ++e) mma_ss_lo(d, vd + 128 * e, v_hi, p_lo + 2 * e, k_hi, idesc, e ? 1u : acc);
    };
    const int v0 = min(nvb, 4), v1 = nvb - v0;  // blocks of values in the two groups
    Ring qk, pv, rot;      // of the group (tile) whose scores, whose output is issued next
    uint32_t s_buf = 0;    // S of the next scores
    uint32_t p_phase = 0;  // parity of the next P
    bool ok = true;
    auto ready = [&](uint64_t* b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test(b, parity)); };
    // Group j of the next tile's scores.
    auto group = [&](int j) {
      if (!wait(&sh->full[qk.slot], qk.turn)) return false;
      tc_fence_after();
      const uint32_t d = tm + 64u * s_buf, kd = k_lo + qk.slot * slot_step;
      if (j == 0) {
        scores(v0, d, q_lo, kd, 0);
        if (rotated) scores(1, d, q_lo + nvb * q_step, r_lo + rot.slot * kKStep, 1);
        rot.advance(L.rot_slots);
      } else {
        scores(v1, d, q_lo + 4 * q_step, kd, 1);
      }
      qk.advance(L.slots);
      if (j + 1 == L.ngroups) {
        mma_commit_elect(&sh->s_full[s_buf]);
        s_buf ^= 1u;
      }
      return true;
    };
    // With room for two tiles only the second group comes after the output that gave it its slot.
    const int early = L.slots > 2 * L.ngroups ? L.ngroups : 1;
    for (int k = 0; ok; ++k) {
      if (!wait(&sh->item_full[k & 1], (k >> 1) & 1)) break;
      const int ntiles = uniform(sh->item[k & 1].ntiles);
      const uint32_t idesc_pv = make_idesc_f16(kBf16, 128, (uniform(sh->item[k & 1].pairs) + 15) & ~15, false) | (1u << 15);  // A MN-major
      give(k);
      if (ntiles < 0) break;
      ok = wait(&sh->q_full, k & 1);
      for (int j = 0; ok && j < L.ngroups; ++j) ok = group(j);
      if (ntiles == 1) mma_commit_elect(&sh->q_empty);
      for (int i = 0; ok && i < ntiles; ++i) {
        const bool more = i + 1 < ntiles;
        int next = 0;  // group of the next tile's scores
        for (; ok && more && next < early; ++next) {
          // Where the keys are late and P is there, P's product comes first: it frees the slots that the next keys wait for.
          bool product = false;
          for (int n = 0; n < 4096 && !product && !ready(&sh->full[qk.slot], qk.turn); ++n) product = ready(&sh->p_ready, p_phase);
          if (product) break;
          ok = group(next);
        }
        ok = ok && wait(&sh->p_ready, p_phase);
        if (ok && i == 0 && k > 0) ok = wait(&sh->o_free, (k - 1) & 1);  // the item before has left O
        if (!ok) break;
        p_phase ^= 1u;
        tc_fence_after();
        const uint32_t d = tm + 128u, acc = i > 0;
        output(v0 / 2, d, v_lo + pv.slot * slot_step, idesc_pv, acc);
        mma_commit_elect(&sh->empty[pv.slot]);
        pv.advance(L.slots);
        if (v1 > 0) {
          // The next tile's scores, where their keys are there: the softmax waits for them.
          if (more && next + 1 == L.ngroups && ready(&sh->full[qk.slot], qk.turn)) ok = group(next++);
          output(v1 / 2, d + 2 * kPairs, v_lo + pv.slot * slot_step, idesc_pv, acc);
          mma_commit_elect(&sh->empty[pv.slot]);
          pv.advance(L.slots);
        }
        mma_commit_elect(&sh->pv_done);
        for (; ok && more && next < L.ngroups; ++next) ok = group(next);
        if (i + 2 == ntiles) mma_commit_elect(&sh->q_empty);  // the item's last scores are issued
      }
    }
    mma_commit_elect(&sh->all_done);
    volatile int zero = 0;  // wait even after an abort: MMAs may still be in flight
    mbar_wait(&sh->all_done, 0, &zero, a.status);
    __syncwarp();
  } else {
    // ================================================================ softmax, output
    const int half = (warp - 4) >> 2, quarter = warp & 3;
    const int me = half * 128 + quarter * 32 + lane;
    // This thread's pair of a tile, with keys [16 part, + 16) of each 64.
    const int m = quarter * 16 + (lane & 15), part = 2 * half + (lane >> 4);
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const int nob = L.nvb / 2;
    int gt = 0;
    Ring ring;
    Item x;
    for (int k = 0;; ++k) {
      // After a wait that gave up, an item's walk goes on without waiting, so that its barriers stay whole; its output is
      // not written, and the warps leave together.
      bool alive = take(k, x);
      if (softmax_any(!alive)) break;
      const int n = x.past + x.rows;  // positions written, this call's rows among them
      const bool row_ok = m < x.pairs, active = quarter * 16 < x.pairs;
      const int tok = (x.first + m) / a.hq;
      uint64_t see_lo = 0, see_hi = 0;  // a tree's row: the call's rows that it sees
      if (a.parents) ancestors(sh->parent[k & 1], row_ok ? tok : -1, see_lo, see_hi);
      give(k);
      float m_run = -INFINITY, l_run = 0.f;
      for (int i = 0; i < x.ntiles; ++i, ++gt) {
        const int j0 = x.j_begin + i * kTile;
        alive = alive && wait(&sh->s_full[gt & 1], (gt >> 1) & 1);
        tc_fence_after();
        uint32_t sv[16];
        uint64_t vis = 0;
        float mx = -INFINITY;
        if (active) {
          tmem_ld16x2<16>(tmem + lane_off + 64u * (gt & 1) + 32u * half, sv);
          tmem_wait_ld();
          const int c = x.past - j0 + (a.parents ? 0 : tok + 1);  // columns [0, c) are seen
          vis = c >= 64 || !row_ok ? ~0ull : c > 0 ? (1ull << c) - 1 : 0;
          if (a.parents && c < 64) vis |= bits_from(see_lo, see_hi, -c);
          const uint32_t v = (uint32_t)(vis >> (16 * part)) & 0xffffu;
          if (v != 0xffffu) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (!((v >> e) & 1)) sv[e] = __float_as_uint(-INFINITY);
          }
          float m4[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            m4[0] = fmax3(m4[0], __uint_as_float(sv[e + 0]), __uint_as_float(sv[e + 1]));
            m4[1] = fmax3(m4[1], __uint_as_float(sv[e + 2]), __uint_as_float(sv[e + 3]));
          }
          mx = fmaxf(m4[0], m4[1]);
        }
        mx *= a.scale_log2;  // scale > 0: it commutes
        const bool raise = softmax_any(row_ok && (mx > m_run + kRescaleLog2 || (m_run == -INFINITY && mx != -INFINITY)));
        if (raise) {
          // A pair's four threads agree on its maximum; one that no score passes by the threshold stays.
          if (row_ok) sh->top[part][m] = mx;
          softmax_sync();
          float alpha = 1.f;
          if (row_ok) {
            mx = fmaxf(fmaxf(sh->top[0][m], sh->top[1][m]), fmaxf(sh->top[2][m], sh->top[3][m]));
            if (mx > m_run + kRescaleLog2 || (m_run == -INFINITY && mx != -INFINITY)) {
              if (m_run != -INFINITY) alpha = ex2_approx(m_run - mx);  // else nothing but zeros so far
              m_run = mx;
              l_run *= alpha;
            }
            if (part == 0) sh->alpha[m] = alpha;
          }
          if (i > 0) {
            softmax_sync();
            alive = alive && wait(&sh->pv_done, (gt - 1) & 1);
            tc_fence_after();
            for (int b = half; b < nob; b += 2)
              for (int c = 0; c < x.pairs; c += 32) {
                const uint32_t col = tmem + lane_off + 128u + (uint32_t)(b * kPairs + c);
                uint32_t ov[32];
                tmem_ld32(col, ov);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                  const float4 f = *reinterpret_cast<const float4*>(&sh->alpha[c + e]);  // of no pair: of no matter
                  ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f.x);
                  ov[e + 1] = __float_as_uint(__uint_as_float(ov[e + 1]) * f.y);
                  ov[e + 2] = __float_as_uint(__uint_as_float(ov[e + 2]) * f.z);
                  ov[e + 3] = __float_as_uint(__uint_as_float(ov[e + 3]) * f.w);
                }
                tmem_st32(col, ov);
              }
            tmem_wait_st();
          }
          softmax_sync();  // maxima and factors are read
        }
        if (active) {
          const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
          float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float x0 = __uint_as_float(sv[2 * c]), x1 = __uint_as_float(sv[2 * c + 1]);
            ffma2(x0, x1, a.scale_log2, neg_m);
            x0 = ex2_approx(x0);
            x1 = ex2_approx(x1);
            fadd2(ps[2 * (c & 1)], ps[2 * (c & 1) + 1], x0, x1);
            sv[c] = pack2<T>(x0, x1);  // V's type: see above
          }
          l_run += (ps[0] + ps[1]) + (ps[2] + ps[3]);
        }
        // The product of the tile before is complete: P may be overwritten.
        if (i > 0) alive = alive && wait(&sh->pv_done, (gt - 1) & 1);
        if (active) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            *reinterpret_cast<uint4*>(sP + m * 128 + (((2 * part + c) ^ (m & 7)) * 16)) =
                make_uint4(sv[4 * c], sv[4 * c + 1], sv[4 * c + 2], sv[4 * c + 3]);
        }
        // ---- values that must not meet a weight of 0
        if (j0 + kTile > n || (x.rows > 1 && j0 + kTile > x.past)) {
          Ring at = ring;
          for (int j = 0; j < L.ngroups; ++j, at.advance(L.slots)) alive = alive && wait(&sh->full[at.slot], at.turn);
          const int st = ring.slot, st1 = st + 1 == L.slots ? 0 : st + 1;  // of the tile's groups
          const int key = me >> 2, own = me & 3;   // four threads a key
          const int chunks = L.nvb * 8;            // its 16-byte chunks, in an order that spreads the threads over the banks
          auto chunk = [&](int c) {
            const int d = (c + key) & 7;
            return reinterpret_cast<uint4*>(sSlot + (c < 32 ? st : st1) * L.slot_bytes + ((c >> 3) & 3) * kBlock + key * 128 + d * 16);
          };
          const bool gone = j0 + key >= n;
          bool bad = gone;
          if (!bad && x.rows > 1 && j0 + key >= x.past)
            for (int c = own; c < chunks; c += 4) bad = bad || nonfinite8<T>(*chunk(c));
          bad = __shfl_xor_sync(0xffffffffu, bad, 1) || bad;
          bad = __shfl_xor_sync(0xffffffffu, bad, 2) || bad;
          if (bad)
            for (int c = own; c < chunks; c += 4) *chunk(c) = make_uint4(0, 0, 0, 0);
          const uint32_t four = __ballot_sync(0xffffffffu, bad && !gone);  // four bits a key
          if (lane == 0) sh->bad[gt & 1][warp - 4] = four;
          softmax_sync();
          uint64_t any = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t y = sh->bad[gt & 1][e];
            if (y)
              for (int c = 0; c < 8; ++c)
                if ((y >> (4 * c)) & 1) any |= 1ull << (8 * e + c);
          }
          if (any & vis) l_run = __int_as_float(0x7fffffff);
        }
        fence_proxy_async_smem();  // the tensor cores read P and V through the async proxy
        tc_fence_before();
        mbar_arrive(&sh->p_ready);
        for (int j = 0; j < L.ngroups; ++j) ring.advance(L.slots);
      }

      // ---- output: a lane holds a channel of each 128, its pairs in the columns
      alive = alive && wait(&sh->pv_done, (gt - 1) & 1);
      tc_fence_after();
      if (row_ok) sh->sum[part][m] = l_run;
      if (softmax_any(!alive)) break;
      if (part == 0 && row_ok) {
        const float l = (l_run + sh->sum[1][m]) + (sh->sum[2][m] + sh->sum[3][m]);
        sh->inv[m] = l == 0.f ? 0.f : 1.f / l;  // a NaN stays
        if (!x.whole) *reinterpret_cast<float2*>(a.part_ml + ((long long)x.part * kPairs + m) * 2) = make_float2(m_run, l);
      }
      softmax_sync();
      if (x.whole) {
        for (int b = half; b < nob; b += 2) {
          T* out = static_cast<T*>(a.out) + ((long long)x.row0 * a.hq + x.first) * a.dv + b * 128 + quarter * 32 + lane;
          for (int c = 0; c < x.pairs; c += 32) {
            uint32_t ov[32];
            tmem_ld32(tmem + lane_off + 128u + (uint32_t)(b * kPairs + c), ov);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e, out += a.dv) {
              if (c + e >= x.pairs) break;
              const float y[2] = {__uint_as_float(ov[e]) * sh->inv[c + e], 0.f};
              *reinterpret_cast<uint16_t*>(out) = (uint16_t)Pack<T>::store(y);
            }
          }
        }
      } else {
        for (int b = half; b < nob; b += 2) {
          float* to = a.part_o + (long long)x.part * kPairs * a.dv + b * 128 + quarter * 32 + lane;
          for (int c = 0; c < x.pairs; c += 32) {
            uint32_t ov[32];
            tmem_ld32(tmem + lane_off + 128u + (uint32_t)(b * kPairs + c), ov);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e, to += a.dv) *to = __uint_as_float(ov[e]);  // up to 31 pairs more than there are: room that nobody reads
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&sh->o_free);
      softmax_sync();  // the sums are read: their place is free
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// A pair's parts are merged in slices -- part i in slice i mod `slices`, a slice's in order
// -- and the slices in order.  dv threads a pair, or a quarter of its channels (`cut` is 4):
// four or sixteen slices, a thread four channels.
template <typename T>
__global__ void __launch_bounds__(512) latent_combine_kernel(const Work a, const int per, const int cut, const int groups,
                                                              const bool by_share) {
  __shared__ float4 so[512];
  __shared__ float2 sml[16];
  pdl_launch_dependents();
  pdl_look_ahead();
  const int nth = blockIdx.x / groups;
  const MergedUnit<Work> x(a, nth, by_share, a.ctas);
  int r = 0, p = 0, row0 = 0;
  const bool found = x.s >= 0 && a.bounds(x.s, r, p, row0);  // the same for all threads
  const int first = found ? x.unit * kPairs : 0, pairs = min(kPairs, r * a.hq - first);
  const int seen = found ? (p + (first + pairs - 1) / a.hq) / kTile + 1 : 1;  // tiles of keys, by the last row
  const UnitShares u(x.all, found ? x.first : 0, found ? x.n : 1, seen, a.ctas);
  pdl_wait();  // on all paths: this kernel's end stands for the parts' kernel's
  if (!found || u.whole || (by_share && u.from != nth)) return;
  const int slices = 4 * cut, c4 = a.dv / slices, mine = threadIdx.x / a.dv, slice = threadIdx.x % a.dv / c4;
  const int group = blockIdx.x % groups, d4 = group % cut * c4 + threadIdx.x % c4;
  for (int m0 = group / cut * per; m0 < pairs; m0 += groups / cut * per) {
    const int m = m0 + mine;
    const bool on = m < pairs;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float mx = -INFINITY, l = 0.f;
    if (on) {
      constexpr int kAhead = 4;
      for (int c0 = u.from + slice; c0 <= u.to; c0 += kAhead * slices) {
        float2 ml[kAhead];
        float4 x[kAhead];
        int n = 0;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int c = c0 + j * slices;
          if (c > u.to) break;
          const int row = u.part(c) * kPairs + m;
          ml[j] = __ldcg(reinterpret_cast<const float2*>(a.part_ml + row * 2));
          x[j] = __ldcg(reinterpret_cast<const float4*>(a.part_o) + row * (a.dv / 4) + d4);
          n = j + 1;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (j >= n) break;
          const float mn = fmaxf(mx, ml[j].x), z = mn == -INFINITY ? 0.f : mn;
          const float k0 = ex2_approx(mx - z), k1 = ex2_approx(ml[j].x - z);
          v.x = v.x * k0 + x[j].x * k1;
          v.y = v.y * k0 + x[j].y * k1;
          v.z = v.z * k0 + x[j].z * k1;
          v.w = v.w * k0 + x[j].w * k1;
          l = l * k0 + ml[j].y * k1;
          mx = mn;
        }
      }
    }
    so[threadIdx.x] = v;
    if (threadIdx.x % c4 == 0) sml[mine * slices + slice] = make_float2(mx, l);
    __syncthreads();
    if (slice == 0 && on) {
      mx = -INFINITY;
      for (int i = 0; i < slices; ++i) mx = fmaxf(mx, sml[mine * slices + i].x);
      const float z = mx == -INFINITY ? 0.f : mx;
      v = make_float4(0.f, 0.f, 0.f, 0.f);
      l = 0.f;
#pragma unroll 4
      for (int i = 0; i < slices; ++i) {
        const float4 x = so[threadIdx.x + i * c4];
        const float2 y = sml[mine * slices + i];
        const float k = ex2_approx(y.x - z);
        v.x = fmaf(k, x.x, v.x);
        v.y = fmaf(k, x.y, v.y);
        v.z = fmaf(k, x.z, v.z);
        v.w = fmaf(k, x.w, v.w);
        l = fmaf(k, y.y, l);
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float o[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
      uint2 b;
      b.x = Pack<T>::store(o);
      b.y = Pack<T>::store(o + 2);
      *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + ((long long)row0 * a.hq + first + m) * a.dv + 4 * d4) = b;
    }
    __syncthreads();  // the slices are read
  }
}

// The lengths of the sequences that the attention took.
__global__ void latent_commit_kernel(int* lens, const SeqRows rows, int total_rows, int max_ctx) {
  pdl_launch_dependents();
  pdl_wait();
  const int s = blockIdx.x * blockDim.x + threadIdx.x;
  int r, p, row0;
  if (s < rows.num_seqs && seq_bounds(rows, lens, total_rows, max_ctx, s, r, p, row0)) lens[s] = p + r;
}

template <typename T, bool kPaged>
cudaError_t launch_t(const RowsAttnArgs& args, int dtype, cudaStream_t st) {
  Work a;
  static_cast<RowsAttnArgs&>(a) = args;
  const Layout l = layout_of(a.dqk, a.dv, a.q_rows);
  CUtensorMap tq, tk;
  const CacheView& c = a.cache;
  const uint64_t slots = kPaged ? c.page_size : c.capacity, planes = kPaged ? c.num_pages : a.rows.num_seqs;
  if (!encode_3d(&tq, dtype, a.q, a.dqk, (uint64_t)a.total_rows * a.hq, 1, 64, a.q_rows, 1) ||
      !encode_3d(&tk, dtype, a.k, a.dqk, slots, planes, 64, kPaged ? std::min(c.page_size, kTile) : kTile, 1))
    return cudaErrorInvalidValue;
  // Raise the dynamic shared-memory limit once per device, so later calls --
  // including ones being captured into a CUDA graph -- only launch.
  static std::atomic<uint64_t> ready_mask{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready_mask.load(std::memory_order_acquire) & bit)) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, latent_kernel<T, kPaged>);
    if (e != cudaSuccess) return e;
    if (fa.sharedSizeBytes != 0) return cudaErrorInvalidDeviceFunction;  // the swizzled tiles start at its beginning
    e = cudaFuncSetAttribute(latent_kernel<T, kPaged>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    ready_mask.fetch_or(bit, std::memory_order_release);
  }
  const uint32_t smem = std::max(l.alloc, 120u * 1024u);  // one CTA an SM: each takes all of TMEM
  e = launch_pdl(latent_kernel<T, kPaged>, dim3(a.ctas), dim3(kThreads), smem, st, tq, tk, a, l);
  if (e != cudaSuccess || !a.split) return e;
  // With few pairs, of up to 152 parts each, their channels go to four CTAs (one row of 32 heads over 8000 keys
  // 22.8 -> 15.2 us in all; past one CTA an SM it was slower: two rows of 64 heads 19 -> 26 us); with many, a CTA
  // takes several pairs of its tile, which it has to find but once (64 rows of 64 heads 168 -> 147 us).
  const int cut = 4 * a.tiles * a.q_rows <= kSms ? 4 : 1, per = cut > 1 ? 1 : std::max(1, 256 / a.dv);
  const bool by_share = a.tiles > a.ctas;  // only units between two CTAs are merged
  const long long units = std::min<long long>(a.tiles, a.ctas), most = std::max<long long>(1, kCombineThreads / (per * a.dv * units));
  const int groups = cut * (int)std::min<long long>((a.q_rows + per - 1) / per, most);
  return launch_pdl(latent_combine_kernel<T>, dim3((unsigned)(units * groups)), dim3(per * a.dv), 0, st, a, per, cut, groups, by_share);
}

}  // namespace

RowsPlan latent_plan(int heads, int dv, bool uniform, long long num_seqs, long long total_rows, int max_ctx) {
  RowsPlan p{};
  const long long pairs = (uniform ? total_rows / num_seqs : total_rows) * heads;  // of a sequence, at most
  const int key_tiles = (max_ctx - 1) / kTile + 1;
  p.q_rows = (int)std::min<long long>(kPairs, pairs);
  p.tiles = uniform ? num_seqs * ((pairs + kPairs - 1) / kPairs) : tiles_at_most(pairs, num_seqs, kPairs);
  p.work = (double)p.tiles * (kStart + key_tiles);
  p.ctas = (int)std::min<double>(p.work, kSms);
  p.split = key_tiles > 1;
  p.part_floats = p.split ? 2LL * kSms * kPairs * dv : 0;
  p.bytes = p.split ? 2LL * kSms * kPairs * (dv + 2) * (long long)sizeof(float) : 0;
  return p;
}

cudaError_t launch_latent(const RowsAttnArgs& a, int dtype, cudaStream_t st) {
  const bool paged = a.cache.kind == CP_CACHE_PAGED;
  if (dtype == CP_BF16) return paged ? launch_t<__nv_bfloat16, true>(a, dtype, st) : launch_t<__nv_bfloat16, false>(a, dtype, st);
  return paged ? launch_t<__half, true>(a, dtype, st) : launch_t<__half, false>(a, dtype, st);
}

cudaError_t launch_latent_commit(int* lens, const SeqRows& rows, int total_rows, int max_ctx, cudaStream_t st) {
  const int block = 128;
  return launch_pdl(latent_commit_kernel, dim3((unsigned)((rows.num_seqs - 1) / block + 1)), dim3(block), 0, st, lens, rows,
                    total_rows, max_ctx);
}

}  // namespace cp
