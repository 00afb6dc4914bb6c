// attn_rows.cu -- attention of few rows (single tokens, short chunks, drafted
// trees) over a long K/V or latent cache, on the sm_103a tensor cores (TMA, tcgen05,
// TMEM), split along the keys.
//
// A KV head's cache is read once for a tile of up to 128 (row, head) pairs -- all
// heads' of a latent cache -- so the path is bound by the cache's bytes until the
// pairs are many.  A latent row is both key and value, 512 + 64 channels: a tile
// of 64 keys is 72 KB, of which shared memory holds two beside the queries, and the
// output of 64 pairs fills 256 columns of TMEM only if its 512 channels are spread
// over the lanes.  Hence the shape, the same for both kinds of cache:
//   S[pairs x 64 keys] = Q K^T     A = Q, B = K, both K-major: a thread owns a pair's
//                                  scores, and its softmax crosses no lanes
//   P -> shared memory             [pair][64 keys] in 16 bits, one swizzled 128-byte row
//   O^T[128 channels x pairs] += V^T P^T   A = V as it lies (MN-major), B = P (K-major),
//                                  a TMEM block for each 128 channels
// A raised maximum scales a column of O^T, which all lanes hold: the pairs' threads
// vote each tile (a barrier that ORs), and only when some maximum grew by more than
// 2^8 do they fetch the factors from shared memory and pass over O.
//
// Warp roles (256 threads): warp 0 TMA producer (a lane a box; paged caches: a box per
// page and 64 channels; page ids out of range read as zeros), warp 1 TMEM and MMA
// issue, warps 4-7 softmax and output.  The MMA warp issues S(i + 1) before P(i) is
// ready whenever tile i + 1 has landed, and S is double-buffered.
//
// What a row does not see: its scores become -inf by a 64-bit mask of the tile's
// columns (a tree's row: its ancestors, as 128 bits found by walking the parents
// once).  Its weight 0 must not meet a NaN or an infinity in V: slots past the
// sequence are overwritten with zeros in shared memory, and so are rows of the call's own
// keys that hold a non-finite value; the pairs that see such a key become NaN by
// their sum.
//
// Splits leave unnormalised fp32 parts and (maximum, sum) in the workspace, which the
// combine kernel merges in a fixed order.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <type_traits>

#include "cp_host.h"
#include "cp_latent.h"
#include "cp_ptx.cuh"
#include "cp_rows.cuh"

namespace cp {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;                 // keys of a tile
constexpr uint32_t kBlock = kTile * 128;  // bytes of 64 keys x 64 channels
constexpr int kMaxStages = 6;
constexpr uint32_t kSmemMax = 232448;     // bytes of shared memory of a CTA, at most,
constexpr uint32_t kSmemSM = 233472;      // and of an SM
// Register split: compiled at kRegsLaunch a thread (the most that two CTAs of 256 threads may have); the control
// warpgroup drops to kRegsControl and hands the rest to the softmax warpgroup.
constexpr int kRegsLaunch = 128;
constexpr int kRegsControl = 64;
constexpr int kRegsSoftmax = 192;
static_assert(128 * kRegsControl + 128 * kRegsSoftmax == kThreads * kRegsLaunch, "the split must add up");
constexpr float kRescaleLog2 = 8.0f;

// A (tile, split) of the call: what the scheduling warp hands to the others.
struct Item {
  int ntiles;               // 0: no more items
  int s, g;
  int row0, rows, past;     // of the sequence
  int first, pairs;         // first (row, head) pair of the sequence, pairs of the tile
  int j_begin, j_end;       // keys
  int whole;                // not split: finished here
  long long part;           // else: its part
};

struct __align__(16) RowsShared {
  uint64_t item_full[2], item_empty[2], q_full, q_empty, full[kMaxStages], empty[kMaxStages], s_full[2], p_ready, pv_done,
      o_free, all_done;
  uint32_t tmem_base;
  int abort;
  Item item[2];
  uint32_t bad[2][4];         // keys of the tile with a non-finite value, 16 a warp
  union __align__(16) {       // the factors are read four at a time
    int parent[CP_TREE_MAX];  // before an item's walk
    float alpha[128];         // during it: the factor of a pair's column for its raised maximum
    float inv[128];           // after it: 1 / sum of a pair
  };
};
static_assert(offsetof(RowsShared, alpha) % 16 == 0, "the factors are read four at a time");

// Shared memory: Q, stages, P, RowsShared.
struct RowsLayout {
  uint32_t q_bytes, stage_bytes, p_off, ctl_off, alloc;
  int nqb, nvb, vb0, nblk, stages;
};

__host__ __device__ inline RowsLayout rows_layout(int dqk, int dv, bool latent, int nr, int ctas) {
  RowsLayout l;
  l.nqb = (dqk + 63) / 64;
  l.nvb = dv / 64;
  l.vb0 = latent ? 0 : l.nqb;
  l.nblk = latent ? l.nqb : l.nqb + l.nvb;
  l.q_bytes = (uint32_t)l.nqb * nr * 128;
  l.stage_bytes = (uint32_t)l.nblk * kBlock;
  const uint32_t fixed = l.q_bytes + nr * 128 + (uint32_t)sizeof(RowsShared);
  int st = (int)((kSmemSM / ctas - 1024 - fixed) / l.stage_bytes);  // 1 KB of each CTA's is the system's
  l.stages = st > kMaxStages ? kMaxStages : st;
  l.p_off = l.q_bytes + l.stages * l.stage_bytes;
  l.ctl_off = l.p_off + nr * 128;
  l.alloc = l.ctl_off + (uint32_t)sizeof(RowsShared);
  return l;
}

// The tile that a CTA takes.
struct TileAt {
  int s, tile;        // sequence, tile within it
  int nt;             // tiles of the sequence
  long long slot;     // first part of the sequence
};

__device__ __forceinline__ int tiles_of(const RowsAttnArgs& a, int s) {
  const int r = seq_rows(a.rows, s);
  if (r < 1) return 0;
  const long long n = ((long long)r * a.group + a.tile_rows - 1) / a.tile_rows;
  return (int)(n <= a.tiles_bound ? n : a.tiles_bound + 1);  // more: offsets that are wrong
}

// Tile w of the call, over the sequences in order (a whole warp asks).
__device__ __forceinline__ bool find_tile(const RowsAttnArgs& a, int w, TileAt& t) {
  if (a.rows.rows_uniform > 0) {
    t.nt = tiles_of(a, 0);
    t.s = w / t.nt;
    t.tile = w % t.nt;
    t.slot = (long long)t.s * rows_slots(t.nt, a.max_splits);
    return t.s < a.rows.num_seqs;
  }
  const int lane = threadIdx.x & 31;
  long long slots = 0;
  for (int q0 = 0; q0 < a.rows.num_seqs; q0 += 32) {
    const int q = q0 + lane, n = q < a.rows.num_seqs ? tiles_of(a, q) : 0;
    const int m = n ? rows_slots(n, a.max_splits) : 0;
    long long inc = n, sl = m;  // inclusive prefix sums over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o), u = __shfl_up_sync(0xffffffffu, sl, o);
      if (lane >= o) {
        inc += v;
        sl += u;
      }
    }
    const long long tot = __shfl_sync(0xffffffffu, inc, 31);
    if (w < tot) {
      const int L = __ffs(__ballot_sync(0xffffffffu, inc > w)) - 1;
      t.s = q0 + L;
      t.nt = __shfl_sync(0xffffffffu, n, L);
      t.tile = (int)(w - __shfl_sync(0xffffffffu, inc - n, L));
      t.slot = slots + __shfl_sync(0xffffffffu, sl - m, L);
      return true;
    }
    w -= (int)tot;
    slots += __shfl_sync(0xffffffffu, sl, 31);
  }
  return false;
}

// A tile's place in the call: its sequence's bounds hold, its pairs and keys.
struct Place {
  int past, row0, rows, n;  // n: positions written, this call's rows among them
  int first, pairs;         // first pair of the sequence, pairs of the tile
  int keys;                 // that the tile's last row sees
  int splits, split_keys;
  int tile_splits;          // splits that hold keys of this tile
};

__device__ __forceinline__ bool place_of(const RowsAttnArgs& a, const TileAt& t, Place& p) {
  p.rows = seq_rows(a.rows, t.s);
  p.row0 = seq_row0(a.rows, t.s);
  p.past = a.past[t.s];
  if (p.past < 0 || (long long)p.past + p.rows > a.max_ctx || p.row0 < 0 || p.row0 > a.total_rows - p.rows ||
      (a.parents && p.rows > CP_TREE_MAX))
    return false;
  p.n = p.past + p.rows;
  p.first = t.tile * a.tile_rows;
  p.pairs = min(a.tile_rows, p.rows * a.group - p.first);
  p.keys = p.past + (p.first + p.pairs - 1) / a.group + 1;
  p.splits = rows_splits(p.n, t.nt);
  p.split_keys = rows_split_keys(p.n, p.splits);
  p.tile_splits = (p.keys - 1) / p.split_keys + 1;
  return p.splits == 1 || t.slot + (long long)t.nt * p.splits <= a.part_slots;
}

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

// Barrier of the four softmax warps that also ORs a predicate.
__device__ __forceinline__ bool softmax_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Item `cand` of the call, if there is one: candidates are (split, KV head, tile), tile fastest, so that the tiles
// that read the same keys run at the same time (a whole warp asks).
__device__ __forceinline__ bool item_of(const RowsAttnArgs& a, int cand, Item& x) {
  const int w = cand % a.tiles_bound, gs = cand / a.tiles_bound, g = gs % a.hkv, split = gs / a.hkv;
  TileAt at;
  Place p;
  if (!find_tile(a, w, at)) return false;
  if (!place_of(a, at, p)) {
    if (a.status && split == 0 && (threadIdx.x & 31) == 0) atomicOr(a.status, CP_DEV_BOUNDS);
    return false;
  }
  if (split >= p.tile_splits) return false;
  x.s = at.s;
  x.g = g;
  x.row0 = p.row0;
  x.rows = p.rows;
  x.past = p.past;
  x.first = p.first;
  x.pairs = p.pairs;
  x.j_begin = split * p.split_keys;
  x.j_end = (int)min((long long)p.keys, (long long)x.j_begin + p.split_keys);
  x.ntiles = (x.j_end - x.j_begin + kTile - 1) / kTile;
  x.whole = p.splits == 1;
  x.part = (at.slot + (long long)at.tile * p.splits + split) * a.hkv + g;
  return true;
}

template <typename T, bool kLatent, bool kPaged>
__global__ void __launch_bounds__(kThreads, 2)
    rows_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const RowsAttnArgs a, const RowsLayout L,
                     const uint32_t tmem_cols) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sStage = smem + L.q_bytes;
  uint8_t* sP = smem + L.p_off;
  RowsShared* sh = reinterpret_cast<RowsShared*>(smem + L.ctl_off);

  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // ---- set-up that reads no global memory: it may overlap the previous kernel
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->item_full[i], 1);
      mbar_init(&sh->item_empty[i], 6);
      mbar_init(&sh->s_full[i], 1);
    }
    mbar_init(&sh->q_full, 1);
    mbar_init(&sh->q_empty, 1);
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], 1);
    }
    mbar_init(&sh->p_ready, 128);
    mbar_init(&sh->pv_done, 1);
    mbar_init(&sh->o_free, 128);
    mbar_init(&sh->all_done, 1);
    sh->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    if (!kLatent) tma_prefetch_desc(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem_base, tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  volatile int* abort_flag = &sh->abort;
  auto wait = [&](uint64_t* b, uint32_t parity) { return warp_wait(b, parity, abort_flag, a.status); };
  // Item k of this CTA, as every role takes it: false when there are no more.
  auto take = [&](int k, Item& x) {
    if (!wait(&sh->item_full[k & 1], (k >> 1) & 1)) return false;
    x = sh->item[k & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->item_empty[k & 1]);
    return x.ntiles > 0;
  };
  pdl_wait();  // everything below reads what earlier kernels wrote

  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
  if (warp == 2) {
    // ================================================================ scheduling
    const int total = a.tiles_bound * a.hkv * a.max_splits;
    int k = 0;
    bool ok = true;
    for (long long cand = blockIdx.x; ok && cand < total; cand += gridDim.x) {
      Item x;
      if (!item_of(a, (int)cand, x)) continue;
      if (k >= 2) ok = wait(&sh->item_empty[k & 1], ((k >> 1) & 1) ^ 1);
      if (!ok) break;
      if (lane == 0) {
        sh->item[k & 1] = x;
        mbar_arrive(&sh->item_full[k & 1]);
      }
      ++k;
    }
    if (ok && k >= 2) ok = wait(&sh->item_empty[k & 1], ((k >> 1) & 1) ^ 1);
    if (ok && lane == 0) {
      sh->item[k & 1].ntiles = 0;
      mbar_arrive(&sh->item_full[k & 1]);
    }
    __syncwarp();
  } else if (warp == 3) {
    if (blockIdx.x == 0 && a.status && a.rows.rows_uniform <= 0)
      for (int s = lane; s < a.rows.num_seqs; s += 32)
        if (seq_rows(a.rows, s) < 1) atomicOr(a.status, CP_DEV_BOUNDS);
  } else if (warp == 0) {
    // ================================================================ producer
    const int ps = kPaged ? min(a.cache.page_size, kTile) : kTile, lps = kPaged ? 31 - __clz(a.cache.page_size) : 0;
    const int npg = kTile / ps;  // boxes of a block
    int gt = 0, queries = 0;     // tiles, items' queries issued so far
    bool ok = true;
    Item x;
    for (int k = 0; ok && take(k, x); ++k) {
      if (k > 0) ok = wait(&sh->q_empty, (k - 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sh->q_full, L.nqb * a.q_rows * 128);
        for (int b = 0; b < L.nqb; ++b) {
          uint8_t* dst = smem + b * a.nr * 128;
          if (kLatent) tma_load_3d(dst, &tm_q, &sh->q_full, b * 64, x.row0 * a.group + x.first, 0);
          else tma_load_3d(dst, &tm_q, &sh->q_full, b * 64, x.g * a.group, x.row0 + x.first / a.group);
        }
      }
      queries = k + 1;
      for (int i = 0; i < x.ntiles; ++i, ++gt) {
        const int st = gt % L.stages;
        const int j0 = x.j_begin + i * kTile;
        // This lane's boxes: idx = lane, lane + 32, ...: page idx % npg of block idx / npg.
        int plane = x.s * a.hkv + x.g, off = j0;
        if (kPaged) {
          const int key = j0 + (lane % npg) * ps, blk = key >> lps;
          plane = a.cache.num_pages * a.hkv;  // out of range: zeros
          if (key < x.j_end) {
            const int page = blk < a.cache.max_blocks ? a.cache.block_table[(long long)x.s * a.cache.max_blocks + blk] : -1;
            if (page >= 0 && page < a.cache.num_pages) plane = page * a.hkv + x.g;
            else if (a.status && lane < npg) atomicOr(a.status, CP_DEV_BOUNDS);
          }
          off = key & (a.cache.page_size - 1);
        }
        if (gt >= L.stages) ok = wait(&sh->empty[st], ((gt / L.stages) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&sh->full[st], L.stage_bytes);
        __syncwarp();
        for (int idx = lane; idx < npg * L.nblk; idx += 32) {  // npg divides 32: the page stays the lane's
          const int b = idx / npg;
          const bool v = !kLatent && b >= L.vb0;
          tma_load_3d(sStage + st * L.stage_bytes + b * kBlock + (idx % npg) * ps * 128, v ? &tm_v : &tm_k, &sh->full[st],
                      (v ? b - L.vb0 : b) * 64, off, plane);
        }
      }
    }
    // Every copy has landed before shared memory is released, also after an abort.
    volatile int zero = 0;
    if (queries > 0) mbar_wait(&sh->q_full, (queries - 1) & 1, &zero, a.status);
    for (int i = max(0, gt - L.stages); i < gt; ++i) mbar_wait(&sh->full[i % L.stages], (i / L.stages) & 1, &zero, a.status);
    __syncwarp();
  } else {
    // ================================================================ MMA issuer
    const uint32_t idesc_qk = make_idesc_f16(kBf16, 128, kTile, false);
    const uint64_t q_desc = make_sdesc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t k_desc = make_sdesc_sw128(smem_u32(sStage), 16, 1024);
    const uint64_t v_desc = make_sdesc_sw128(smem_u32(sStage) + L.vb0 * kBlock, kBlock, 1024);
    const uint64_t p_desc = make_sdesc_sw128(smem_u32(sP), 16, 1024);
    const uint32_t q_step = (uint32_t)a.nr * 128;
    const int nob = (L.nvb + 1) / 2;
    auto test = [&](uint64_t* b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test(b, parity)) != 0; };
    int g0 = 0;  // tiles of the items before
    bool ok = true;
    Item x;
    for (int k = 0; ok && take(k, x); ++k) {
      const uint32_t idesc_pv = make_idesc_f16(kBf16, 128, (x.pairs + 15) & ~15, false) | (1u << 15);  // A MN-major
      ok = wait(&sh->q_full, k & 1);
      int next = 0;  // tile whose scores are issued next
      for (int i = 0; ok && i < x.ntiles; ++i) {
        uint64_t t0 = 0;
        for (uint32_t it = 1;; ++it) {
          const int gn = g0 + next;
          if (next < x.ntiles && next <= i + 1 && test(&sh->full[gn % L.stages], (gn / L.stages) & 1)) {
            tc_fence_after();
            const uint64_t kd = k_desc + (((uint32_t)(gn % L.stages) * L.stage_bytes) >> 4);
            for (int b = 0; b < L.nqb; ++b)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ss_elect(tmem + 64u * (gn & 1), q_desc + ((b * q_step + kk * 32) >> 4),
                             kd + ((b * kBlock + kk * 32) >> 4), idesc_qk, (b | kk) != 0);
            mma_commit_elect(&sh->s_full[gn & 1]);
            if (++next == x.ntiles) mma_commit_elect(&sh->q_empty);
            continue;
          }
          if (next > i && test(&sh->p_ready, (g0 + i) & 1)) break;
          if ((it & 63u) == 0) {
            int stop = 0;
            if (lane == 0) {
              stop = *abort_flag;
              if (t0 == 0) t0 = global_timer_ns();
              if (!stop && global_timer_ns() - t0 > kWaitLimitNs) {
                *abort_flag = stop = 1;
                if (a.status) atomicOr(a.status, CP_DEV_TIMEOUT);
              }
            }
            if (__shfl_sync(0xffffffffu, stop, 0)) {
              ok = false;
              break;
            }
          }
        }
        if (ok && i == 0 && k > 0) ok = wait(&sh->o_free, (k - 1) & 1);  // the item before has left O
        if (!ok) break;
        tc_fence_after();
        const int st = (g0 + i) % L.stages;
        const uint64_t vd = v_desc + (((uint32_t)st * L.stage_bytes) >> 4);
        for (int b = 0; b < nob; ++b)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss_elect(tmem + 128u + (uint32_t)(b * a.nr), vd + ((b * 2 * kBlock + kk * 2048) >> 4), p_desc + ((kk * 32) >> 4),
                         idesc_pv, i > 0 || kk > 0);
        mma_commit_elect(&sh->empty[st]);
        mma_commit_elect(&sh->pv_done);
      }
      g0 += x.ntiles;
    }
    mma_commit_elect(&sh->all_done);
    volatile int zero = 0;  // wait even after an abort: MMAs may still be in flight
    mbar_wait(&sh->all_done, 0, &zero, a.status);
    __syncwarp();
  }
  } else {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
  // ================================================================ softmax, output
  const int quarter = warp - 4, m = quarter * 32 + lane;  // this thread's pair of the tile
  const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
  const int nob = (L.nvb + 1) / 2;
  int gt = 0;
  Item x;
  for (int k = 0;; ++k) {
    // After a wait that gave up, an item's walk goes on without waiting, so that its barriers stay whole; its output is
    // not written, and all four warps leave together.
    bool alive = take(k, x);
    if (softmax_any(!alive)) break;
    const int n = x.past + x.rows;  // positions written, this call's rows among them
    const bool row_ok = m < x.pairs, active = quarter * 32 < x.pairs;
    const int pair = x.first + m, tok = pair / a.group;
    uint64_t see_lo = 0, see_hi = 0;  // a tree's row: the call's rows that it sees
    if (a.parents) {
      if (m < x.rows) {
        int up = a.parents[x.row0 + m];
        if (up < -1 || up >= m) {
          up = -1;
          if (a.status) atomicOr(a.status, CP_DEV_BOUNDS);
        }
        sh->parent[m] = up;
      }
      softmax_sync();
      for (int j = row_ok ? tok : -1; j >= 0; j = sh->parent[j]) {
        if (j < 64) see_lo |= 1ull << j;
        else see_hi |= 1ull << (j - 64);
      }
      softmax_sync();  // the factors take the parents' place
    }
    float m_run = -INFINITY, l_run = 0.f;
    for (int i = 0; i < x.ntiles; ++i, ++gt) {
      const int j0 = x.j_begin + i * kTile;
      alive = alive && wait(&sh->s_full[gt & 1], (gt >> 1) & 1);
      tc_fence_after();
      uint32_t sv[64];
      uint64_t vis = 0;
      float alpha = 1.f;
      if (active) {
        tmem_ld32(tmem + lane_off + 64u * (gt & 1), &sv[0]);
        tmem_ld32(tmem + lane_off + 64u * (gt & 1) + 32u, &sv[32]);
        tmem_wait_ld();
        if (row_ok) {
          const int c = x.past - j0 + (a.parents ? 0 : tok + 1);  // columns [0, c) are seen
          vis = c >= 64 ? ~0ull : c > 0 ? (1ull << c) - 1 : 0;
          if (a.parents && c < 64) vis |= bits_from(see_lo, see_hi, -c);
        }
        if (vis != ~0ull) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!((vis >> c) & 1)) sv[c] = __float_as_uint(-INFINITY);
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 64; c += 8) {
          m4[0] = fmax3(m4[0], __uint_as_float(sv[c + 0]), __uint_as_float(sv[c + 1]));
          m4[1] = fmax3(m4[1], __uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3]));
          m4[2] = fmax3(m4[2], __uint_as_float(sv[c + 4]), __uint_as_float(sv[c + 5]));
          m4[3] = fmax3(m4[3], __uint_as_float(sv[c + 6]), __uint_as_float(sv[c + 7]));
        }
        const float mx2 = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]) * a.scale_log2;  // scale > 0: it commutes
        const bool first = m_run == -INFINITY;
        if (mx2 > m_run + kRescaleLog2 || (first && mx2 != -INFINITY)) {
          if (!first) alpha = ex2_approx(m_run - mx2);  // first: nothing but zeros so far
          m_run = mx2;
        }
        const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
        float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          float x0 = __uint_as_float(sv[2 * c]), x1 = __uint_as_float(sv[2 * c + 1]);
          ffma2(x0, x1, a.scale_log2, neg_m);
          x0 = ex2_approx(x0);
          x1 = ex2_approx(x1);
          fadd2(ps[2 * (c & 1)], ps[2 * (c & 1) + 1], x0, x1);
          sv[c] = pack2<T>(x0, x1);
        }
        l_run = l_run * alpha + ((ps[0] + ps[1]) + (ps[2] + ps[3]));
      }
      sh->alpha[m] = alpha;
      const bool scale = softmax_any(alpha != 1.f);
      // The product of the tile before is complete: P may be overwritten, O rescaled.
      if (i > 0) alive = alive && wait(&sh->pv_done, (gt - 1) & 1);
      if (scale) {
        if (i > 0) {
          tc_fence_after();
          for (int b = 0; b < nob; ++b)
            for (int c = 0; c < x.pairs; c += 32) {
              const uint32_t col = tmem + lane_off + 128u + (uint32_t)(b * a.nr + c);
              uint32_t ov[32];
              tmem_ld32(col, ov);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&sh->alpha[c + e]);
                ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f.x);
                ov[e + 1] = __float_as_uint(__uint_as_float(ov[e + 1]) * f.y);
                ov[e + 2] = __float_as_uint(__uint_as_float(ov[e + 2]) * f.z);
                ov[e + 3] = __float_as_uint(__uint_as_float(ov[e + 3]) * f.w);
              }
              tmem_st32(col, ov);
            }
          tmem_wait_st();
        }
        softmax_sync();  // the factors are read
      }
      if (active) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(sP + m * 128 + ((c ^ (m & 7)) * 16)) =
              make_uint4(sv[4 * c], sv[4 * c + 1], sv[4 * c + 2], sv[4 * c + 3]);
      }
      // ---- values that must not meet a weight of 0
      if (j0 + kTile > n || (x.rows > 1 && j0 + kTile > x.past)) {
        const int st = gt % L.stages;
        alive = alive && wait(&sh->full[st], (gt / L.stages) & 1);
        uint8_t* v = sStage + st * L.stage_bytes + L.vb0 * kBlock;
        const int key = m >> 1, half = m & 1;
        uint8_t* row = v + key * 128;
        bool bad = j0 + key >= n;
        const bool gone = bad;
        if (!bad && x.rows > 1 && j0 + key >= x.past) {
          for (int b = half; b < L.nvb; b += 2)
#pragma unroll
            for (int c = 0; c < 8; ++c)
              bad = bad || nonfinite8<T>(*reinterpret_cast<const uint4*>(row + b * kBlock + (((c + key + 4 * half) & 7) * 16)));
        }
        bad = __shfl_xor_sync(0xffffffffu, bad, 1) || bad;
        if (bad)
          for (int b = half; b < L.nvb; b += 2)
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<uint4*>(row + b * kBlock + (((c + key + 4 * half) & 7) * 16)) = make_uint4(0, 0, 0, 0);
        const uint32_t two = __ballot_sync(0xffffffffu, bad && !gone);  // two bits a key
        if (lane == 0) sh->bad[gt & 1][quarter] = two;
        softmax_sync();
        uint64_t any = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t y = sh->bad[gt & 1][e];
          if (y)
            for (int c = 0; c < 16; ++c)
              if ((y >> (2 * c)) & 1) any |= 1ull << (16 * e + c);
        }
        if (any & vis) l_run = __int_as_float(0x7fffffff);
      }
      fence_proxy_async_smem();  // the tensor cores read P and V through the async proxy
      tc_fence_before();
      mbar_arrive(&sh->p_ready);
    }

    // ---- output: a lane holds a channel of each 128, its pairs in the columns
    alive = alive && wait(&sh->pv_done, (gt - 1) & 1);
    tc_fence_after();
    sh->inv[m] = l_run == 0.f ? 0.f : 1.f / l_run;  // a NaN stays
    if (softmax_any(!alive)) break;
    if (x.whole) {
      const int span = kLatent ? 0 : a.hq - a.group;  // (row, head) rows between a token's last head and the next one's first
      for (int b = 0; b < nob; ++b) {
        const int ch = b * 128 + m;
        T* out = static_cast<T*>(a.out) + ((long long)(x.row0 + x.first / a.group) * a.hq + x.g * a.group + x.first % a.group) * a.dv + ch;
        int head = kLatent ? 0 : x.first % a.group;
        for (int c = 0; c < x.pairs; c += 32) {
          uint32_t ov[32];
          tmem_ld32(tmem + lane_off + 128u + (uint32_t)(b * a.nr + c), ov);
          tmem_wait_ld();
          if (ch >= a.dv) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            if (c + e >= x.pairs) break;
            const float y[2] = {__uint_as_float(ov[e]) * sh->inv[c + e], 0.f};
            *reinterpret_cast<uint16_t*>(out) = (uint16_t)Pack<T>::store(y);
            out += a.dv;
            if (!kLatent && ++head == a.group) {
              head = 0;
              out += (long long)span * a.dv;
            }
          }
        }
      }
    } else {
      if (row_ok) *reinterpret_cast<float2*>(a.part_ml + (x.part * a.nr + m) * 2) = make_float2(m_run, l_run);
      for (int b = 0; b < nob; ++b) {
        const int ch = b * 128 + m;
        float* part = a.part_o + x.part * a.nr * a.dv + ch;
        for (int c = 0; c < x.pairs; c += 32) {
          uint32_t ov[32];
          tmem_ld32(tmem + lane_off + 128u + (uint32_t)(b * a.nr + c), ov);
          tmem_wait_ld();
          if (ch >= a.dv) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e) {  // up to 31 columns behind the last pair's: room that nobody reads
            *part = __uint_as_float(ov[e]);
            part += a.dv;
          }
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
    tmem_dealloc(tmem, tmem_cols);
  }
}

// A pair's splits are merged in four slices -- split i in slice i % 4, a slice's in
// order -- and the slices in order.  dv threads a pair: a slice is dv / 4 of them, a
// thread four channels.
constexpr int kSlices = 4;

template <typename T>
__global__ void __launch_bounds__(512) rows_combine_kernel(const RowsAttnArgs a, const int per) {
  __shared__ float4 so[512];
  __shared__ float2 sml[4 * kSlices];
  pdl_launch_dependents();
  pdl_wait();
  const int g = blockIdx.y, groups = (a.tile_rows + per - 1) / per;
  const int w = blockIdx.x / groups;
  TileAt at;
  Place p;
  if (!find_tile(a, w, at) || !place_of(a, at, p) || p.splits == 1) return;  // the same for all threads
  const int c4 = a.dv / 4, mine = threadIdx.x / a.dv, slice = threadIdx.x % a.dv / c4, d4 = threadIdx.x % c4;
  const int r = blockIdx.x % groups * per + mine;
  const bool on = r < p.pairs;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  if (on) {
    const long long part0 = at.slot + (long long)at.tile * p.splits;
    constexpr int kAhead = 4;
    for (int i0 = slice; i0 < p.tile_splits; i0 += kAhead * kSlices) {
      float2 ml[kAhead];
      float4 x[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int i = i0 + j * kSlices;
        if (i >= p.tile_splits) break;
        const long long row = ((part0 + i) * a.hkv + g) * a.nr + r;
        ml[j] = __ldcg(reinterpret_cast<const float2*>(a.part_ml + row * 2));
        x[j] = __ldcg(reinterpret_cast<const float4*>(a.part_o + row * a.dv + 4 * d4));
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (i0 + j * kSlices >= p.tile_splits) break;
        const float mn = fmaxf(m, ml[j].x), z = mn == -INFINITY ? 0.f : mn;
        const float k0 = ex2_approx(m - z), k1 = ex2_approx(ml[j].x - z);
        v.x = v.x * k0 + x[j].x * k1;
        v.y = v.y * k0 + x[j].y * k1;
        v.z = v.z * k0 + x[j].z * k1;
        v.w = v.w * k0 + x[j].w * k1;
        l = l * k0 + ml[j].y * k1;
        m = mn;
      }
    }
  }
  so[threadIdx.x] = v;
  if (d4 == 0) sml[mine * kSlices + slice] = make_float2(m, l);
  __syncthreads();
  if (slice != 0 || !on) return;
  m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kSlices; ++i) m = fmaxf(m, sml[mine * kSlices + i].x);
  const float z = m == -INFINITY ? 0.f : m;
  v = make_float4(0.f, 0.f, 0.f, 0.f);
  l = 0.f;
#pragma unroll
  for (int i = 0; i < kSlices; ++i) {
    const float4 x = so[threadIdx.x + i * c4];
    const float2 y = sml[mine * kSlices + i];
    const float k = ex2_approx(y.x - z);
    v.x = fmaf(k, x.x, v.x);
    v.y = fmaf(k, x.y, v.y);
    v.z = fmaf(k, x.z, v.z);
    v.w = fmaf(k, x.w, v.w);
    l = fmaf(k, y.y, l);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int pair = p.first + r;
  const long long row = (long long)(p.row0 + pair / a.group) * a.hq + g * a.group + pair % a.group;
  const float o[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
  uint2 b;
  b.x = Pack<T>::store(o);
  b.y = Pack<T>::store(o + 2);
  *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * a.dv + 4 * d4) = b;
}

template <typename T, bool kLatent, bool kPaged>
cudaError_t launch_t(const RowsAttnArgs& a, int dtype, cudaStream_t st) {
  // Two CTAs an SM where their halves of TMEM and shared memory hold two stages.
  const int used = 128 + (a.dv + 127) / 128 * a.nr;
  const int ctas = used <= 256 && rows_layout(a.dqk, a.dv, kLatent, a.nr, 2).stages >= 2 ? 2 : 1;
  const RowsLayout l = rows_layout(a.dqk, a.dv, kLatent, a.nr, ctas);
  CUtensorMap tq, tk, tv;
  const CacheView& c = a.cache;
  const uint64_t slots = kPaged ? c.page_size : c.capacity;
  const uint64_t planes = (uint64_t)(kPaged ? c.num_pages : a.rows.num_seqs) * a.hkv;
  const uint32_t box = kPaged ? std::min(c.page_size, kTile) : kTile;
  const bool ok = (kLatent ? encode_3d(&tq, dtype, a.q, a.dqk, (uint64_t)a.total_rows * a.hq, 1, 64, a.q_rows, 1)
                           : encode_3d(&tq, dtype, a.q, a.dqk, a.hq, a.total_rows, 64, a.group, a.q_rows / a.group)) &&
                  encode_3d(&tk, dtype, a.k, a.dqk, slots, planes, 64, box, 1) &&
                  encode_3d(&tv, dtype, a.v, kLatent ? a.dqk : a.dv, slots, planes, 64, box, 1);
  if (!ok) return cudaErrorInvalidValue;
  // Raise the dynamic shared-memory limit once per device, so later calls --
  // including ones being captured into a CUDA graph -- only launch.
  static std::atomic<uint64_t> ready_mask{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready_mask.load(std::memory_order_acquire) & bit)) {
    // The register split is only sound at the per-thread count it was sized
    // for: refuse to launch a build that came out at another count.
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, rows_attn_kernel<T, kLatent, kPaged>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kRegsLaunch || fa.sharedSizeBytes != 0) return cudaErrorInvalidDeviceFunction;
    e = cudaFuncSetAttribute(rows_attn_kernel<T, kLatent, kPaged>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    ready_mask.fetch_or(bit, std::memory_order_release);
  }
  // As many CTAs an SM as meant, so that none waits for another's columns of TMEM.
  const uint32_t cols = ctas == 2 ? 256 : 512;
  const uint32_t smem = std::max(l.alloc, kSmemSM / (ctas + 1));
  const long long items = (long long)a.tiles_bound * a.hkv * a.max_splits;
  const dim3 grid((unsigned)std::min<long long>(items, 152 * ctas));
  e = launch_pdl(rows_attn_kernel<T, kLatent, kPaged>, grid, dim3(kThreads), smem, st, tq, tk, tv, a, l, cols);
  if (e != cudaSuccess || a.max_splits == 1) return e;
  const int per = std::max(1, 256 / a.dv);
  const dim3 cgrid((unsigned)(a.tiles_bound * ((a.tile_rows + per - 1) / per)), a.hkv);
  return launch_pdl(rows_combine_kernel<T>, cgrid, dim3(per * a.dv), 0, st, a, per);
}

template <typename T>
cudaError_t launch_type(const RowsAttnArgs& a, int dtype, cudaStream_t st) {
  const bool paged = a.cache.kind == CP_CACHE_PAGED;
  if (a.latent) return paged ? launch_t<T, true, true>(a, dtype, st) : launch_t<T, true, false>(a, dtype, st);
  return paged ? launch_t<T, false, true>(a, dtype, st) : launch_t<T, false, false>(a, dtype, st);
}

}  // namespace

RowsPlan rows_plan(int hq, int hkv, bool latent, int dv, bool uniform, long long num_seqs, long long total_rows, int max_ctx) {
  RowsPlan p;
  const int group = hq / hkv;
  const long long pairs = (uniform ? total_rows / num_seqs : total_rows) * group;  // of a sequence, at most
  p.nr = dv > 256 ? 64 : 128;  // what the output's columns of TMEM leave room for
  p.tile_rows = latent ? p.nr : p.nr / group * group;
  p.q_rows = (int)std::min<long long>(p.tile_rows, pairs);
  p.tiles = uniform ? num_seqs * ((pairs + p.tile_rows - 1) / p.tile_rows) : pairs / p.tile_rows + 1 + num_seqs;
  p.max_splits = rows_max_splits(max_ctx, 1);
  p.slots = p.max_splits == 1 ? 0 : std::min(p.tiles * p.max_splits, num_seqs * kRowsMaxSlots);
  p.bytes = (double)p.slots * hkv * p.nr * (dv + 2) * sizeof(float);
  return p;
}

cudaError_t launch_rows_attn(const RowsAttnArgs& a, int dtype, cudaStream_t st) {
  return dtype == CP_BF16 ? launch_type<__nv_bfloat16>(a, dtype, st) : launch_type<__half>(a, dtype, st);
}

}  // namespace cp
