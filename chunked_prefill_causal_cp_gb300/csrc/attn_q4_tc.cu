// attn_q4_tc.cu -- chunks of query rows over a 4-bit cache on the sm_103a tensor
// cores (tcgen05 + TMEM).
//
// A chunk's row does 4 D operations per key and head while the cache's bytes
// are shared by 256 packed rows, so the path is bound by the tensor cores, and
// the codes have to become matrix operands beside them.  The work is cut as in
// the 16-bit kernel (attn_tc.cu): 128-row Q tiles of 128 / G tokens x G heads, a
// cluster of two CTAs owning a pair of Q tiles, each CTA holding both and
// walking every other 128-key tile, so that a tile is converted once for 256
// rows.  In place of the TMA producer seven warps convert: a thread takes one
// group of 32 channels of one key (16 bytes of codes, one pair of parameters,
// copied ahead to shared memory by cp.async), turns each word into four pairs of
// 16-bit values (cp_q4.cuh) and stores them, 16 bytes at a time, where the
// 128-byte-swizzled operand wants them.  The next tile's codes are on their way before
// the current one's are all converted (held in registers instead, they spilled, the
// loads ran one after another and the kernel took 1.8 times as long; as it is, 60
// bytes a thread spill at 128 channels).  The values are rounded to 16 bits once, as
// the cache's format defines them.  The softmax's weights are rounded to 16 bits too,
// as the tensor cores take both operands in the layer's type; their sum is not.
// Keys past the sequence's positions, and keys on a bad page, are written as
// zeros, so nothing unwritten reaches a product; their scores are masked.
//
// Warp roles (512 threads per CTA, four warpgroups):
//   warps 0, 2-7   conversion (warp 0 also issues the Q tiles' TMA loads)
//   warp 1         TMEM allocation and MMA issue:  S0 = Q0 K^T, S1 = Q1 K^T,
//                  O0 += P0 V, O1 += P1 V per tile
//   warps 8-11, 12-15  softmax of Q tile 0 and 1, a thread per row
// TMEM: group w has [256w, 256w + 128) for S and P, [256w + 128, + D) for O.
// The MMA warp issues S_w(i + 1) after O_w += P_w(i) V(i), and tcgen05 operations of
// one thread complete in order, so S_w(i + 1) complete means P_w(i) may be
// overwritten and O_w rescaled.  O is rescaled only when a row's maximum has grown
// by more than 2^8.
//
// Measured (32/8 heads x 128, bf16): 8128 rows over 8128 cached keys in 1.31 ms, 1.24
// PFLOP/s, 0.65 of the measured bf16 rate; the 16-bit kernel takes about 1.21 ms for
// the same rows.  Copies that leave work out: no conversion 1.22 ms, no conversion
// and no copies of codes 1.15 ms -- the conversion's instructions compete with
// the softmax's.  On the way: three conversion warps 2.0 ms; lanes by group, with
// reordered stores, 1.44 ms; 56 / 64 / 80 / 88 control registers 1.67 / 1.32 / 1.31 /
// 1.41 ms; twice the blocks for the warp beside the MMA warp 1.36 against 1.32 ms.
//
// Merge: each CTA's (max, sum, unnormalised O) of the Q tile that its peer
// finishes goes to the peer in 16 KB column chunks over distributed shared
// memory; even tiles' half first, so the order is fixed.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cp_host.h"
#include "cp_ptx.cuh"
#include "cp_q4.cuh"
#include "cp_q4.h"
#include "cp_rows.cuh"

namespace cp {
namespace {

constexpr int kThreads = 512;
constexpr int kConvWarps = 7;
constexpr int kConvThreads = kConvWarps * 32;
// Register split: compiled at kRegsLaunch a thread (the most 512 threads may
// have); the two control warpgroups drop to kRegsControl and hand the rest to
// the softmax warpgroups.
constexpr int kRegsLaunch = 128;
constexpr int kRegsControl = 72;
constexpr int kRegsSoftmax = 184;
static_assert(256 * kRegsControl + 256 * kRegsSoftmax == kThreads * kRegsLaunch, "the split must add up");
constexpr int kStages = 2;
constexpr uint32_t kBlockBytes = 128 * 128;  // [128 rows][64 x 16-bit] = 16 KB
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.0f;

struct __align__(16) Q4Barriers {
  uint64_t q_full[2];
  uint64_t k_full[kStages], v_full[kStages], k_empty[kStages], v_empty[kStages];
  uint64_t s_full[2], p_ready[2];
  uint64_t o_final;
  uint64_t merge_full[4];  // column chunk c of the peer's part for this CTA's rows has landed
  uint64_t peer_free;      // the peer's K/V stages may receive this CTA's part
  uint32_t tmem_base;
  int abort;
  int bad_tile[kStages];   // the last tile of the stage with a non-finite V group, of those that hide keys from a row
  __align__(16) float peer_ml[256];  // the peer's maximum [0, 128) and sum [128, 256) of this CTA's rows
  __align__(16) float out_ml[256];   // this CTA's for the peer's rows
};

template <int D>
struct Q4Smem {
  static constexpr int DB = D / 64;
  static constexpr uint32_t q_off = 0;
  static constexpr uint32_t k_off = q_off + 2 * DB * kBlockBytes;
  static constexpr uint32_t v_off = k_off + kStages * DB * kBlockBytes;
  static constexpr uint32_t bar_off = v_off + kStages * DB * kBlockBytes;
  static constexpr uint32_t raw_off = bar_off + sizeof(Q4Barriers);  // codes and parameters on their way (see Conv)
  static constexpr uint32_t raw_bytes = 2u * ((4 * D / 32 + kConvWarps - 1) / kConvWarps) * kConvThreads * 20u;
  static constexpr uint32_t alloc = raw_off + raw_bytes + 1024;  // slack for 1024-byte alignment
  static_assert(alloc <= 232448, "one CTA's shared memory");
  // After the main loop the K stages hold the outgoing part, the V stages the
  // peer's: 128 rows x D fp32 as D / 32 column chunks.
  static constexpr int kMergeChunks = D / 32;
  static constexpr uint32_t kChunkBytes = 128u * 32u * 4u;
  static_assert(kStages * DB * kBlockBytes == 128u * D * 4u, "a part is exactly the K (or V) stages");
};

// Byte offset of 16-byte piece e (columns 32c + 4e .. +3) of row m in a merge
// buffer: chunk c is a contiguous [128 rows][128 B] block, and the pieces of
// a row are XOR-swizzled by (m mod 8), so the 8 rows a quarter-warp touches at
// once fall on distinct banks.
__device__ __forceinline__ uint32_t merge_off(int m, int c, int e) {
  return (uint32_t)c * (128u * 128u) + (uint32_t)m * 128u + (uint32_t)((e ^ (m & 7)) * 16);
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Which (sequence, first token) a cluster owns; a pair covers 2 * 128 / G tokens.
// Within a sequence the pairs are handed out last-first, so those with the most
// keys start earliest.  Every warp of the CTA calls this with all lanes: for
// ragged rows each warp scans the sequences 32 at a time.
__device__ __forceinline__ bool find_pair(const Q4AttnArgs& a, int ppt, int w, int& s, int& t0) {
  if (a.rows.rows_uniform > 0) {
    const int np = (a.rows.rows_uniform + ppt - 1) / ppt;
    const int pair = np - 1 - w / a.rows.num_seqs;
    s = w % a.rows.num_seqs;
    if (pair < 0) return false;
    t0 = pair * ppt;
    return true;
  }
  const int lane = threadIdx.x & 31;
  for (int q0 = 0; q0 < a.rows.num_seqs; q0 += 32) {
    const int q = q0 + lane;
    int np = 0;
    if (q < a.rows.num_seqs) {
      const int r = seq_rows(a.rows, q);
      np = r < a.min_rows ? 0 : (r + ppt - 1) / ppt;
    }
    int inc = np;  // inclusive prefix sum over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const int tot = __shfl_sync(0xffffffffu, inc, 31);
    if (w < tot) {
      const int L = __ffs(__ballot_sync(0xffffffffu, inc > w)) - 1;
      const int before = __shfl_sync(0xffffffffu, inc - np, L);
      const int npl = __shfl_sync(0xffffffffu, np, L);
      s = q0 + L;
      t0 = (npl - 1 - (w - before)) * ppt;
      return true;
    }
    w -= tot;
  }
  return false;
}

// 16- or 4-byte asynchronous copies to shared memory; `on` false: zeros, nothing is read.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's share of a tile of K or V: blocks of 32 groups of 32 channels -- kKeys
// keys, lane kKeys j + k taking group j of the block's key k -- warp cw taking
// blocks cw, cw + kConvWarps, ....  The codes pass through slots of shared memory
// that only their own thread writes and reads, so a copy needs no barrier, and no
// registers while it is in flight.
template <typename T, int D, bool kPaged>
struct Conv {
  static constexpr int kGroups = D / 32;
  static constexpr int kKeys = 32 / kGroups;
  static constexpr int kBlocks = 128 / kKeys;
  static constexpr int kPer = (kBlocks + kConvWarps - 1) / kConvWarps;
  struct Slots {
    uint4 w[kPer][kConvThreads];
    uint32_t p[kPer][kConvThreads];
  };
  static_assert(sizeof(Slots) * 2 == Q4Smem<D>::raw_bytes, "the slots' place");

  // Page of each of the tile's pages, in lane's turn (-1: a bad page, or none).
  static __device__ __forceinline__ int tile_pages(const Q4AttnArgs& a, int s, int j0, int n) {
    const int lane = threadIdx.x & 31, lps = 31 - __clz(a.cache.page_size);
    const int key = j0 + (lane << lps), blk = key >> lps;
    if ((lane << lps) >= kTcBlockN || key >= n) return -1;
    int page = blk < a.cache.max_blocks ? a.cache.block_table[(long long)s * a.cache.max_blocks + blk] : -1;
    if (page < 0 || page >= a.cache.num_pages) {
      page = -1;
      if (a.status) atomicOr(a.status, CP_DEV_BOUNDS);
    }
    return page;
  }

  // Starts the copies of keys j0 + ... < n; others become zeros.
  static __device__ __forceinline__ void load(const Q4AttnArgs& a, const uint8_t* codes, const uint32_t* params, int s,
                                              int g, int pages, int j0, int n, int cw, Slots& x) {
    const int lane = threadIdx.x & 31, grp = lane / kKeys, key0 = cw * kKeys + lane % kKeys;
    const int ps = a.cache.page_size, lps = kPaged ? 31 - __clz(ps) : 0;
    const uint8_t* par = reinterpret_cast<const uint8_t*>(params);
    // Bytes of codes before the tile's (page's) first row; a row has a quarter as many bytes of parameters.
    const long long base = kPaged ? (long long)(g << lps) * (D / 2)
                                  : (((long long)s * a.hkv + g) * a.cache.capacity + j0 + key0) * (D / 2);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (kBlocks % kConvWarps != 0 && cw + i * kConvWarps >= kBlocks) break;  // whole warps
      const int key = key0 + i * (kConvWarps * kKeys);
      bool on = j0 + key < n;
      long long at = base + i * (kConvWarps * kKeys * (D / 2));
      if constexpr (kPaged) {
        const int page = __shfl_sync(0xffffffffu, pages, key >> lps);
        on = on && page >= 0;
        at = base + (long long)page * (a.hkv * ps * (D / 2)) + (key & (ps - 1)) * (D / 2);
      }
      if (!on) at = 0;
      cp_async16(&x.w[i][cw * 32 + lane], codes + at + grp * 16, on);
      cp_async4(&x.p[i][cw * 32 + lane], par + (at >> 2) + grp * 4, on);
    }
    cp_async_commit();
  }

  // The values into a stage: key row of 128 bytes in 64-channel block grp / 2,
  // 16-byte chunks XOR-swizzled by key mod 8: the eight threads of a store phase
  // hold the same chunk of eight keys, on distinct banks.  With `guard`, groups that
  // are not finite are stored as zeros; true if there were any.
  static __device__ __forceinline__ bool store(const Slots& from, uint8_t* stage, int cw, uint32_t magic, bool guard) {
    bool bad = false;
    const int lane = threadIdx.x & 31, grp = lane / kKeys, k = lane % kKeys;
    uint8_t* at = stage + (grp >> 1) * kBlockBytes + (cw * kKeys + k) * 128;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (kBlocks % kConvWarps != 0 && cw + i * kConvWarps >= kBlocks) break;
      const uint4 w = from.w[i][cw * 32 + lane];
      uint32_t p = from.p[i][cw * 32 + lane];
      if (guard && q4_nonfinite<T>(p)) {
        p = 0;
        bad = true;
      }
      const Q4Scale sm = q4_scale<T>(q4_scale2(p), q4_low2(p));
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t v[4];
        q4_four<T>(x[c], sm, magic, v);
        *reinterpret_cast<uint4*>(at + i * (kConvWarps * kKeys * 128) + ((((grp & 1) * 4 + c) ^ (k & 7)) * 16)) =
            make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
    return bad;
  }
};

template <typename T, int D, bool kPaged>
__global__ void __launch_bounds__(kThreads, 1)
    q4_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_o,
                 const Q4AttnArgs a) {
  using L = Q4Smem<D>;
  constexpr int DB = L::DB;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kIdescQK = make_idesc_f16(kBf16, 128, 128, false);
  constexpr uint32_t kIdescPV = make_idesc_f16(kBf16, 128, D, true);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + L::q_off;
  uint8_t* sK = smem + L::k_off;
  uint8_t* sV = smem + L::v_off;
  Q4Barriers* bar = reinterpret_cast<Q4Barriers*>(smem + L::bar_off);

  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.group;
  const int rpt = kTcBlockM / G;  // tokens per Q tile
  const int g = blockIdx.y;
  const int rank = (int)cluster_ctarank();

  // ---- set-up that reads no global memory: it may overlap the previous kernel
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar->k_full[i], kConvThreads);
      mbar_init(&bar->v_full[i], kConvThreads);
      mbar_init(&bar->k_empty[i], 1);
      mbar_init(&bar->v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->q_full[i], 1);
      mbar_init(&bar->s_full[i], 1);
      mbar_init(&bar->p_ready[i], 128);
    }
    mbar_init(&bar->o_final, 1);
    for (int c = 0; c < L::kMergeChunks; ++c) mbar_init(&bar->merge_full[c], 1);
    mbar_init(&bar->peer_free, 1);
    bar->abort = 0;
    for (int i = 0; i < kStages; ++i) bar->bad_tile[i] = -1;
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_o);
  }
  if (warp == 1) {
    tmem_alloc(&bar->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_arrive();  // barrier inits are visible cluster-wide before any remote access (waited below)
  const uint32_t tmem = bar->tmem_base;
  volatile int* abort_flag = &bar->abort;
  pdl_wait();  // everything below reads what earlier kernels wrote
  if (a.commit_lens && blockIdx.x == 0 && blockIdx.y == 0)  // `past` is a copy: the lengths may advance at once
    for (int q = threadIdx.x; q < a.rows.num_seqs; q += kThreads) a.commit_lens[q] += seq_rows(a.rows, q);

  // ---- this cluster's pair (the same for both CTAs, so both leave together)
  int s = 0, t0 = 0, rows = 0, past = 0, row0 = 0;
  bool have_pair = find_pair(a, 2 * rpt, (int)(blockIdx.x >> 1), s, t0);
  if (have_pair) {
    rows = seq_rows(a.rows, s);
    past = a.past[s];
    row0 = seq_row0(a.rows, s);
    if (past < 0 || (long long)past + rows > a.max_ctx || row0 < 0 || row0 > a.total_rows - rows) {
      if (a.status && threadIdx.x == 0 && rank == 0) atomicOr(a.status, CP_DEV_BOUNDS);
      have_pair = false;
    }
  }
  if (!have_pair) {
    cluster_wait();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
      tc_fence_after();
      tmem_dealloc(tmem, kTmemCols);
    }
    return;
  }
  const int n = past + rows;  // positions written, this call's rows among them
  const int t_end = min(t0 + 2 * rpt, rows);
  const int ntiles = (past + t_end + kTcBlockN - 1) / kTcBlockN;
  const int nmine = ntiles > rank ? (ntiles - rank + 1) / 2 : 0;  // this CTA's tiles: rank + 2i
  const bool q1 = t0 + rpt < rows;  // Q tile 1 holds at least one row (else it is skipped)
  const bool own_tile = rank == 0 || q1;   // Q tile `rank` (finished here) has rows
  const bool peer_tile = rank == 1 || q1;  // Q tile `1 - rank` (finished by the peer) has rows
  const uint32_t peer = (uint32_t)(1 - rank);
  if (threadIdx.x == 0 && own_tile)
    for (int c = 0; c < L::kMergeChunks; ++c)  // chunk 0 also brings the peer's (max, sum)
      mbar_arrive_expect_tx(&bar->merge_full[c], L::kChunkBytes + (c == 0 ? 256u * 4u : 0u));

  if (warp < 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
  if (warp != 1) {
    // ================================================================ conversion
    if (threadIdx.x == 0 && nmine > 0)
      for (int w = 0; w < (q1 ? 2 : 1); ++w) {
        mbar_arrive_expect_tx(&bar->q_full[w], DB * kBlockBytes);
        for (int db = 0; db < DB; ++db)
          tma_load_3d(sQ + (w * DB + db) * kBlockBytes, &tm_q, &bar->q_full[w], db * 64, g * G, row0 + t0 + w * rpt);
      }
    // The tile's blocks do not divide evenly: the warps that take one more of K are not those of V.
    const int cw = warp == 0 ? 0 : warp - 1;
    const int ck = cw, cv = (cw + 5) % kConvWarps;
    using C = Conv<T, D, kPaged>;
    const uint32_t magic = q4_magic<T>();
    auto* raw = reinterpret_cast<typename C::Slots*>(smem + L::raw_off);  // K's and V's
    int pages = -1;  // of the tile whose copies start next
    if (nmine > 0) {
      const int j0 = rank * kTcBlockN;
      if (kPaged) pages = C::tile_pages(a, s, j0, n);
      C::load(a, a.k_codes, a.k_params, s, g, pages, j0, n, ck, raw[0]);
      C::load(a, a.v_codes, a.v_params, s, g, pages, j0, n, cv, raw[1]);
    }
    for (int i = 0; i < nmine; ++i) {
      const int st = i & 1;
      const int j1 = (rank + 2 * i + 2) * kTcBlockN;  // this CTA's next tile
      const bool more = i + 1 < nmine;
      if (kPaged && more) pages = C::tile_pages(a, s, j1, n);
      const uint32_t free_ph = ((i >> 1) & 1) ^ 1;
      if (!warp_wait(&bar->k_empty[st], free_ph, abort_flag, a.status)) break;
      cp_async_wait<1>();  // K of this tile
      C::store(raw[0], sK + st * DB * kBlockBytes, ck, magic, false);
      fence_proxy_async_smem();  // the tensor cores read the stage through the async proxy
      mbar_arrive(&bar->k_full[st]);
      if (more) C::load(a, a.k_codes, a.k_params, s, g, pages, j1, n, ck, raw[0]);
      else cp_async_commit();  // the groups stay in step
      if (!warp_wait(&bar->v_empty[st], free_ph, abort_flag, a.status)) break;
      cp_async_wait<1>();  // V of this tile
      // A tile with keys that some row of the pair does not see: 0 * NaN must not reach that row's sum.
      const int tile = rank + 2 * i;
      const bool guard = tile * kTcBlockN + kTcBlockN - 1 > past + t0;
      if (C::store(raw[1], sV + st * DB * kBlockBytes, cv, magic, guard)) bar->bad_tile[st] = tile;
      fence_proxy_async_smem();
      mbar_arrive(&bar->v_full[st]);
      if (more) C::load(a, a.v_codes, a.v_params, s, g, pages, j1, n, cv, raw[1]);
      else cp_async_commit();
    }
    cp_async_wait<0>();
    if (threadIdx.x == 0 && nmine > 0 && *abort_flag) {
      // Let the Q copies in flight land before the CTA's shared memory is released.
      volatile int zero = 0;
      mbar_wait(&bar->q_full[0], 0, &zero, nullptr);
      if (q1) mbar_wait(&bar->q_full[1], 0, &zero, nullptr);
    }
    __syncwarp();
  } else {
    // ================================================================ MMA issuer
    // The whole warp runs the loop, converged; one elected lane issues.
    auto wait = [&](uint64_t* b, uint32_t parity) { return warp_wait(b, parity, abort_flag, a.status); };
    constexpr uint64_t kTileStep = (DB * kBlockBytes) >> 4;
    const uint64_t q_desc0 = make_sdesc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t k_desc0 = make_sdesc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t v_desc0 = make_sdesc_sw128(smem_u32(sV), kBlockBytes, 1024);
    auto issue_qk = [&](int w, int i) {  // S_w = Q_w K_i^T
      const uint64_t q_desc = q_desc0 + w * kTileStep;
      const uint64_t k_desc = k_desc0 + (i & 1) * kTileStep;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = ((kk >> 2) * kBlockBytes + (kk & 3) * 32) >> 4;
        mma_ss_elect(tmem + 256u * w, q_desc + off, k_desc + off, kIdescQK, kk > 0);
      }
      mma_commit_elect(&bar->s_full[w]);
    };
    auto issue_pv = [&](int w, int i) {  // O_w += P_w V_i
      const uint64_t v_desc = v_desc0 + (i & 1) * kTileStep;
#pragma unroll
      for (int kk = 0; kk < kTcBlockN / 16; ++kk)
        mma_ts_elect(tmem + 256u * w + 128u, tmem + 256u * w + kk * 8, v_desc + ((kk * 2048) >> 4), kIdescPV,
                     (i > 0 || kk > 0) ? 1u : 0u);
    };
    bool ok = nmine > 0 && wait(&bar->q_full[0], 0) && wait(&bar->k_full[0], 0);
    if (ok) {
      tc_fence_after();
      issue_qk(0, 0);
    }
    if (ok && q1) {
      ok = wait(&bar->q_full[1], 0);
      if (ok) {
        tc_fence_after();
        issue_qk(1, 0);
      }
    }
    if (ok) mma_commit_elect(&bar->k_empty[0]);  // K's stage is free long before V's
    for (int i = 0; ok && i < nmine; ++i) {
      const bool more = i + 1 < nmine;
      if (!wait(&bar->p_ready[0], i & 1)) break;
      if (!wait(&bar->v_full[i & 1], (i >> 1) & 1)) break;
      tc_fence_after();
      issue_pv(0, i);
      if (more) {
        if (!wait(&bar->k_full[(i + 1) & 1], ((i + 1) >> 1) & 1)) break;
        tc_fence_after();
        issue_qk(0, i + 1);
      }
      if (q1) {
        if (!wait(&bar->p_ready[1], i & 1)) break;
        tc_fence_after();
        issue_pv(1, i);
      }
      mma_commit_elect(&bar->v_empty[i & 1]);
      if (more) {
        if (q1) issue_qk(1, i + 1);
        mma_commit_elect(&bar->k_empty[(i + 1) & 1]);
      }
    }
    // o_final: every MMA issued has completed (the epilogue and the TMEM release wait for it).
    mma_commit_elect(&bar->o_final);
    volatile int zero = 0;  // wait even after an abort: MMAs may still be in flight
    mbar_wait(&bar->o_final, 0, &zero, a.status);
    __syncwarp();
  }
  cluster_wait();  // the peer's barriers are initialised
  if (warp == 1 && lane == 0 && own_tile) {
    // This CTA's MMAs are complete (the issuer waited o_final): its K/V stages are free.
    mbar_arrive_remote(mapa_shared(smem_u32(&bar->peer_free), peer));
  }
  } else {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
  // ================================================================ softmax groups
  const int grp = (warp - 8) >> 2;          // Q tile of this group
  const int quarter = warp & 3;             // TMEM lanes [32*quarter, +32)
  const int mrow = quarter * 32 + lane;     // this thread's row of its Q tile
  const int tok = t0 + grp * rpt + mrow / G;
  const int head = g * G + mrow % G;
  const bool row_ok = tok < t_end;
  const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
  const uint32_t s_col = tmem + lane_off + 256u * grp;
  const uint32_t o_col = s_col + 128u;
  float m_run = -INFINITY;  // max used for exponentiation (log2 domain)
  float l_run = 0.f;
  bool alive = true;
  if (grp == 0 || q1) {
    const int p_row = row_ok ? past + tok : -1;  // absolute query position
    const float sl2 = a.scale_log2;
    for (int i = 0; i < nmine; ++i) {
      if (!warp_wait(&bar->s_full[grp], i & 1, abort_flag, a.status)) { alive = false; break; }
      tc_fence_after();
      uint32_t sv[128];
      tmem_ld32(s_col + 0, &sv[0]);
      tmem_ld32(s_col + 32, &sv[32]);
      tmem_ld32(s_col + 64, &sv[64]);
      tmem_ld32(s_col + 96, &sv[96]);
      tmem_wait_ld();
      const int c_hi = p_row + 1 - (rank + 2 * i) * kTcBlockN;  // visible columns [0, c_hi)
      if (c_hi < kTcBlockN) {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= c_hi) sv[c] = __float_as_uint(-INFINITY);
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
      const float mx2 = mx * sl2;  // scale > 0, so the max commutes with it
      const bool grow = mx2 > m_run + kRescaleLog2 || (m_run == -INFINITY && mx2 != -INFINITY);
      const float m_new = grow ? mx2 : m_run;
      const float alpha = grow ? (m_run == -INFINITY ? 0.f : ex2_approx(m_run - m_new)) : 1.f;
      const float neg_m = (m_new == -INFINITY) ? 0.f : -m_new;
      float ps4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 64; ++c) {
        float x0 = __uint_as_float(sv[2 * c]), x1 = __uint_as_float(sv[2 * c + 1]);
        ffma2(x0, x1, sl2, neg_m);
        const float p0 = ex2_approx(x0);
        const float p1 = ex2_approx(x1);
        fadd2(ps4[2 * (c & 1)], ps4[2 * (c & 1) + 1], p0, p1);
        sv[c] = pack2<T>(p0, p1);
      }
      const float psum = (ps4[0] + ps4[1]) + (ps4[2] + ps4[3]);
      l_run = l_run * alpha + psum;
      m_run = m_new;
      tmem_st32(s_col + 0, &sv[0]);
      tmem_st32(s_col + 32, &sv[32]);
      // O holds P V of this group's earlier tiles (complete: see the ordering
      // note above).  Rows whose max grew rescale it; the others multiply by 1.
      if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32(o_col + 32 * c, ov);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
          tmem_st32(o_col + 32 * c, ov);
        }
      }
      // A non-finite V group stands as zeros where keys are hidden from a row of the pair: the rows that see it
      // become NaN by their sum.
      const int tile = rank + 2 * i;
      if (tile * kTcBlockN + kTcBlockN - 1 > past + t0) {
        if (!warp_wait(&bar->v_full[i & 1], (i >> 1) & 1, abort_flag, a.status)) { alive = false; break; }
        if (*static_cast<volatile int*>(&bar->bad_tile[i & 1]) == tile) {
          for (int c = 0; c < min(c_hi, kTcBlockN); ++c) {
            const long long row = cache_row(a.cache, a.hkv, s, g, tile * kTcBlockN + c, a.max_ctx);
            for (int j = 0; row >= 0 && j < D / 32; ++j)
              if (q4_nonfinite<T>(a.v_params[row * (D / 32) + j])) l_run = __int_as_float(0x7fffffff);
          }
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bar->p_ready[grp]);
    }
  }

  // ================================================================ merge across the pair
  volatile int zero = 0;
  const bool done = warp_wait(&bar->o_final, 0, &zero, a.status) && alive;
  tc_fence_after();
  __syncwarp();
  cluster_wait();  // the peer's barriers are initialised
  const bool have_o = nmine > 0;  // this CTA wrote O (else its TMEM O is unset: send zeros)
  if (grp != rank && peer_tile) {
    // Rows of Q tile (1 - rank) are finished by the peer: stage this CTA's
    // partial one 32-column chunk at a time and send each chunk as soon as it
    // is staged, so one chunk's transfer overlaps the staging of the next.
    bar->out_ml[mrow] = have_o ? m_run : -INFINITY;
    bar->out_ml[128 + mrow] = have_o ? l_run : 0.f;
    bool send = true;  // (meaningful in the thread of row 0, which sends)
#pragma unroll
    for (int c = 0; c < L::kMergeChunks; ++c) {
      uint32_t ov[32];
      if (have_o) {
        tmem_ld32(o_col + 32 * c, ov);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) ov[e] = 0u;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        *reinterpret_cast<uint4*>(sK + merge_off(mrow, c, e)) =
            make_uint4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
      fence_proxy_async_smem();  // the bulk copy reads these through the async proxy
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (mrow == 0) {
        if (c == 0) send = mbar_wait_cluster(&bar->peer_free, 0, a.status);
        if (send) {
          const uint32_t rbar = mapa_shared(smem_u32(&bar->merge_full[c]), peer);
          bulk_copy_to_peer(mapa_shared(smem_u32(sV + c * L::kChunkBytes), peer), sK + c * L::kChunkBytes,
                            L::kChunkBytes, rbar);
          if (c == 0) bulk_copy_to_peer(mapa_shared(smem_u32(bar->peer_ml), peer), bar->out_ml, 256u * 4u, rbar);
        }
      }
    }
  }
  if (grp == rank && own_tile) {
    // Fixed order: the even-tile half (rank 0's partial) first.  Chunk 0
    // brings the peer's (max, sum); each chunk is combined as it lands.
    bool got = mbar_wait_cluster(&bar->merge_full[0], 0, a.status);
    const float m_own = have_o ? m_run : -INFINITY, l_own = have_o ? l_run : 0.f;
    const float m_peer = bar->peer_ml[mrow], l_peer = bar->peer_ml[128 + mrow];
    const float mA = rank == 0 ? m_own : m_peer, lA = rank == 0 ? l_own : l_peer;
    const float mB = rank == 0 ? m_peer : m_own, lB = rank == 0 ? l_peer : l_own;
    const float mm = fmaxf(mA, mB);
    const float wA = (mA == -INFINITY) ? 0.f : ex2_approx(mA - mm);
    const float wB = (mB == -INFINITY) ? 0.f : ex2_approx(mB - mm);
    const float lsum = lA * wA + lB * wB;
    const float inv = lsum == 0.f ? 0.f : 1.f / lsum;  // a NaN stays
    // A tile whose rows all belong to this sequence leaves through a TMA store
    // from the (now unused) Q buffer; a ragged tile row by row.
    const int tile_tok0 = t0 + rank * rpt;
    const bool full_tile = tile_tok0 + rpt <= t_end;
    uint8_t* sOut = sQ + rank * DB * kBlockBytes;
    T* out = static_cast<T*>(a.out) + ((long long)(row0 + tok) * a.hq + head) * D;
#pragma unroll
    for (int c = 0; c < L::kMergeChunks; ++c) {
      if (c > 0 && got) got = mbar_wait_cluster(&bar->merge_full[c], 0, a.status);
      uint32_t ov[32];
      if (have_o) {
        tmem_ld32(o_col + 32 * c, ov);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) ov[e] = 0u;
      }
      uint32_t pk[16];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 pr = *reinterpret_cast<const float4*>(sV + merge_off(mrow, c, e));
        const float own[4] = {__uint_as_float(ov[4 * e]), __uint_as_float(ov[4 * e + 1]),
                              __uint_as_float(ov[4 * e + 2]), __uint_as_float(ov[4 * e + 3])};
        const float prv[4] = {pr.x, pr.y, pr.z, pr.w};
        float x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = rank == 0 ? own[u] * wA + prv[u] * wB : prv[u] * wA + own[u] * wB;
        pk[2 * e] = pack2<T>(x[0] * inv, x[1] * inv);
        pk[2 * e + 1] = pack2<T>(x[2] * inv, x[3] * inv);
      }
      if (full_tile) {
        // Columns [32c, 32c + 32) are 16-byte chunks 4(c%2) .. 4(c%2)+3 of box c/2 (128B swizzle).
        uint8_t* box = sOut + (c >> 1) * kBlockBytes + mrow * 128;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int chunk = (c & 1) * 4 + e;
          *reinterpret_cast<uint4*>(box + ((chunk ^ (mrow & 7)) * 16)) =
              make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
        }
      } else if (done && got && row_ok) {
        uint4* dst = reinterpret_cast<uint4*>(out + 32 * c);
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[e] = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
      }
    }
    if (full_tile) {
      fence_proxy_async_smem();  // the TMA store reads the tile through the async proxy
      asm volatile("bar.sync 2, 128;" ::: "memory");
      if (mrow == 0 && done && got) {
        for (int db = 0; db < DB; ++db)
          tma_store_3d(&tm_o, sOut + db * kBlockBytes, db * 64, g * G, row0 + tile_tok0);
        bulk_commit_group();
        bulk_wait_read_all();  // the Q buffer is read out; the writes finish with the grid
      }
    }
  }
  }  // softmax warpgroups

  // Both CTAs leave together: the copies each sent into the other have landed
  // and been read before either CTA's shared memory is released.
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <typename T, int D, bool kPaged>
cudaError_t launch_t(const Q4AttnArgs& a, const CUtensorMap& tq, const CUtensorMap& to, int pairs_bound,
                     cudaStream_t st) {
  // D = 64 would fit two CTAs per SM, but each CTA takes all 512 TMEM columns;
  // ask for enough shared memory to keep it at one CTA per SM.
  const uint32_t smem = Q4Smem<D>::alloc < 120u * 1024u ? 120u * 1024u : Q4Smem<D>::alloc;
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
    e = cudaFuncGetAttributes(&fa, q4_tc_kernel<T, D, kPaged>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidDeviceFunction;
    e = cudaFuncSetAttribute(q4_tc_kernel<T, D, kPaged>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    ready_mask.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(2 * pairs_bound, a.hkv);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, q4_tc_kernel<T, D, kPaged>, tq, to, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_q4_tc(const Q4AttnArgs& a, int dtype, int d, int pairs_bound, cudaStream_t st) {
  if (pairs_bound <= 0) return cudaSuccess;
  // Q and out rows [total_rows, Hq, D] in boxes of 64 channels, G heads, 128 / G tokens.
  CUtensorMap tq, to;
  if (!encode_3d(&tq, dtype, a.q, d, a.hq, a.total_rows, 64, a.group, kTcBlockM / a.group) ||
      !encode_3d(&to, dtype, a.out, d, a.hq, a.total_rows, 64, a.group, kTcBlockM / a.group))
    return cudaErrorInvalidValue;
  const bool paged = a.cache.kind == CP_CACHE_PAGED;
  if (dtype == CP_BF16)
    return d == 64 ? (paged ? launch_t<__nv_bfloat16, 64, true> : launch_t<__nv_bfloat16, 64, false>)(a, tq, to, pairs_bound, st)
                   : (paged ? launch_t<__nv_bfloat16, 128, true> : launch_t<__nv_bfloat16, 128, false>)(a, tq, to, pairs_bound, st);
  return d == 64 ? (paged ? launch_t<__half, 64, true> : launch_t<__half, 64, false>)(a, tq, to, pairs_bound, st)
                 : (paged ? launch_t<__half, 128, true> : launch_t<__half, 128, false>)(a, tq, to, pairs_bound, st);
}

}  // namespace cp
