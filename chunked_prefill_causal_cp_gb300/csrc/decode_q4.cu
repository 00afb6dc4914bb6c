// decode_q4.cu -- single rows and short chunks over a 4-bit cache, split along
// the keys.
//
// A decode row reads its sequence's cache once and does about 13 operations of
// attention per byte, so the path is bound by the bytes of the cache (160 per
// key and KV head at 128 channels) as long as the codes turn into matrix
// operands quickly enough: at full bandwidth an SM has some 28 instructions per
// key, and turning 256 codes into 16-bit values takes 13 of them.  One CTA takes
// 256 to 1024 keys of a (sequence, KV head), four warps a quarter each; the k rows
// of the sequence times the G heads of the group (k * G <= 16) ride in the columns of
// m16n8k16 products, so every row shares one read of the cache and one
// conversion of its codes.  A warp walks its keys 16 at a time, in a rolled loop
// (unrolled over the whole range, the code outgrew the instruction cache and
// took 585 instructions a tile):
//   Copies: the tile's codes and parameters come through a four-stage ring of
//   shared memory of the warp's own, by cp.async, three tiles ahead.
//   Scores: S^T[16 keys x 8 columns] = K Q^T.  Lane (g, q) = (lane / 4, lane % 4)
//   holds keys g and g + 8 and the words of D / 4 channels from q * D / 4 on: one
//   load, one group's parameters, and every pair of codes of a word (adjacent
//   channels, as stored) is one operand register.  The query is loaded in the
//   same order; the sum over channels does not depend on it.
//   Softmax: a running maximum per column, raised only when a score passes it by
//   more than 2^8 (a vote per tile; the sums are in fp32 and a weight is at most
//   2^8), weights rounded to 16 bits for the product with V (the tensor cores take
//   both operands in the layer's type), not for their sum.
//   Output: O^T[16 channels x 8 columns] += V^T P^T.  The weights reach their
//   operand layout by an 8 x 8 transpose between lanes.  Lane (g, q) holds keys 2q,
//   2q + 1, 2q + 8, 2q + 9 and the words of D / 8 channels from g * D / 8 on; a byte
//   permute of two keys' words puts the same channel of both keys side by side,
//   4 bits at a time, ready for the same conversion.  V's rows are placed in the
//   ring so that these loads fall on distinct banks.
//   The four warps' parts are merged in warp order; a sequence that fits one
//   split is finished there, others write their part, and the splits are merged in
//   a fixed order by the combine kernel (by the last CTA of a (sequence, KV head) to
//   finish, counted by tickets, it took as long).  A row's result depends on its own
//   sequence only.
//
// Measured (32/8 heads x 128, bf16): 4 rows over 100001 keys in 105.0 us, of which
// the split kernel 103, 4.88 TB/s, 0.72 of a plain copy's rate; DRAM reads equal the
// cache's bytes; 400 instructions a tile, issue slots 68% busy.  Four sequences of 4 rows
// (16 columns, three CTAs an SM) take 163 us, of 2 rows (8 columns) 119.  Leaving out the
// subtraction, the mask, the shift or the multiply-add of the conversion alone
// gained 6 to 14% each (before the shifts went, 7%): the conversion as a whole is
// what is left.  Two tiles an iteration, three or six ring stages, eight warps,
// three, five or six CTAs an SM, and KV heads side by side in the grid were no faster;
// splits merged in a cluster instead of by the combine kernel took 5.7 instead of 6.6 us
// for one row over 1025 keys, but 53 instead of 35 for 64 rows over up to 2000.
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "cp_ptx.cuh"
#include "cp_q4.cuh"
#include "cp_q4.h"
#include "cp_rows.cuh"

namespace cp {
namespace {

constexpr int kWarps = 4;
constexpr int kRing = 4;                      // stages of a warp's ring, one 16-key tile each

// N bytes of an asynchronous copy to shared memory; `on` false: zeros, nothing is read.
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool on) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(on ? 8 : 0) : "memory");
}

// The 8 x 8 matrix of 16-bit elements that a warp holds (lane: row lane / 4, columns 2 (lane % 4) and the next), transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A stage of a warp's ring.
template <int D>
struct Stage {
  static constexpr int kRow = D / 2, kPar = D / 8;  // bytes of a key's codes and parameters
  static constexpr int k = 0, v = 16 * kRow, kp = 32 * kRow, vp = kp + 16 * kPar, bytes = vp + 16 * kPar;
  // V's place of 16-byte chunk c of a key: four keys two apart are read at once, and must not share banks.
  static __device__ __forceinline__ int v_at(int key, int c) {
    if (D == 128) return ((key & 12) | ((key & 1) << 1) | ((key >> 1) & 1)) * kRow + (c ^ ((key >> 1) & 2)) * 16;
    return ((key & 8) | ((key & 1) << 2) | ((key >> 1) & 3)) * kRow + c * 16;
  }
};

// D (16x8, fp32) += A (16x16, row) * B (16x8, col), 16-bit inputs.
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// The rows that a slot of the split path's grid takes: kr of them, from place `first`
// of sequence s on, a sequence of n rows.
struct SlotRows {
  int s, first, n;
  int past, row0;  // keys before the slot's first row, and that row's place in the call
};

// (Out of line: a well-formed call never comes here.)
__device__ __noinline__ SlotRows slot_of_row(SeqRows rows, int row) {
  SlotRows r;
  r.s = row_seq(rows, row);
  r.first = row_place(rows, r.s, row);
  r.n = seq_rows(rows, r.s);
  return r;
}

// Slot i takes sequence i, if that has exactly kr rows.  by_row, for a ragged call with
// no more rows than sequences: it takes row i, whichever sequence that belongs to.  In a
// batch of single rows that is the same; where some sequences have no rows, so others
// may have several, every row still finds a slot (no tensor-core kernel follows).
__device__ __forceinline__ bool slot_rows(const Q4AttnArgs& a, int i, int kr, bool by_row, SlotRows& r) {
  r.s = i;
  r.first = 0;
  r.n = seq_rows(a.rows, i);
  if (!by_row) return r.n == kr;
  if (r.n != 1 || seq_row0(a.rows, i) != i) {
    if (i >= a.total_rows) return false;
    r = slot_of_row(a.rows, i);
    if (r.first < 0) return false;
  }
  return true;
}

// Whether the call's bounds allow the slot's sequence; its place, if so.
__device__ __forceinline__ bool slot_place(const Q4AttnArgs& a, SlotRows& r) {
  r.past = a.past[r.s];
  r.row0 = seq_row0(a.rows, r.s);
  if (r.past < 0 || (long long)r.past + r.n > a.max_ctx || r.row0 < 0 || r.row0 > a.total_rows - r.n) return false;
  r.past += r.first;
  r.row0 += r.first;
  return true;
}

// kOne: single rows, which see every key.
template <typename T, int D, int NF, bool kOne>
__global__ void __launch_bounds__(kWarps * 32, NF == 1 ? 4 : D == 64 ? 4 : 3) q4_split_kernel(const Q4AttnArgs a) {
  constexpr int NC = 8 * NF;     // (row, head) columns
  constexpr int KW = D / 32;     // score phase: words of a lane's channels
  constexpr int VW = D / 64;     // output phase
  using S = Stage<D>;
  // A warp's ring, whose place its output part takes at the end.
  constexpr int kWarpBytes = kRing * S::bytes > NC * D * 4 ? kRing * S::bytes : NC * D * 4;
  __shared__ __align__(128) uint8_t sWarp[kWarps][kWarpBytes];
  __shared__ float sM[kWarps][NC], sL[kWarps][NC];

  pdl_launch_dependents();
  const int split = blockIdx.x % a.max_splits, slot = blockIdx.x / a.max_splits, gk = blockIdx.y;
  pdl_wait();  // everything below reads what earlier kernels wrote
  if (a.commit_lens && blockIdx.x == 0 && blockIdx.y == 0)  // `past` is a copy: the lengths may advance at once
    for (int i = threadIdx.x; i < a.rows.num_seqs; i += kWarps * 32) a.commit_lens[i] += seq_rows(a.rows, i);
  const bool reports = a.status && split == 0 && gk == 0 && threadIdx.x == 0;
  if (reports && seq_rows(a.rows, slot) < 1) atomicOr(a.status, CP_DEV_BOUNDS);
  const int kr = kOne ? 1 : a.dec_rows;
  SlotRows mine;
  if (!slot_rows(a, slot, kr, kOne && a.by_row, mine)) return;
  if (!slot_place(a, mine)) {
    if (reports) atomicOr(a.status, CP_DEV_BOUNDS);
    return;
  }
  const int s = mine.s, past = mine.past, row0 = mine.row0;
  const int n = past + kr;  // keys, this call's rows among them
  const int split_keys = q4_split_keys(n), warp_keys = split_keys / kWarps;  // at most 256: a lane knows one tile's place
  if (split > (n - 1) / split_keys) return;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, q4 = lane & 3;
  const int G = a.group, ncols = kr * G, lg = 31 - __clz(G);  // G is a power of two
  const int kw = split * split_keys + warp * warp_keys;  // the warp's first key
  const int nkw = max(0, min(n - kw, warp_keys));        // its keys
  const int ntile = (nkw + 15) / 16;

  // First cache row of each of the warp's tiles (a page holds whole tiles): lane t has tile t's, -1 for a bad page.
  long long my_row = -1;
  if (lane < ntile) {
    my_row = cache_row(a.cache, a.hkv, s, gk, kw + 16 * lane, a.max_ctx);
    if (my_row < 0 && a.status) atomicOr(a.status, CP_DEV_BOUNDS);
  }

  const uint32_t bad_tiles = __ballot_sync(0xffffffffu, lane < ntile && my_row < 0);
  const uint32_t magic = q4_magic<T>();

  // ---- copies: lane's pieces of a tile
  const uint32_t ring = smem_u32(sWarp[warp]);
  constexpr int kChunks = D / 32;                    // 16-byte pieces of a key's codes
  constexpr int kIter = 16 * kChunks / 32;           // pieces of K (and of V) per lane
  const bool v_par = lane >= 16;                     // lanes 0-15 copy K's parameters, 16-31 V's
  const uint8_t* par = reinterpret_cast<const uint8_t*>(v_par ? a.v_params : a.k_params) + (lane & 15) * S::kPar;
  const uint8_t* kc = a.k_codes + lane * 16;
  const uint8_t* vc = a.v_codes + lane * 16;
  auto copy = [&](int t) {
    if (t < ntile) {
      const long long row = __shfl_sync(0xffffffffu, my_row, t);
      const int left = row < 0 ? 0 : nkw - 16 * t;   // keys of the tile
      const long long at = row < 0 ? 0 : row;
      const uint32_t st = ring + (t % kRing) * S::bytes;
      const uint8_t *k = kc + at * S::kRow, *v = vc + at * S::kRow;
      const uint32_t pd = st + (v_par ? S::vp : S::kp) + (lane & 15) * S::kPar;
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const int e = lane + 32 * i, key = e / kChunks, c = e % kChunks;
        cp_async<16>(st + S::k + e * 16, k + i * 512, key < left);
        cp_async<16>(st + S::v + S::v_at(key, c), v + i * 512, key < left);
      }
      cp_async<S::kPar>(pd, par + at * S::kPar, (lane & 15) < left);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int t = 0; t < kRing - 1; ++t) copy(t);

  // Query fragments: column 8f + g8 = (row, head), zero past the call's columns.
  uint4 qf[NF][KW];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int c = 8 * f + g8;
    const bool on = c < ncols;
    const uint4* q = reinterpret_cast<const uint4*>(
        static_cast<const T*>(a.q) + ((long long)(row0 + (on ? c >> lg : 0)) * a.hq + gk * G + (on ? c & (G - 1) : 0)) * D);
#pragma unroll
    for (int w = 0; w < KW; ++w) qf[f][w] = on ? q[q4 * KW + w] : make_uint4(0, 0, 0, 0);
  }
  float m[NF][2], l[NF][2], o[NF][VW * 4][4];
  int lim[NF][2];  // last key of the warp that column 8f + 2q4 + e sees
#pragma unroll
  for (int f = 0; f < NF; ++f) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[f][e] = -INFINITY;
      l[f][e] = 0.f;
      lim[f][e] = past + min((8 * f + 2 * q4 + e) >> lg, kr - 1) - kw;
    }
#pragma unroll
    for (int b = 0; b < VW * 4; ++b) o[f][b][0] = o[f][b][1] = o[f][b][2] = o[f][b][3] = 0.f;
  }

#pragma unroll 1
  for (int t = 0; t < ntile; ++t) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
    __syncwarp();  // every lane's copies of this tile have landed, and its reads of the stage that the next copy takes are done
    copy(t + kRing - 1);
    const uint8_t* st = sWarp[warp] + (t % kRing) * S::bytes;

    // ---- scores: keys g8 and g8 + 8, columns 8f + 2q4 and 8f + 2q4 + 1
    float c[NF][4];
#pragma unroll
    for (int f = 0; f < NF; ++f) c[f][0] = c[f][1] = c[f][2] = c[f][3] = 0.f;
    {
      uint32_t w[2][KW];
      uint32_t p[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint8_t* x = st + S::k + (g8 + 8 * r) * S::kRow + q4 * (4 * KW);
        if constexpr (KW == 4) *reinterpret_cast<uint4*>(w[r]) = *reinterpret_cast<const uint4*>(x);
        else *reinterpret_cast<uint2*>(w[r]) = *reinterpret_cast<const uint2*>(x);
        p[r] = *reinterpret_cast<const uint32_t*>(st + S::kp + (g8 + 8 * r) * S::kPar + q4 * KW / 4 * 4);
      }
      const Q4Scale p0 = q4_scale<T>(q4_scale2(p[0]), q4_low2(p[0])), p1 = q4_scale<T>(q4_scale2(p[1]), q4_low2(p[1]));
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        uint32_t x0[4], x1[4];
        q4_four<T>(w[0][i], p0, magic, x0);
        q4_four<T>(w[1][i], p1, magic, x1);
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          mma16816<T>(c[f], x0[0], x1[0], x0[1], x1[1], qf[f][i].x, qf[f][i].y);
          mma16816<T>(c[f], x0[2], x1[2], x0[3], x1[3], qf[f][i].z, qf[f][i].w);
        }
      }
    }
    const bool bad = (bad_tiles >> t) & 1;
    if (bad || 16 * t + 15 > past - kw) {  // a bad page, or keys that row 0 does not see
      // A V group of such a key that is not finite becomes zeros, so that 0 * NaN does not reach the rows that do
      // not see it; the rows that do become NaN by their sum.
      const int jv = 16 * t + (lane & 15);
      bool nan_v = false;
      if (!kOne && jv > past - kw && jv < nkw) {
        uint32_t* vp = reinterpret_cast<uint32_t*>(sWarp[warp] + (t % kRing) * S::bytes + S::vp + (lane & 15) * S::kPar);
#pragma unroll
        for (int i = 0; i < S::kPar / 4; ++i)
          if (q4_nonfinite<T>(vp[i])) nan_v = true;
      }
      const uint32_t nan_keys = __ballot_sync(0xffffffffu, nan_v);  // bits 0-15: the tile's keys
      if (nan_v) {
        uint32_t* vp = reinterpret_cast<uint32_t*>(sWarp[warp] + (t % kRing) * S::bytes + S::vp + (lane & 15) * S::kPar);
#pragma unroll
        for (int i = 0; i < S::kPar / 4; ++i)
          if (q4_nonfinite<T>(vp[i])) vp[i] = 0;
      }
      __syncwarp();
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool sees = 16 * t + g8 + 8 * (e >> 1) <= lim[f][e & 1];
          if (bad || !sees) c[f][e] = -INFINITY;
          else if ((nan_keys >> (g8 + 8 * (e >> 1))) & 1) l[f][e & 1] = __int_as_float(0x7fffffff);
        }
    }

    // ---- softmax: raise the maxima when a score passes one by more than 2^8
    bool grow = false;
    float mx[NF][2];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[f][e] = fmaxf(c[f][e], c[f][e + 2]) * a.scale_log2;
        grow = grow || mx[f][e] > m[f][e] + 8.f;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(mx[f][e], m[f][e]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          const float k = m[f][e] == -INFINITY ? 0.f : ex2_approx(m[f][e] - x);
          m[f][e] = x;
          l[f][e] *= k;
#pragma unroll
          for (int b = 0; b < VW * 4; ++b) {
            o[f][b][e] *= k;
            o[f][b][e + 2] *= k;
          }
        }
    }
    uint32_t b0[NF], b1[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const float z0 = m[f][0] == -INFINITY ? 0.f : -m[f][0], z1 = m[f][1] == -INFINITY ? 0.f : -m[f][1];
      const float p[4] = {ex2_approx(fmaf(c[f][0], a.scale_log2, z0)), ex2_approx(fmaf(c[f][1], a.scale_log2, z1)),
                          ex2_approx(fmaf(c[f][2], a.scale_log2, z0)), ex2_approx(fmaf(c[f][3], a.scale_log2, z1))};
      l[f][0] += p[0] + p[2];
      l[f][1] += p[1] + p[3];
      b0[f] = transpose8x8(Pack<T>::store(p));
      b1[f] = transpose8x8(Pack<T>::store(p + 2));
    }

    // ---- output: channels 8(VW g8 + m) + 2i (+1) for columns 8f + 2q4, 8f + 2q4 + 1
    {
      uint32_t w[4][VW], p[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int key = 2 * q4 + (r & 1) + 8 * (r >> 1);  // 2q, 2q + 1, 2q + 8, 2q + 9
        const uint8_t* x = st + S::v + S::v_at(key, g8 * VW / 4) + g8 * VW % 4 * 4;
        if constexpr (VW == 2) *reinterpret_cast<uint2*>(w[r]) = *reinterpret_cast<const uint2*>(x);
        else w[r][0] = *reinterpret_cast<const uint32_t*>(x);
        p[r] = *reinterpret_cast<const uint32_t*>(st + S::vp + key * S::kPar + g8 * VW / 4 * 4);
      }
      const Q4Scale p01 = q4_scale<T>(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[0], p[1], 0x7632));
      const Q4Scale p23 = q4_scale<T>(__byte_perm(p[2], p[3], 0x5410), __byte_perm(p[2], p[3], 0x7632));
#pragma unroll
      for (int k = 0; k < VW; ++k) {
        uint32_t e01[4], d01[4], e23[4], d23[4];  // even and odd channels of keys 0, 1 and of keys 2, 3
        q4_four<T>(__byte_perm(w[0][k], w[1][k], 0x5410), p01, magic, e01);
        q4_four<T>(__byte_perm(w[0][k], w[1][k], 0x7632), p01, magic, d01);
        q4_four<T>(__byte_perm(w[2][k], w[3][k], 0x5410), p23, magic, e23);
        q4_four<T>(__byte_perm(w[2][k], w[3][k], 0x7632), p23, magic, d23);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int f = 0; f < NF; ++f) mma16816<T>(o[f][k * 4 + i], e01[i], d01[i], e23[i], d23[i], b0[f], b1[f]);
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();  // the ring is read
  float(*ow)[D] = reinterpret_cast<float(*)[D]>(sWarp[warp]);
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int c0 = 8 * f + 2 * q4;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[f][e] += __shfl_xor_sync(0xffffffffu, l[f][e], d);
#pragma unroll
    for (int k = 0; k < VW; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d0 = 8 * (VW * g8 + k) + 2 * i;
        if (c0 < ncols) *reinterpret_cast<float2*>(&ow[c0][d0]) = make_float2(o[f][k * 4 + i][0], o[f][k * 4 + i][2]);
        if (c0 + 1 < ncols)
          *reinterpret_cast<float2*>(&ow[c0 + 1][d0]) = make_float2(o[f][k * 4 + i][1], o[f][k * 4 + i][3]);
      }
    if (g8 == 0) {
      sM[warp][c0] = m[f][0];
      sL[warp][c0] = l[f][0];
      sM[warp][c0 + 1] = m[f][1];
      sL[warp][c0 + 1] = l[f][1];
    }
  }
  __syncthreads();

  // ---- the split's part: the warps' parts merged in warp order
  const bool whole = n <= split_keys;
  for (int i = threadIdx.x; i < ncols * (D / 4); i += kWarps * 32) {
    const int c = i / (D / 4), d4 = i % (D / 4);
    float mc = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mc = fmaxf(mc, sM[w][c]);
    const float z = mc == -INFINITY ? 0.f : mc;
    float v[4] = {0.f, 0.f, 0.f, 0.f}, lsum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float k = ex2_approx(sM[w][c] - z);
      const float4 p = reinterpret_cast<const float4*>(sWarp[w])[c * (D / 4) + d4];
      v[0] = fmaf(k, p.x, v[0]);
      v[1] = fmaf(k, p.y, v[1]);
      v[2] = fmaf(k, p.z, v[2]);
      v[3] = fmaf(k, p.w, v[3]);
      lsum = fmaf(k, sL[w][c], lsum);
    }
    const long long row = row0 + (c >> lg), h = gk * G + (c & (G - 1));
    if (whole) {
      const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
      const float r[4] = {v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
      uint2 b;
      b.x = Pack<T>::store(r);
      b.y = Pack<T>::store(r + 2);
      *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (row * a.hq + h) * D + 4 * d4) = b;
    } else {
      const long long part = (((long long)slot * kr + (c >> lg)) * a.hq + h) * a.max_splits + split;
      *reinterpret_cast<float4*>(a.part_o + part * D + 4 * d4) = make_float4(v[0], v[1], v[2], v[3]);
      if (d4 == 0) {
        a.part_ml[part * 2] = mc;
        a.part_ml[part * 2 + 1] = lsum;
      }
    }
  }
}

// A row's splits are merged in eight slices -- split i in slice i % 8, a slice's
// splits in order -- and the slices in order, whatever the number of splits: the
// order is the row's own.  (With four slices, the merge of 98 splits took 6 us
// longer, that of 9 as long.)  A (row, head) belongs to kSlices groups of D / 4
// threads, a group a slice, a thread four channels.
constexpr int kSlices = 8;

// Four channels of a merge in progress: unnormalised output, maximum, sum.
struct Part {
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  // Adds a split: its maximum and sum, and its four channels.
  __device__ __forceinline__ void add(const float2& ml, const float4& p) {
    const float mn = fmaxf(m, ml.x), z = mn == -INFINITY ? 0.f : mn;
    const float k0 = ex2_approx(m - z), k1 = ex2_approx(ml.x - z);
    v[0] = v[0] * k0 + p.x * k1;
    v[1] = v[1] * k0 + p.y * k1;
    v[2] = v[2] * k0 + p.z * k1;
    v[3] = v[3] * k0 + p.w * k1;
    l = l * k0 + ml.y * k1;
    m = mn;
  }
  // Adds a slice to a sum of slices whose common maximum is z.
  __device__ __forceinline__ void add_scaled(const float4& p, float pm, float pl, float z) {
    const float k = ex2_approx(pm - z);
    v[0] = fmaf(k, p.x, v[0]);
    v[1] = fmaf(k, p.y, v[1]);
    v[2] = fmaf(k, p.z, v[2]);
    v[3] = fmaf(k, p.w, v[3]);
    l = fmaf(k, pl, l);
  }
  template <typename T>
  __device__ __forceinline__ void write(T* out) const {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float o[4] = {v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
    uint2 b;
    b.x = Pack<T>::store(o);
    b.y = Pack<T>::store(o + 2);
    *reinterpret_cast<uint2*>(out) = b;
  }
};

constexpr int kCombineThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kCombineThreads) q4_combine_kernel(const Q4AttnArgs a) {
  constexpr int C4 = D / 4, kPer = kCombineThreads / (C4 * kSlices);  // (row, head) pairs of a CTA
  __shared__ float4 so[kPer][kSlices][C4];
  __shared__ float sm[kPer][kSlices], sl[kPer][kSlices];
  pdl_launch_dependents();
  pdl_wait();
  const int kr = a.dec_rows;
  const int d4 = threadIdx.x % C4, slice = threadIdx.x / C4 % kSlices, pair = threadIdx.x / (C4 * kSlices);
  const long long id = (long long)blockIdx.x * kPer + pair;  // (slot, row, head)
  const long long sr = id / a.hq;
  const int h = (int)(id % a.hq), slot = (int)(sr / kr), r = (int)(sr % kr);
  SlotRows mine;
  bool on = slot < a.rows.num_seqs && slot_rows(a, slot, kr, a.by_row, mine);
  int row0 = 0, nsplit = 0;
  if (on) {
    on = slot_place(a, mine);
    row0 = mine.row0;
    if (on) nsplit = q4_splits(mine.past + kr);  // the last may hold keys of later rows only: a part of weight 0
    on = on && nsplit > 1;                       // one split: finished by the split kernel
  }
  Part part;
  if (on) {
    // Four splits' loads on their way together, written out: an unrolled loop came out with them one by one
    // (the merge of 98 splits 4 us longer).
    constexpr int kAhead = 4;
    for (int i0 = slice; i0 < nsplit; i0 += kAhead * kSlices) {
      float2 ml[kAhead];
      float4 p[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const long long at = id * a.max_splits + i0 + j * kSlices;
        if (i0 + j * kSlices >= nsplit) break;
        ml[j] = __ldcg(reinterpret_cast<const float2*>(a.part_ml + at * 2));
        p[j] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D + 4 * d4));
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (i0 + j * kSlices >= nsplit) break;
        part.add(ml[j], p[j]);
      }
    }
  }
  so[pair][slice][d4] = make_float4(part.v[0], part.v[1], part.v[2], part.v[3]);
  if (d4 == 0) {
    sm[pair][slice] = part.m;
    sl[pair][slice] = part.l;
  }
  __syncthreads();
  if (slice != 0 || !on) return;
  Part all;
#pragma unroll
  for (int i = 0; i < kSlices; ++i) all.m = fmaxf(all.m, sm[pair][i]);
  const float z = all.m == -INFINITY ? 0.f : all.m;
#pragma unroll
  for (int i = 0; i < kSlices; ++i) all.add_scaled(so[pair][i][d4], sm[pair][i], sl[pair][i], z);
  all.write(static_cast<T*>(a.out) + ((long long)(row0 + r) * a.hq + h) * D + 4 * d4);
}

template <typename T, int D>
cudaError_t launch_t(const Q4AttnArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)(a.rows.num_seqs * (long long)a.max_splits), a.hkv);
  const bool one = a.dec_rows == 1, wide = a.dec_rows * a.group > 8;
  const auto kernel = wide ? (one ? q4_split_kernel<T, D, 2, true> : q4_split_kernel<T, D, 2, false>)
                           : (one ? q4_split_kernel<T, D, 1, true> : q4_split_kernel<T, D, 1, false>);
  const cudaError_t e = launch_pdl(kernel, grid, dim3(kWarps * 32), 0, st, a);
  if (e != cudaSuccess || a.max_splits == 1) return e;
  constexpr int kPer = kCombineThreads / (D / 4 * kSlices);
  const long long pairs = (long long)a.rows.num_seqs * a.dec_rows * a.hq;
  return launch_pdl(q4_combine_kernel<T, D>, dim3((unsigned)((pairs + kPer - 1) / kPer)), dim3(kCombineThreads), 0, st,
                    a);
}

}  // namespace

cudaError_t launch_q4_decode(const Q4AttnArgs& a, int dtype, int d, cudaStream_t st) {
  if (dtype == CP_BF16) return d == 64 ? launch_t<__nv_bfloat16, 64>(a, st) : launch_t<__nv_bfloat16, 128>(a, st);
  return d == 64 ? launch_t<__half, 64>(a, st) : launch_t<__half, 128>(a, st);
}

}  // namespace cp
