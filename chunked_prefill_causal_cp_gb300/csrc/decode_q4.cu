// decode_q4.cu -- single rows and short chunks over a 4-bit cache, split along
// the keys.
//
// A decode row reads its sequence's cache once and does about 13 operations of
// attention per byte, so the path is bound by the bytes of the cache (160 per
// key and KV head at 128 channels) as long as the codes turn into matrix
// operands quickly enough.  One CTA takes 512 keys of a (sequence, KV head), four
// warps 128 each; the k rows of the sequence times the G heads of the group
// (k * G <= 16) ride in the columns of m16n8k16 products, so every row shares one
// read of the cache and one conversion of its codes.
//   Scores: S^T[16 keys x 8 columns] = K Q^T.  Lane (g, q) = (lane / 4, lane % 4)
//   holds keys g and g + 8 of a tile and the words of D / 4 channels from q * D / 4
//   on: one load, one group's parameters, and every pair of codes of a word
//   (adjacent channels, as stored) is one operand register.  The query is loaded
//   in the same order; the sum over channels does not depend on it.
//   Softmax: each warp's own maximum per column over its 128 keys, weights in 16
//   bits for the product with V (the tensor cores take both operands in the
//   layer's type), their sum in fp32.
//   Output: O^T[16 channels x 8 columns] += V^T P^T.  Lane (g, q) holds keys 2q,
//   2q + 1, 2q + 8, 2q + 9 and the words of D / 8 channels from g * D / 8 on; a byte
//   permute of two keys' words puts the same channel of both keys side by side,
//   4 bits at a time, ready for the same conversion.
//   The four warps' parts are merged in warp order; a sequence that fits one
//   split is finished there, others write their part for the combine kernel,
//   which merges the splits in order.  A row's result depends on its own
//   sequence only.
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
constexpr int kWarpKeys = kQ4Split / kWarps;  // 128
constexpr int kTiles = kWarpKeys / 16;
constexpr int kPStride = kWarpKeys + 8;       // 16-bit P row stride: conflict-free fragment reads
constexpr int kAhead = 4;                     // K tiles in flight per warp

__device__ __forceinline__ uint32_t ldg32(const void* p) {
  uint32_t r;
  asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(r) : "l"(p));
  return r;
}

// N consecutive words that are read once.
template <int N>
__device__ __forceinline__ void ldg_words(const void* p, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p));
  else if constexpr (N == 2)
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  else
    w[0] = ldg32(p);
}

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

// 16-bit bits of x in the low half.
template <typename T>
__device__ __forceinline__ uint16_t bits16(float x) {
  const float two[2] = {x, 0.f};
  return (uint16_t)Pack<T>::store(two);
}

template <typename T, int D, int NF>
__global__ void __launch_bounds__(kWarps * 32, NF == 1 ? 4 : 3) q4_split_kernel(const Q4AttnArgs a) {
  constexpr int NC = 8 * NF;     // (row, head) columns
  constexpr int KW = D / 32;     // score phase: words of a lane's channels
  constexpr int VW = D / 64;     // output phase
  constexpr int kRowBytes = D / 2, kRowGroups = D / 32;
  // A warp's output part takes the place of its own weights once it has read them.
  constexpr int kWarpWords = NC * (D > kPStride / 2 ? D : kPStride / 2);
  __shared__ __align__(16) float sWarp[kWarps][kWarpWords];
  __shared__ float sM[kWarps][NC], sL[kWarps][NC];

  pdl_launch_dependents();
  const int split = blockIdx.x % a.max_splits, s = blockIdx.x / a.max_splits, gk = blockIdx.y;
  pdl_wait();  // everything below reads what earlier kernels wrote
  if (a.commit_lens && blockIdx.x == 0 && blockIdx.y == 0)  // `past` is a copy: the lengths may advance at once
    for (int i = threadIdx.x; i < a.rows.num_seqs; i += kWarps * 32) a.commit_lens[i] += seq_rows(a.rows, i);
  const int rows = seq_rows(a.rows, s);
  const bool reports = a.status && split == 0 && gk == 0 && threadIdx.x == 0;
  if (reports && rows < 1) atomicOr(a.status, CP_DEV_BOUNDS);
  const int kr = a.dec_rows;
  if (rows != kr) return;
  const int past = a.past[s];
  const int row0 = seq_row0(a.rows, s);
  if (past < 0 || (long long)past + kr > a.max_ctx || row0 < 0 || row0 > a.total_rows - kr) {
    if (reports) atomicOr(a.status, CP_DEV_BOUNDS);
    return;
  }
  const int n = past + kr;  // keys, this call's rows among them
  const int k0 = split * kQ4Split;
  if (k0 >= n) return;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, q4 = lane & 3;
  const int G = a.group, ncols = kr * G;
  const int kw = warp * kWarpKeys;                                        // the warp's first key in the split
  const int nkw = max(0, min(min(n - k0, kQ4Split) - kw, kWarpKeys));     // its keys
  const int ntile = (nkw + 15) / 16;
  const bool paged = a.cache.kind == CP_CACHE_PAGED;
  const int ps = a.cache.page_size;

  // First cache row of each of the warp's tiles (a page holds whole tiles): lane t has tile t's, -1 for a bad page.
  long long my_row = -1;
  if (lane < ntile) {
    const int key = k0 + kw + 16 * lane;
    my_row = cache_row(a.cache, a.hkv, s, gk, key, a.max_ctx);
    if (my_row < 0 && a.status) atomicOr(a.status, CP_DEV_BOUNDS);
  }
  auto tile_row = [&](int t) -> long long { return __shfl_sync(0xffffffffu, my_row, t); };

  // Query fragments: column 8f + g8 = (row, head), zero past the call's columns.
  uint4 qf[NF][KW];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int c = 8 * f + g8;
    const bool on = c < ncols;
    const uint4* q = reinterpret_cast<const uint4*>(
        static_cast<const T*>(a.q) + ((long long)(row0 + (on ? c / G : 0)) * a.hq + gk * G + (on ? c % G : 0)) * D);
#pragma unroll
    for (int w = 0; w < KW; ++w) qf[f][w] = on ? q[q4 * KW + w] : make_uint4(0, 0, 0, 0);
  }

  // ---- scores: keys g8 and g8 + 8 of each tile, columns 8f + 2q4 and 8f + 2q4 + 1
  struct KTile {
    uint32_t w[2][KW], p[2];
  };
  auto load_k = [&](int t, KTile& x) {
    const long long row = tile_row(t);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (row >= 0 && 16 * t + g8 + 8 * r < nkw) {
        const long long at = row + g8 + 8 * r;
        ldg_words<KW>(a.k_codes + at * kRowBytes + q4 * (4 * KW), x.w[r]);
        x.p[r] = ldg32(a.k_params + at * kRowGroups + q4 * KW / 4);
      } else {
#pragma unroll
        for (int w = 0; w < KW; ++w) x.w[r][w] = 0;
        x.p[r] = 0;
      }
    }
  };
  float sc[kTiles][NF][4];
  float mx[NF][2];
  int lim[NF][2];  // last key of the split that column 8f + 2q4 + e sees; -1: none
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[f][e] = -INFINITY;
      const int c = 8 * f + 2 * q4 + e;
      lim[f][e] = c < ncols ? past + c / G - k0 - kw : -1;
    }
  KTile kb[kAhead];
#pragma unroll
  for (int t = 0; t < kAhead - 1; ++t) load_k(t, kb[t]);
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    if (t + kAhead - 1 < kTiles) load_k(t + kAhead - 1, kb[(t + kAhead - 1) % kAhead]);
    const KTile& x = kb[t % kAhead];
    const bool have = tile_row(t) >= 0;
    float c[NF][4];
#pragma unroll
    for (int f = 0; f < NF; ++f) c[f][0] = c[f][1] = c[f][2] = c[f][3] = 0.f;
    if (t < ntile) {  // the same for the whole warp
      const uint32_t s0 = q4_scale2(x.p[0]), m0 = q4_low2(x.p[0]), s1 = q4_scale2(x.p[1]), m1 = q4_low2(x.p[1]);
#pragma unroll
      for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t a0 = q4_pair<T>(x.w[0][w] >> (8 * u), s0, m0), a1 = q4_pair<T>(x.w[1][w] >> (8 * u), s1, m1);
          const uint32_t a2 = q4_pair<T>(x.w[0][w] >> (8 * u + 4), s0, m0);
          const uint32_t a3 = q4_pair<T>(x.w[1][w] >> (8 * u + 4), s1, m1);
#pragma unroll
          for (int f = 0; f < NF; ++f)
            mma16816<T>(c[f], a0, a1, a2, a3, u ? qf[f][w].z : qf[f][w].x, u ? qf[f][w].w : qf[f][w].y);
        }
    }
    const int j0 = 16 * t + g8, j1 = j0 + 8;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      sc[t][f][0] = have && j0 <= lim[f][0] && j0 < nkw ? c[f][0] * a.scale_log2 : -INFINITY;
      sc[t][f][1] = have && j0 <= lim[f][1] && j0 < nkw ? c[f][1] * a.scale_log2 : -INFINITY;
      sc[t][f][2] = have && j1 <= lim[f][0] && j1 < nkw ? c[f][2] * a.scale_log2 : -INFINITY;
      sc[t][f][3] = have && j1 <= lim[f][1] && j1 < nkw ? c[f][3] * a.scale_log2 : -INFINITY;
      mx[f][0] = fmaxf(mx[f][0], fmaxf(sc[t][f][0], sc[t][f][2]));
      mx[f][1] = fmaxf(mx[f][1], fmaxf(sc[t][f][1], sc[t][f][3]));
    }
  }

  // ---- values: the first tiles are in flight while the softmax runs
  struct VTile {
    uint32_t w[4][VW], p[4];
  };
  auto load_v = [&](int t, VTile& x) {
    const long long row = tile_row(t);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int kt = 2 * q4 + (r & 1) + 8 * (r >> 1);  // 2q, 2q + 1, 2q + 8, 2q + 9
      if (row >= 0 && 16 * t + kt < nkw) {
        const long long at = row + kt;
        ldg_words<VW>(a.v_codes + at * kRowBytes + g8 * (4 * VW), x.w[r]);
        x.p[r] = ldg32(a.v_params + at * kRowGroups + g8 * VW / 4);
      } else {
#pragma unroll
        for (int w = 0; w < VW; ++w) x.w[r][w] = 0;
        x.p[r] = 0;
      }
    }
  };
  constexpr int kAheadV = 3;
  VTile vb[kAheadV];
#pragma unroll
  for (int t = 0; t < kAheadV - 1; ++t) load_v(t, vb[t]);

  float l[NF][2];
  uint16_t(*pw)[kPStride] = reinterpret_cast<uint16_t(*)[kPStride]>(sWarp[warp]);
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    // A NaN score must not vanish: fmaxf drops it, the sum below keeps it.
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      mx[f][0] = fmaxf(mx[f][0], __shfl_xor_sync(0xffffffffu, mx[f][0], o));
      mx[f][1] = fmaxf(mx[f][1], __shfl_xor_sync(0xffffffffu, mx[f][1], o));
    }
    const float z0 = mx[f][0] == -INFINITY ? 0.f : mx[f][0], z1 = mx[f][1] == -INFINITY ? 0.f : mx[f][1];
    l[f][0] = l[f][1] = 0.f;
    const int c0 = 8 * f + 2 * q4;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const float p0 = ex2_approx(sc[t][f][0] - z0), p1 = ex2_approx(sc[t][f][1] - z1);
      const float p2 = ex2_approx(sc[t][f][2] - z0), p3 = ex2_approx(sc[t][f][3] - z1);
      l[f][0] += p0 + p2;
      l[f][1] += p1 + p3;
      pw[c0][16 * t + g8] = bits16<T>(p0);
      pw[c0 + 1][16 * t + g8] = bits16<T>(p1);
      pw[c0][16 * t + g8 + 8] = bits16<T>(p2);
      pw[c0 + 1][16 * t + g8 + 8] = bits16<T>(p3);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l[f][0] += __shfl_xor_sync(0xffffffffu, l[f][0], o);
      l[f][1] += __shfl_xor_sync(0xffffffffu, l[f][1], o);
    }
  }
  __syncwarp();

  // ---- output: channels 8(VW g8 + m) + 2i (+1) for columns 8f + 2q4, 8f + 2q4 + 1
  float o[NF][VW * 4][4];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int b = 0; b < VW * 4; ++b) o[f][b][0] = o[f][b][1] = o[f][b][2] = o[f][b][3] = 0.f;
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    if (t + kAheadV - 1 < kTiles) load_v(t + kAheadV - 1, vb[(t + kAheadV - 1) % kAheadV]);
    if (t < ntile) {
      const VTile& x = vb[t % kAheadV];
      const uint32_t s01 = __byte_perm(x.p[0], x.p[1], 0x5410), m01 = __byte_perm(x.p[0], x.p[1], 0x7632);
      const uint32_t s23 = __byte_perm(x.p[2], x.p[3], 0x5410), m23 = __byte_perm(x.p[2], x.p[3], 0x7632);
      uint32_t b[NF][2];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        b[f][0] = *reinterpret_cast<const uint32_t*>(&pw[8 * f + g8][16 * t + 2 * q4]);
        b[f][1] = *reinterpret_cast<const uint32_t*>(&pw[8 * f + g8][16 * t + 2 * q4 + 8]);
      }
#pragma unroll
      for (int m = 0; m < VW; ++m) {
        const uint32_t e01 = __byte_perm(x.w[0][m], x.w[1][m], 0x5410);  // even channels of keys 0, 1
        const uint32_t d01 = __byte_perm(x.w[0][m], x.w[1][m], 0x7632);  // odd channels
        const uint32_t e23 = __byte_perm(x.w[2][m], x.w[3][m], 0x5410);
        const uint32_t d23 = __byte_perm(x.w[2][m], x.w[3][m], 0x7632);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a0 = q4_pair<T>(e01 >> (4 * i), s01, m01), a1 = q4_pair<T>(d01 >> (4 * i), s01, m01);
          const uint32_t a2 = q4_pair<T>(e23 >> (4 * i), s23, m23), a3 = q4_pair<T>(d23 >> (4 * i), s23, m23);
#pragma unroll
          for (int f = 0; f < NF; ++f) mma16816<T>(o[f][m * 4 + i], a0, a1, a2, a3, b[f][0], b[f][1]);
        }
      }
    }
  }
  __syncwarp();  // the weights are read
  float(*ow)[D] = reinterpret_cast<float(*)[D]>(sWarp[warp]);
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int c0 = 8 * f + 2 * q4;
#pragma unroll
    for (int m = 0; m < VW; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d0 = 8 * (VW * g8 + m) + 2 * i;
        if (c0 < ncols)
          *reinterpret_cast<float2*>(&ow[c0][d0]) = make_float2(o[f][m * 4 + i][0], o[f][m * 4 + i][2]);
        if (c0 + 1 < ncols)
          *reinterpret_cast<float2*>(&ow[c0 + 1][d0]) = make_float2(o[f][m * 4 + i][1], o[f][m * 4 + i][3]);
      }
    if (g8 == 0) {
      sM[warp][c0] = mx[f][0];
      sL[warp][c0] = l[f][0];
      sM[warp][c0 + 1] = mx[f][1];
      sL[warp][c0 + 1] = l[f][1];
    }
  }
  __syncthreads();

  // ---- the split's part: the warps' parts merged in warp order
  const bool whole = a.max_splits == 1;
  for (int i = threadIdx.x; i < ncols * (D / 4); i += kWarps * 32) {
    const int c = i / (D / 4), d4 = i % (D / 4);
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sM[w][c]);
    const float z = m == -INFINITY ? 0.f : m;
    float v[4] = {0.f, 0.f, 0.f, 0.f}, lsum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float k = ex2_approx(sM[w][c] - z);
      const float4 p = *reinterpret_cast<const float4*>(&sWarp[w][c * D + 4 * d4]);
      v[0] = fmaf(k, p.x, v[0]);
      v[1] = fmaf(k, p.y, v[1]);
      v[2] = fmaf(k, p.z, v[2]);
      v[3] = fmaf(k, p.w, v[3]);
      lsum = fmaf(k, sL[w][c], lsum);
    }
    const long long row = row0 + c / G, h = gk * G + c % G;
    if (whole) {
      const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
      const float r[4] = {v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
      uint2 b;
      b.x = Pack<T>::store(r);
      b.y = Pack<T>::store(r + 2);
      *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (row * a.hq + h) * D + 4 * d4) = b;
    } else {
      const long long part = (((long long)s * kr + c / G) * a.hq + h) * a.max_splits + split;
      *reinterpret_cast<float4*>(a.part_o + part * D + 4 * d4) = make_float4(v[0], v[1], v[2], v[3]);
      if (d4 == 0) {
        a.part_ml[part * 2] = m;
        a.part_ml[part * 2 + 1] = lsum;
      }
    }
  }
}

// A row's splits merged: eight split slices times D / 4 four-channel columns, each slice in split order, then
// the slices in order.
template <typename T, int D>
__global__ void __launch_bounds__(8 * D / 4) q4_combine_kernel(const Q4AttnArgs a) {
  constexpr int C4 = D / 4;
  __shared__ float4 so[8][C4];
  __shared__ float sm[8], sl[8];
  pdl_launch_dependents();
  pdl_wait();
  const int kr = a.dec_rows;
  const int s = blockIdx.x / kr, r = blockIdx.x % kr, h = blockIdx.y;
  if (seq_rows(a.rows, s) != kr) return;
  const int past = a.past[s], row0 = seq_row0(a.rows, s);
  if (past < 0 || (long long)past + kr > a.max_ctx || row0 < 0 || row0 > a.total_rows - kr) return;
  const int nsplit = (past + r + kQ4Split) / kQ4Split;  // of the past + r + 1 keys the row sees
  const int slice = threadIdx.x / C4, d4 = threadIdx.x % C4;
  const long long base = (((long long)s * kr + r) * a.hq + h) * a.max_splits;
  float m = -INFINITY, l = 0.f;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = slice; i < nsplit; i += 8) {
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + (base + i) * 2);
    const float4 p = *reinterpret_cast<const float4*>(a.part_o + (base + i) * D + 4 * d4);
    const float mn = fmaxf(m, ml.x), z = mn == -INFINITY ? 0.f : mn;
    const float k0 = ex2_approx(m - z), k1 = ex2_approx(ml.x - z);
    v[0] = v[0] * k0 + p.x * k1;
    v[1] = v[1] * k0 + p.y * k1;
    v[2] = v[2] * k0 + p.z * k1;
    v[3] = v[3] * k0 + p.w * k1;
    l = l * k0 + ml.y * k1;
    m = mn;
  }
  so[slice][d4] = make_float4(v[0], v[1], v[2], v[3]);
  if (d4 == 0) {
    sm[slice] = m;
    sl[slice] = l;
  }
  __syncthreads();
  if (slice != 0) return;
  m = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, sm[i]);
  const float z = m == -INFINITY ? 0.f : m;
  l = v[0] = v[1] = v[2] = v[3] = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float k = ex2_approx(sm[i] - z);
    const float4 p = so[i][d4];
    v[0] = fmaf(k, p.x, v[0]);
    v[1] = fmaf(k, p.y, v[1]);
    v[2] = fmaf(k, p.z, v[2]);
    v[3] = fmaf(k, p.w, v[3]);
    l = fmaf(k, sl[i], l);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const float o[4] = {v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
  uint2 b;
  b.x = Pack<T>::store(o);
  b.y = Pack<T>::store(o + 2);
  *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + ((long long)(row0 + r) * a.hq + h) * D + 4 * d4) = b;
}

template <typename T, int D>
cudaError_t launch_t(const Q4AttnArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)(a.rows.num_seqs * (long long)a.max_splits), a.hkv);
  cudaError_t e = a.dec_rows * a.group <= 8 ? launch_pdl(q4_split_kernel<T, D, 1>, grid, dim3(kWarps * 32), 0, st, a)
                                            : launch_pdl(q4_split_kernel<T, D, 2>, grid, dim3(kWarps * 32), 0, st, a);
  if (e != cudaSuccess || a.max_splits == 1) return e;
  return launch_pdl(q4_combine_kernel<T, D>, dim3((unsigned)(a.rows.num_seqs * a.dec_rows), a.hq), dim3(8 * D / 4), 0,
                    st, a);
}

}  // namespace

cudaError_t launch_q4_decode(const Q4AttnArgs& a, int dtype, int d, cudaStream_t st) {
  if (dtype == CP_BF16) return d == 64 ? launch_t<__nv_bfloat16, 64>(a, st) : launch_t<__nv_bfloat16, 128>(a, st);
  return d == 64 ? launch_t<__half, 64>(a, st) : launch_t<__half, 128>(a, st);
}

}  // namespace cp
