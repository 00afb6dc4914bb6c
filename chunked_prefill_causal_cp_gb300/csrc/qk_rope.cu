// qk_rope.cu -- norm of every query and key head and rotary position, in one
// pass over the rows, and optionally the keys and values into their cache.
//
//   y = x * rsqrt(mean(x^2) + eps) * w;  (a, b) -> (a cos u - b sin u, b cos u + a sin u)
//
// Each element is read once and written once and costs a few operations, so
// the pass is bound by bytes.  A head row of D channels belongs to LPR lanes,
// each holding two 16-byte chunks of it, chosen so that both members of every
// rotated pair are in one lane: with half-split pairs lane l < P holds chunks l
// and l + P (P = rot_dim / 2 channels in chunks) and the lanes from P on take the
// unrotated chunks two by two; with adjacent pairs lane l holds chunks 2l and
// 2l + 1.  Either way lane l < P rotates EPC pairs, of frequencies l * EPC on, and
// the others none, so no channel crosses lanes and the only shuffles are the
// sum of squares over LPR lanes.  A warp takes RPW = 32 / LPR head rows of one
// token at a time, the next ones' loads ahead of the work; the token's sines and
// cosines are computed once per warp, each row group taking EPC / RPW of the pairs.
// The arithmetic is in packed pairs of fp32.
// Measured (32/8 heads x 128, bf16, rows of a fused projection): 8192 rows in
// 30.1 us, 5.6 TB/s of the bytes read and written, 0.82 of a plain copy's rate (with
// 79 registers and fewer CTAs an SM 32.6 us, with 64 or fewer 29.9 to 35); one row
// 2.3 us, a launch's length.
//
// Angles: inv_freq is turned into a 64-bit fixed-point fraction of a turn per
// position (integer product of its significand with 2^66 / 2 pi), so
// position * step mod 2^64 is the angle mod one turn for any int32 position,
// with no reduction error to speak of.  The nearest quarter turn comes off in whole
// numbers too, and the top 32 bits of the rest, at most an eighth of a turn, go to
// sincospif as a float: the angle's error is below 2^-25 (half a unit of that float,
// 2^-25.4, and the cut bits), whatever the position.  (With the whole turn as one float it
// was 2^-23.3, and 8192 rows took 29.9 instead of 30.1 us.)
#include <algorithm>
#include <cstdint>

#include "cp_q4.h"
#include "cp_rows.cuh"

namespace cp {
namespace {

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

template <typename T, int D>
struct RopeShape {
  static constexpr int kPer16 = 16 / (int)sizeof(T);  // EPC: channels of a chunk
  static constexpr int kLanes = D / (2 * kPer16);     // LPR
  static constexpr int kRows = 32 / kLanes;           // RPW
  static constexpr int kShare = kPer16 / kRows;       // pairs whose angle a row group computes
  static_assert(kShare >= 1, "a warp's row groups share a lane's pairs evenly");
};

constexpr int kRopeThreads = 128;

// A warp takes per_warp blocks of kRows head rows of one token: all of them, or
// the blockIdx.y-th share.
template <typename T, int D, bool kAppend>
__global__ void __launch_bounds__(kRopeThreads, 6) qk_rope_kernel(const RopeArgs a, int per_warp) {
  using S = RopeShape<T, D>;
  constexpr int E = S::kPer16, L = S::kLanes, R = S::kRows;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long t_wide = ((long long)blockIdx.x * kRopeThreads + threadIdx.x) >> 5;
  if (t_wide >= a.total_rows) return;
  const int t = (int)t_wide;
  const int l = lane % L, rg = lane / L;
  const bool rot = l < a.pairs;

  // Chunks of this lane within a head row.
  int c0 = 2 * l, c1 = 2 * l + 1;
  if (!a.interleaved && rot) {
    c0 = l;
    c1 = l + a.pairs;
  }
  // Head rows in order: queries, keys, values (append).  The next block's loads are
  // on their way while a block is worked on, the first one's before the angles.
  const int heads = a.hq + a.hkv + (kAppend ? a.hkv : 0);
  const int h_begin = (int)blockIdx.y * per_warp * R, h_end = min(heads, h_begin + per_warp * R);
  uint4 n0 = make_uint4(0, 0, 0, 0), n1 = n0;
  auto load = [&](int h) {
    if (h >= h_end) return;
    const T* src;
    if (h < a.hq) src = static_cast<const T*>(a.q) + t * a.q_stride + (long long)h * D;
    else if (h < a.hq + a.hkv) src = static_cast<const T*>(a.k) + t * a.k_stride + (long long)(h - a.hq) * D;
    else src = static_cast<const T*>(a.v) + t * a.v_stride + (long long)(h - a.hq - a.hkv) * D;
    n0 = reinterpret_cast<const uint4*>(src)[c0];
    n1 = reinterpret_cast<const uint4*>(src)[c1];
  };
  load(h_begin + rg);

  long long pos = 0;  // position within the sequence, from the cached length
  int s = 0;
  bool older = false;  // a ring: newer rows of this call take the row's slot
  if (kAppend || !a.positions) {
    s = row_seq(a.rows, t);
    const int i = row_place(a.rows, s, t);
    if (i < 0) return;  // the whole warp has this token
    older = kAppend && a.cache.kind == CP_CACHE_ROLLING && seq_rows(a.rows, s) - i > a.cache.capacity;
    pos = (long long)a.past[s] + i;
  }
  const long long ang = a.positions ? a.positions[t] : pos;

  // Cosines and sines of the lane's pairs, two pairs to a register pair: (cos, cos')
  // and (sin, sin') of pairs 2i, 2i + 1.
  float2 cs[E / 2], sn[E / 2];
  if (a.pairs > 0) {
    float c[S::kShare], n[S::kShare];
#pragma unroll
    for (int i = 0; i < S::kShare; ++i) {
      c[i] = 1.f;
      n[i] = 0.f;
      if (rot) {
        sincos_turns((uint64_t)ang * turn_step(a.inv_freq[l * E + rg * S::kShare + i]), &n[i], &c[i]);
      }
    }
    auto of = [&](const float* x, int e) {
      return __shfl_sync(0xffffffffu, x[e % S::kShare], (e / S::kShare) * L + l);
    };
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      cs[i] = make_float2(of(c, 2 * i), of(c, 2 * i + 1));
      sn[i] = make_float2(of(n, 2 * i), of(n, 2 * i + 1));
    }
  }

  for (int h0 = h_begin; h0 < h_end; h0 += R) {
    const int h = h0 + rg;
    const bool on = h < h_end;
    const bool is_q = h < a.hq, is_v = kAppend && h >= a.hq + a.hkv;
    const int g = is_q ? h : is_v ? h - a.hq - a.hkv : h - a.hq;
    uint4 v0 = n0, v1 = n1;
    load(h + R);
    float2 x0[E / 2], x1[E / 2];  // the two chunks
    unpack16<T>(v0, reinterpret_cast<float*>(x0));
    unpack16<T>(v1, reinterpret_cast<float*>(x1));
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) s2 = fma2(x1[i], x1[i], fma2(x0[i], x0[i], s2));
    float ss = s2.x + s2.y;
#pragma unroll
    for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const T* wt = static_cast<const T*>(is_q ? a.q_weight : a.k_weight);
    if (!is_v) {
      if (wt) {
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        const float2 r2 = make_float2(r, r);
        float2 w0[E / 2], w1[E / 2];
        unpack16<T>(reinterpret_cast<const uint4*>(wt)[c0], reinterpret_cast<float*>(w0));
        unpack16<T>(reinterpret_cast<const uint4*>(wt)[c1], reinterpret_cast<float*>(w1));
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          x0[i] = mul2(mul2(x0[i], r2), w0[i]);
          x1[i] = mul2(mul2(x1[i], r2), w1[i]);
        }
      }
      if (rot) {
        if (a.interleaved) {
          // Pair i of a chunk is a register pair: (p, q) (c, c) + (q, p) (-s, s).
          auto turn = [](float2 x, float c, float s) {
            return fma2(make_float2(x.y, x.x), make_float2(-s, s), mul2(x, make_float2(c, c)));
          };
#pragma unroll
          for (int i = 0; i < E / 2; ++i) {
            const int j = i + E / 2;  // chunk 1's pairs follow chunk 0's
            x0[i] = turn(x0[i], i & 1 ? cs[i / 2].y : cs[i / 2].x, i & 1 ? sn[i / 2].y : sn[i / 2].x);
            x1[i] = turn(x1[i], j & 1 ? cs[j / 2].y : cs[j / 2].x, j & 1 ? sn[j / 2].y : sn[j / 2].x);
          }
        } else {
#pragma unroll
          for (int i = 0; i < E / 2; ++i) {
            const float2 p = x0[i], q = x1[i];
            x0[i] = fma2(q, make_float2(-sn[i].x, -sn[i].y), mul2(p, cs[i]));
            x1[i] = fma2(p, sn[i], mul2(q, cs[i]));
          }
        }
      }
      v0 = pack16<T>(reinterpret_cast<const float*>(x0));
      v1 = pack16<T>(reinterpret_cast<const float*>(x1));
    }
    if (!on) continue;
    T* dst;
    if (is_q) {
      dst = static_cast<T*>(a.q_out) + ((long long)t * a.hq + g) * D;
    } else if (!kAppend) {
      dst = static_cast<T*>(a.k_out) + ((long long)t * a.hkv + g) * D;
    } else {
      // (A ring holds a sequence's newest rows; the host's bound on them trusts that every sequence has one.)
      const long long row = older ? -1 : cache_row(a.cache, a.hkv, s, g, pos, a.max_ctx);
      if (row < 0) {
        if (a.status && l == 0) atomicOr(a.status, CP_DEV_BOUNDS);
        continue;
      }
      dst = static_cast<T*>(is_v ? a.v_cache : a.k_cache) + row * D;
    }
    reinterpret_cast<uint4*>(dst)[c0] = v0;
    reinterpret_cast<uint4*>(dst)[c1] = v1;
  }
}

template <typename T, int D>
cudaError_t launch_t(RopeArgs a, cudaStream_t st) {
  using S = RopeShape<T, D>;
  a.pairs = a.half / S::kPer16;
  const int heads = a.hq + a.hkv + (a.k_cache ? a.hkv : 0);
  const int blocks = (heads + S::kRows - 1) / S::kRows;
  // One warp per token does a token's angles once; with fewer tokens than warps
  // that fill the GPU (152 SMs x 32), a token's blocks are shared out over more.
  const int splits = (int)std::min<long long>(blocks, (152LL * 32 + a.total_rows - 1) / a.total_rows);
  const int per_warp = (blocks + splits - 1) / splits;
  const dim3 grid((unsigned)(((long long)a.total_rows * 32 + kRopeThreads - 1) / kRopeThreads),
                  (unsigned)((blocks + per_warp - 1) / per_warp));
  if (grid.y > 65535) return cudaErrorInvalidValue;
  if (a.k_cache) return launch_pdl(qk_rope_kernel<T, D, true>, grid, dim3(kRopeThreads), 0, st, a, per_warp);
  return launch_pdl(qk_rope_kernel<T, D, false>, grid, dim3(kRopeThreads), 0, st, a, per_warp);
}

}  // namespace

cudaError_t launch_qk_rope(const RopeArgs& a, int dtype, int d, cudaStream_t st) {
  if (a.total_rows == 0 || a.hq + a.hkv == 0) return cudaSuccess;
  if (dtype == CP_F32) return d == 64 ? launch_t<float, 64>(a, st) : launch_t<float, 128>(a, st);
  if (dtype == CP_BF16) return d == 64 ? launch_t<__nv_bfloat16, 64>(a, st) : launch_t<__nv_bfloat16, 128>(a, st);
  return d == 64 ? launch_t<__half, 64>(a, st) : launch_t<__half, 128>(a, st);
}

}  // namespace cp
