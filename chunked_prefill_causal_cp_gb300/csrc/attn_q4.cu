// attn_q4.cu -- causal attention over a cache held in 4 bits.
//
// One warp per (query row, head): 32 keys at a time, a lane per key for the
// scores, then the lanes over the channels for the weighted sum of the values,
// with the running maximum and sum of an online softmax in fp32.
#include <cmath>
#include <cstdint>

#include "cp_q4.h"
#include "cp_ptx.cuh"
#include "cp_rows.cuh"

namespace cp {
namespace {

constexpr int kWarps = 4;

// The value a code stands for: m + c s rounded to the layer's type.
template <typename T>
__device__ __forceinline__ float code_value(uint32_t word, int i, uint32_t params) {
  float sm[2], x[2], y[2];
  Pack<T>::load(params, sm);
  x[0] = x[1] = fmaf((float)((word >> (4 * (i >> 1) + 16 * (i & 1))) & 15u), sm[0], sm[1]);
  Pack<T>::load(Pack<T>::store(x), y);
  return y[0];
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) q4_attn_rows_kernel(const Q4AttnArgs a) {
  constexpr int W = D / 8;  // words of a row
  __shared__ float sq[kWarps][D];
  pdl_launch_dependents();
  pdl_wait();
  if (a.commit_lens && blockIdx.x == 0)  // `past` is a copy: the lengths may advance at once
    for (int i = threadIdx.x; i < a.rows.num_seqs; i += kWarps * 32) a.commit_lens[i] += seq_rows(a.rows, i);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long id = (long long)blockIdx.x * kWarps + warp;
  const int t = (int)(id / a.hq), h = (int)(id % a.hq);
  if (t >= a.total_rows) return;
  const int s = row_seq(a.rows, t), g = h / a.group;
  const int rows = seq_rows(a.rows, s), past = a.past[s], r = t - seq_row0(a.rows, s);
  if (rows < a.min_rows) return;
  if (past < 0 || (long long)past + rows > a.max_ctx || r < 0 || r >= rows) {
    if (a.status && lane == 0) atomicOr(a.status, CP_DEV_BOUNDS);
    return;
  }
  const T* q = static_cast<const T*>(a.q) + ((long long)t * a.hq + h) * D;
  for (int i = lane; i < D; i += 32) sq[warp][i] = (float)q[i];
  __syncwarp();
  const int n = past + r + 1;
  float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  for (int j0 = 0; j0 < n; j0 += 32) {
    const int j = j0 + lane;
    const long long row = j < n ? cache_row(a.cache, a.hkv, s, g, j, a.max_ctx) : -1;
    if (j < n && row < 0 && a.status) atomicOr(a.status, CP_DEV_BOUNDS);
    float x = -INFINITY;
    if (row >= 0) {
      x = 0.f;
      for (int w = 0; w < W; ++w) {
        const uint32_t word = reinterpret_cast<const uint32_t*>(a.k_codes)[row * W + w];
        const uint32_t p = a.k_params[row * (W / 4) + w / 4];
#pragma unroll
        for (int i = 0; i < 8; ++i) x = fmaf(sq[warp][8 * w + i], code_value<T>(word, i, p), x);
      }
      x *= a.scale_log2;
    }
    float mx = x;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    const float mn = fmaxf(m, mx);
    const float shift = mn == -INFINITY ? 0.f : mn;
    const float alpha = ex2_approx(m - shift);
    const float pr = ex2_approx(x - shift);
    m = mn;
    l = l * alpha + pr;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= alpha;
    for (int k = 0; k < min(32, n - j0); ++k) {
      const long long rk = __shfl_sync(0xffffffffu, row, k);
      const float pk = __shfl_sync(0xffffffffu, pr, k);
      if (rk < 0) continue;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int c = lane + 32 * i;
        o[i] = fmaf(pk, code_value<T>(reinterpret_cast<const uint32_t*>(a.v_codes)[rk * W + c / 8], c % 8,
                                      a.v_params[rk * (W / 4) + i]),
                    o[i]);
      }
    }
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  T* out = static_cast<T*>(a.out) + ((long long)t * a.hq + h) * D;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) out[lane + 32 * i] = (T)(l > 0.f ? o[i] / l : 0.f);
}

template <typename T, int D>
cudaError_t launch_t(const Q4AttnArgs& a, cudaStream_t st) {
  const long long grid = ((long long)a.total_rows * a.hq + kWarps - 1) / kWarps;
  if (grid >= (1ll << 31)) return cudaErrorInvalidValue;
  return launch_pdl(q4_attn_rows_kernel<T, D>, dim3((unsigned)grid), dim3(kWarps * 32), 0, st, a);
}

}  // namespace

cudaError_t launch_q4_attn_rows(const Q4AttnArgs& a, int dtype, int d, cudaStream_t st) {
  if (a.total_rows == 0) return cudaSuccess;
  if (dtype == CP_BF16) return d == 64 ? launch_t<__nv_bfloat16, 64>(a, st) : launch_t<__nv_bfloat16, 128>(a, st);
  return d == 64 ? launch_t<__half, 64>(a, st) : launch_t<__half, 128>(a, st);
}

}  // namespace cp
