// attn_expanded.cu -- attention of chunks over expanded keys and values.
//
// One warp a (row, head), lanes over channels, keys one by one with a running
// maximum and sum.
#include <cmath>
#include <cstdint>

#include "cp_latent.h"
#include "cp_ptx.cuh"
#include "cp_rows.cuh"

namespace cp {
namespace {

constexpr int kThreads = 128;
constexpr int kChunks = 3;  // 16-byte chunks of a row a lane holds: up to 768 channels

// A warp's running softmax; lane holds chunks lane, lane + 32, lane + 64 of a row.
template <typename T>
struct Walk {
  float q[kChunks][8], o[kChunks][8];
  float m = -INFINITY, l = 0.f;

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) q[i][e] = o[i][e] = 0.f;
  }
  __device__ __forceinline__ float dot(int i, const uint4& w) const {
    float x[8], d = 0.f;
    unpack16<T>(w, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) d = fmaf(q[i][e], x[e], d);
    return d;
  }
  __device__ __forceinline__ void key(float d, float scale, const T* v, int dv) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) d += __shfl_xor_sync(0xffffffffu, d, k);
    const float sc = d * scale, mn = fmaxf(m, sc), z = mn == -INFINITY ? 0.f : mn;
    const float k0 = ex2_approx(m - z), p = ex2_approx(sc - z);
    l = l * k0 + p;
    m = mn;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      if ((lane + 32 * i) * 8 < dv) {
        float x[8];
        unpack16<T>(reinterpret_cast<const uint4*>(v)[lane + 32 * i], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[i][e] = fmaf(p, x[e], o[i][e] * k0);
      }
  }
  __device__ __forceinline__ void write(T* out, int dv) {
    const int lane = threadIdx.x & 31;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      if ((lane + 32 * i) * 8 < dv) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[i][e] *= inv;
        reinterpret_cast<uint4*>(out)[lane + 32 * i] = pack16<T>(o[i]);
      }
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) expanded_kernel(const ExpandedArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long w = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
  if (w == 0)
    for (int s = lane; s < a.rows.num_seqs; s += 32)
      if (seq_rows(a.rows, s) < 1 && a.status) atomicOr(a.status, CP_DEV_BOUNDS);
  const int t = (int)(w / a.heads), h = (int)(w % a.heads);
  if (t >= a.total_rows) return;
  const int s = row_seq(a.rows, t), i = row_place(a.rows, s, t), r = seq_rows(a.rows, s), row0 = seq_row0(a.rows, s);
  if (i < 0) return;
  const int key0 = seq_row0(a.keys, s), n = seq_rows(a.keys, s);
  if (row0 < 0 || row0 > a.total_rows - r || n < 0 || key0 < 0 || key0 > a.total_keys - n) {
    if (a.status && lane == 0) atomicOr(a.status, CP_DEV_BOUNDS);
    return;
  }
  Walk<T> x;
  x.init();
  const int d = a.dn + a.r;
  const T* q = static_cast<const T*>(a.q) + ((long long)t * a.heads + h) * d;
  if (lane * 8 < d) unpack16<T>(reinterpret_cast<const uint4*>(q)[lane], x.q[0]);
  for (int j = 0; j <= n - r + i; ++j) {
    const T* k = static_cast<const T*>(a.k_nope) + (key0 + j) * a.k_row + h * a.k_head;
    if (lane * 8 >= a.dn) k = static_cast<const T*>(a.k_rope) + (key0 + j) * a.r_row - a.dn;
    const float p = lane * 8 < d ? x.dot(0, reinterpret_cast<const uint4*>(k)[lane]) : 0.f;
    x.key(p, a.scale_log2, static_cast<const T*>(a.v) + (key0 + j) * a.v_row + h * a.v_head, a.dv);
  }
  x.write(static_cast<T*>(a.out) + ((long long)t * a.heads + h) * a.dv, a.dv);
}

}  // namespace

cudaError_t launch_expanded(const ExpandedArgs& a, int dtype, cudaStream_t st) {
  const long long warps = (long long)a.total_rows * a.heads;
  const dim3 grid((unsigned)((warps + 3) / 4));
  if (dtype == CP_BF16) return launch_pdl(expanded_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, a);
  return launch_pdl(expanded_kernel<__half>, grid, dim3(kThreads), 0, st, a);
}

}  // namespace cp
