// kv_q4.cu -- rows into and out of a cache held in 4 bits.
//
// Append: a group of 32 channels belongs to four lanes of 8 channels (16 bytes)
// each.  Two shuffles give the group's smallest and largest value; the scale is
// their difference over 15, cut toward zero to the layer's type, so that no
// stored value leaves the group's range (a rounded-up scale could push the top
// code past the type's largest value); the codes are rounded against the scale
// as stored.  Every step is one IEEE operation in fp32, so the stored bits follow
// from the inputs alone.  Each lane writes one 32-bit word of codes, the first
// lane of a group its scale and smallest value.  Reading is the reverse: m + c s
// in fp32 (c s is exact) rounded once.  Both are bound by bytes.
#include <cstdint>

#include "cp_q4.h"
#include "cp_rows.cuh"

namespace cp {
namespace {

constexpr int kQ4Threads = 256;

// fp32 -> 16 bits, toward zero.
template <typename T>
__device__ __forceinline__ uint16_t bits_rz(float x);
template <>
__device__ __forceinline__ uint16_t bits_rz<__nv_bfloat16>(float x) {
  return __bfloat16_as_ushort(__float2bfloat16_rz(x));
}
template <>
__device__ __forceinline__ uint16_t bits_rz<__half>(float x) {
  return __half_as_ushort(__float2half_rz(x));
}

// Codes of a lane's 8 channels (a word) and its group's params, from all four
// lanes of the group.
template <typename T>
__device__ __forceinline__ void quantize(const uint4& v, uint32_t& word, uint32_t& params) {
  float x[8];
  unpack16<T>(v, x);
  float lo = x[0], hi = x[0], bad = 0.f;  // bad: NaN as soon as a value is not finite
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    bad += x[i] * 0.f;
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    bad += __shfl_xor_sync(0xffffffffu, bad, o);
  }
  const float range = __fadd_rn(hi, -lo);
  uint16_t sb = bits_rz<T>(__fdiv_rn(range, 15.f));
  if (!(range <= 3.402823466e38f) || bad != bad) sb = 0x7fffu;  // NaN in both types
  float m2[2] = {lo, lo};
  params = (Pack<T>::store(m2) & 0xffff0000u) | sb;
  float s2[2];
  Pack<T>::load(sb, s2);
  const float s = s2[0];
  word = 0;
  if (s > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = fminf(rintf(__fdiv_rn(__fadd_rn(x[i], -lo), s)), 15.f);
      word |= (uint32_t)c << (4 * (i >> 1) + 16 * (i & 1));
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kQ4Threads) q4_append_kernel(const Q4Args a) {
  constexpr int V = D / 8;  // lanes of a row
  pdl_launch_dependents();
  pdl_wait();
  if (a.past_snapshot && blockIdx.x == 0)
    for (int s = threadIdx.x; s < a.rows.num_seqs; s += kQ4Threads) a.past_snapshot[s] = a.past[s];
  const long long id = (long long)blockIdx.x * kQ4Threads + threadIdx.x;
  const long long row = id / V;
  const int c = (int)(id % V);
  const bool on = row < (long long)a.total_rows * a.hkv;
  uint4 kv = make_uint4(0, 0, 0, 0), vv = kv;
  if (on) {
    kv = static_cast<const uint4*>(a.k_new)[row * V + c];
    vv = static_cast<const uint4*>(a.v_new)[row * V + c];
  }
  uint32_t kw, kp, vw, vp;
  quantize<T>(kv, kw, kp);  // shuffles: every lane takes part
  quantize<T>(vv, vw, vp);
  if (!on) return;
  const int t = (int)(row / a.hkv), g = (int)(row % a.hkv);
  const int s = row_seq(a.rows, t);
  const long long dst = cache_row(a.cache, a.hkv, s, g, (long long)a.past[s] + t - seq_row0(a.rows, s), a.max_ctx);
  if (dst < 0) {
    if (a.status && c == 0) atomicOr(a.status, CP_DEV_BOUNDS);
    return;
  }
  reinterpret_cast<uint32_t*>(a.k_codes)[dst * V + c] = kw;
  reinterpret_cast<uint32_t*>(a.v_codes)[dst * V + c] = vw;
  if (c % 4 == 0) {
    a.k_params[dst * (V / 4) + c / 4] = kp;
    a.v_params[dst * (V / 4) + c / 4] = vp;
  }
}

template <typename T>
__device__ __forceinline__ uint4 dequantize(uint32_t word, uint32_t params) {
  float sm[2], x[8];
  Pack<T>::load(params, sm);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x[i] = fmaf((float)((word >> (4 * (i >> 1) + 16 * (i & 1))) & 15u), sm[0], sm[1]);
  return pack16<T>(x);
}

template <typename T, int D>
__global__ void __launch_bounds__(kQ4Threads) q4_read_kernel(const Q4Args a) {
  constexpr int V = D / 8;
  pdl_launch_dependents();
  pdl_wait();
  const long long id = (long long)blockIdx.x * kQ4Threads + threadIdx.x;
  const long long row = id / V;
  const int c = (int)(id % V);
  if (row >= (long long)a.total_rows * a.hkv) return;
  const int t = (int)(row / a.hkv), g = (int)(row % a.hkv);
  const int s = row_seq(a.rows, t);
  const long long src = cache_row(a.cache, a.hkv, s, g, (long long)a.past[s] + t - seq_row0(a.rows, s), a.max_ctx);
  if (src < 0) {
    if (a.status && c == 0) atomicOr(a.status, CP_DEV_BOUNDS);
    return;
  }
  if (a.k_out)
    static_cast<uint4*>(a.k_out)[row * V + c] =
        dequantize<T>(reinterpret_cast<const uint32_t*>(a.k_codes)[src * V + c], a.k_params[src * (V / 4) + c / 4]);
  if (a.v_out)
    static_cast<uint4*>(a.v_out)[row * V + c] =
        dequantize<T>(reinterpret_cast<const uint32_t*>(a.v_codes)[src * V + c], a.v_params[src * (V / 4) + c / 4]);
}

template <typename K>
cudaError_t launch_rows(K kernel, const Q4Args& a, int d, cudaStream_t st) {
  const long long threads = (long long)a.total_rows * a.hkv * (d / 8);
  if (threads == 0) return cudaSuccess;
  const long long grid = (threads + kQ4Threads - 1) / kQ4Threads;
  if (grid >= (1ll << 31)) return cudaErrorInvalidValue;
  return launch_pdl(kernel, dim3((unsigned)grid), dim3(kQ4Threads), 0, st, a);
}

}  // namespace

cudaError_t launch_q4_append(const Q4Args& a, int dtype, int d, cudaStream_t st) {
  if (dtype == CP_BF16)
    return d == 64 ? launch_rows(q4_append_kernel<__nv_bfloat16, 64>, a, d, st)
                   : launch_rows(q4_append_kernel<__nv_bfloat16, 128>, a, d, st);
  return d == 64 ? launch_rows(q4_append_kernel<__half, 64>, a, d, st)
                 : launch_rows(q4_append_kernel<__half, 128>, a, d, st);
}

cudaError_t launch_q4_read(const Q4Args& a, int dtype, int d, cudaStream_t st) {
  if (dtype == CP_BF16)
    return d == 64 ? launch_rows(q4_read_kernel<__nv_bfloat16, 64>, a, d, st)
                   : launch_rows(q4_read_kernel<__nv_bfloat16, 128>, a, d, st);
  return d == 64 ? launch_rows(q4_read_kernel<__half, 64>, a, d, st)
                 : launch_rows(q4_read_kernel<__half, 128>, a, d, st);
}

}  // namespace cp
