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
#include <cmath>
#include <cstdint>

#include "cp_q4.cuh"
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
  if (!(s > 0.f)) return;
  // The quotient's rounding decides a code only near a half: a product with the
  // reciprocal is within 2^-22 of it (two roundings of up to 2^4), so anything
  // further than 2^-20 from a half rounds alike, and the rest divides.  Adding
  // 1.5 * 2^23 rounds to a whole number, ties to even, in the low bits.
  const float inv = __fdiv_rn(1.f, s);
  float q[8], near = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = __fmul_rn(__fadd_rn(x[i], -lo), inv);
    const float r = __fadd_rn(__fadd_rn(q[i], 12582912.f), -12582912.f);
    near = fmaxf(near, fabsf(__fadd_rn(q[i], -r)));
  }
  if (!(near < 0.5f - 0x1p-20f) || !(inv < INFINITY)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(__fadd_rn(x[i], -lo), s);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t c = __float_as_uint(__fadd_rn(fminf(q[i], 15.f), 12582912.f)) & 15u;
    word |= c << (4 * (i >> 1) + 16 * (i & 1));
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kQ4Threads) q4_append_kernel(const Q4Args a) {
  constexpr int V = D / 8;  // lanes of a row
  pdl_launch_dependents();
  pdl_wait();
  if (a.past_snapshot && blockIdx.x == 0)
    for (int s = threadIdx.x; s < a.rows.num_seqs; s += kQ4Threads) a.past_snapshot[s] = a.past[s];
  const uint32_t row = blockIdx.x * (uint32_t)(kQ4Threads / V) + threadIdx.x / V;  // at most INT32_MAX + a block's
  const int c = threadIdx.x % V;
  const bool on = row < (uint32_t)a.total_rows * (uint32_t)a.hkv;
  uint4 kv = make_uint4(0, 0, 0, 0), vv = kv;
  if (on) {
    kv = static_cast<const uint4*>(a.k_new)[(long long)row * V + c];
    vv = static_cast<const uint4*>(a.v_new)[(long long)row * V + c];
  }
  uint32_t kw, kp, vw, vp;
  quantize<T>(kv, kw, kp);  // shuffles: every lane takes part
  quantize<T>(vv, vw, vp);
  if (!on) return;
  const int t = (int)(row / (uint32_t)a.hkv), g = (int)(row % (uint32_t)a.hkv);
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
__device__ __forceinline__ uint4 dequantize(uint32_t word, uint32_t params, uint32_t magic) {
  const uint32_t s2 = q4_scale2(params), m2 = q4_low2(params);
  return make_uint4(q4_pair<T>(word, s2, m2, magic), q4_pair<T>(word >> 4, s2, m2, magic),
                    q4_pair<T>(word >> 8, s2, m2, magic), q4_pair<T>(word >> 12, s2, m2, magic));
}

template <typename T, int D>
__global__ void __launch_bounds__(kQ4Threads) q4_read_kernel(const Q4Args a) {
  constexpr int V = D / 8;
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t row = blockIdx.x * (uint32_t)(kQ4Threads / V) + threadIdx.x / V;
  const int c = threadIdx.x % V;
  if (row >= (uint32_t)a.total_rows * (uint32_t)a.hkv) return;
  const int t = (int)(row / (uint32_t)a.hkv), g = (int)(row % (uint32_t)a.hkv);
  const int s = row_seq(a.rows, t);
  const long long src = cache_row(a.cache, a.hkv, s, g, (long long)a.past[s] + t - seq_row0(a.rows, s), a.max_ctx);
  if (src < 0) {
    if (a.status && c == 0) atomicOr(a.status, CP_DEV_BOUNDS);
    return;
  }
  if (a.k_out)
    static_cast<uint4*>(a.k_out)[(long long)row * V + c] =
        dequantize<T>(reinterpret_cast<const uint32_t*>(a.k_codes)[src * V + c], a.k_params[src * (V / 4) + c / 4], q4_magic<T>());
  if (a.v_out)
    static_cast<uint4*>(a.v_out)[(long long)row * V + c] =
        dequantize<T>(reinterpret_cast<const uint32_t*>(a.v_codes)[src * V + c], a.v_params[src * (V / 4) + c / 4], q4_magic<T>());
}

template <typename K>
cudaError_t launch_rows(K kernel, const Q4Args& a, int d, cudaStream_t st) {
  const long long rows = (long long)a.total_rows * a.hkv, per = kQ4Threads / (d / 8);
  if (rows == 0) return cudaSuccess;
  if (rows > INT32_MAX) return cudaErrorInvalidValue;
  const long long grid = (rows + per - 1) / per;
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
