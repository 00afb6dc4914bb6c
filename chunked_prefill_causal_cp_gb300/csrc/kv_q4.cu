// kv_q4.cu -- rows into and out of a cache held in 4 bits.
//
// Append: a group of 32 channels belongs to four lanes of 8 channels (16 bytes)
// each.  The group's smallest and largest value come from 16-bit minima of (x, -x)
// and two shuffles; the scale is their difference over 15, cut toward zero to the
// layer's type, so that no stored value leaves the group's range (a rounded-up
// scale could push the top code past the type's largest value); the codes are
// rounded against the scale as stored.  Every result is that of IEEE operations in
// fp32, so the stored bits follow from the inputs alone.  Each lane writes one
// 32-bit word of codes, the first lane of a group its scale and smallest value.
// Reading is the reverse: m + c s, rounded once.
// Both are bound by bytes in principle; the append is held back by its arithmetic
// (issue slots 73% busy).  8192 rows of 8 KV heads x 128 in bf16: the append 11.2 us
// and the read 7.5, 44 MB each (3.9 and 5.9 TB/s); one after the other 18.8 us.  With two
// IEEE divisions a channel pair the two took 26.6 us, with a division near halves only 22.9
// (half the warps meet an exact half).
// Two or four rows a thread were slower (23.9 and 26.5 us against 22.9).
#include <cmath>
#include <cstdint>
#include <type_traits>

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

// min and max of two pairs of 16-bit elements; a NaN stays.
template <typename T>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  typedef typename Two<T>::type V;
  const V r = __hmin2_nan(*reinterpret_cast<V*>(&a), *reinterpret_cast<V*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  typedef typename Two<T>::type V;
  const V r = __hmax2_nan(*reinterpret_cast<V*>(&a), *reinterpret_cast<V*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Codes of a lane's 8 channels (a word) and its group's params, from all four
// lanes of the group.
template <typename T>
__device__ __forceinline__ void quantize(const uint4& v, uint32_t& word, uint32_t& params) {
  // Smallest and largest in 16 bits, the largest as the smallest of the negated: (lo, -hi) in one word.
  const uint32_t mn = min2<T>(min2<T>(v.x, v.y), min2<T>(v.z, v.w));
  const uint32_t mx = max2<T>(max2<T>(v.x, v.y), max2<T>(v.z, v.w)) ^ 0x80008000u;
  uint32_t r = min2<T>(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) r = min2<T>(r, __shfl_xor_sync(0xffffffffu, r, o));
  float ends[2];
  Pack<T>::load(r, ends);
  const float lo = ends[0], range = __fadd_rn(-ends[1], -lo);
  // Quotients as IEEE division has them, in three operations: q0 = a y with y close
  // to 1 / b, r = a - q0 b (exact: q0 is within a few units of its last place),
  // q1 = q0 + r y.  Before its rounding q1 is within 2^-18 of a unit of a / b, and
  // with b of at most 11 significant bits a / b is never within 2^-12 of a unit
  // of a point halfway between two floats, so q1 rounds as a / b does.
  float step = __fmul_rn(range, 1.f / 15.f);
  step = __fmaf_rn(__fmaf_rn(-step, 15.f, range), 1.f / 15.f, step);
  if (!(range >= 0x1p-80f)) step = __fdiv_rn(range, 15.f);  // (a remainder could underflow)
  uint32_t sb = bits_rz<T>(step);
  if (!(range <= 3.402823466e38f)) sb = 0x7fffu;  // NaN in both types
  params = (r << 16) | sb;
  float s2[2];
  Pack<T>::load(sb, s2);
  const float s = s2[0];
  word = 0;
  if (!(s > 0.f)) return;
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
  const float2 nlo = make_float2(-lo, -lo), ns = make_float2(-s, -s), y2 = make_float2(y, y);
  const float2 up = make_float2(12582912.f, 12582912.f), down = make_float2(-12582912.f, -12582912.f);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float2 c[4];
  // From the type's smallest normal scale on, a quotient is at most 15 (1 + 2^-7), so rounds to 15 at most.
  if (s >= (std::is_same<T, __half>::value ? 0x1p-14f : 0x1p-80f) && s <= 0x1p100f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[2];
      Pack<T>::load(w[i], x);
      const float2 d = add2(make_float2(x[0], x[1]), nlo);
      float2 q = mul2(d, y2);
      q = fma2(fma2(q, ns, d), y2, q);
      c[i] = add2(add2(q, up), down);  // to a whole number, ties to even
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[2];
      Pack<T>::load(w[i], x);
      c[i].x = fminf(rintf(__fdiv_rn(__fadd_rn(x[0], -lo), s)), 15.f);
      c[i].y = fminf(rintf(__fdiv_rn(__fadd_rn(x[1], -lo), s)), 15.f);
    }
  }
  // Even and odd channels' codes as two whole numbers below 2^16.
  const float2 k16 = make_float2(16.f, 16.f);
  float2 h = fma2(c[3], k16, c[2]);
  h = fma2(h, k16, c[1]);
  h = fma2(h, k16, c[0]);
  h = add2(h, make_float2(8388608.f, 8388608.f));
  word = __byte_perm(__float_as_uint(h.x), __float_as_uint(h.y), 0x5410);
}


template <typename T, int D>
__global__ void __launch_bounds__(kQ4Threads) q4_append_kernel(const Q4Args a) {
  constexpr int V = D / 8;  // lanes of a row
  pdl_launch_dependents();
  pdl_wait();
  if (a.past_snapshot && blockIdx.x == 0)
    for (int s = threadIdx.x; s < a.rows.num_seqs; s += kQ4Threads) a.past_snapshot[s] = a.past[s];
  const uint32_t row = blockIdx.x * (uint32_t)(kQ4Threads / V) + threadIdx.x / V;  // at most INT32_MAX + a CTA's
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
  const int s = row_seq(a.rows, t), i = row_place(a.rows, s, t);
  if (i < 0) return;
  const long long dst = cache_row(a.cache, a.hkv, s, g, (long long)a.past[s] + i, a.max_ctx);
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
  uint32_t r[4];
  q4_four<T>(word, q4_scale<T>(q4_scale2(params), q4_low2(params)), magic, r);
  return make_uint4(r[0], r[1], r[2], r[3]);
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
  const int s = row_seq(a.rows, t), i = row_place(a.rows, s, t);
  if (i < 0) return;
  const long long src = cache_row(a.cache, a.hkv, s, g, (long long)a.past[s] + i, a.max_ctx);
  if (src < 0) {
    if (a.status && c == 0) atomicOr(a.status, CP_DEV_BOUNDS);
    return;
  }
  const uint32_t magic = q4_magic<T>();
  uint32_t kw = 0, kp = 0, vw = 0, vp = 0;  // every load before the first use
  if (a.k_out) {
    kw = reinterpret_cast<const uint32_t*>(a.k_codes)[src * V + c];
    kp = a.k_params[src * (V / 4) + c / 4];
  }
  if (a.v_out) {
    vw = reinterpret_cast<const uint32_t*>(a.v_codes)[src * V + c];
    vp = a.v_params[src * (V / 4) + c / 4];
  }
  if (a.k_out) static_cast<uint4*>(a.k_out)[(long long)row * V + c] = dequantize<T>(kw, kp, magic);
  if (a.v_out) static_cast<uint4*>(a.v_out)[(long long)row * V + c] = dequantize<T>(vw, vp, magic);
}

// `lanes`: threads of a row.
template <typename K>
cudaError_t launch_rows(K kernel, const Q4Args& a, int lanes, cudaStream_t st) {
  const long long rows = (long long)a.total_rows * a.hkv, per = kQ4Threads / lanes;
  if (rows == 0) return cudaSuccess;
  if (rows > INT32_MAX) return cudaErrorInvalidValue;
  const long long grid = (rows + per - 1) / per;
  return launch_pdl(kernel, dim3((unsigned)grid), dim3(kQ4Threads), 0, st, a);
}

}  // namespace

cudaError_t launch_q4_append(const Q4Args& a, int dtype, int d, cudaStream_t st) {
  if (dtype == CP_BF16)
    return d == 64 ? launch_rows(q4_append_kernel<__nv_bfloat16, 64>, a, 8, st)
                   : launch_rows(q4_append_kernel<__nv_bfloat16, 128>, a, 16, st);
  return d == 64 ? launch_rows(q4_append_kernel<__half, 64>, a, 8, st)
                 : launch_rows(q4_append_kernel<__half, 128>, a, 16, st);
}

cudaError_t launch_q4_read(const Q4Args& a, int dtype, int d, cudaStream_t st) {
  if (dtype == CP_BF16)
    return d == 64 ? launch_rows(q4_read_kernel<__nv_bfloat16, 64>, a, 8, st)
                   : launch_rows(q4_read_kernel<__nv_bfloat16, 128>, a, 16, st);
  return d == 64 ? launch_rows(q4_read_kernel<__half, 64>, a, 8, st)
                 : launch_rows(q4_read_kernel<__half, 128>, a, 16, st);
}

}  // namespace cp
