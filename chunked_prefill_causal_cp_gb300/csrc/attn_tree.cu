// attn_tree.cu -- attention of drafted trees over a K/V cache, on the kernel of
// attn_pairs.cuh.
//
// A tree's up to 128 nodes x G heads are one to a few (pairs of) Q tiles that read the
// whole context, and the CTAs share their tiles of keys out evenly (cp_latent.h); a unit
// of more than one leaves unnormalised fp32 parts in the workspace, which the combine
// kernel merges in order.  Each key's bytes are read once for a KV head's up to 256 rows:
// 24 trees of 61 nodes, 32/8 heads x 128, over 4000 to 24000 keys in pages of 16: 264 us,
// 5.3 TB/s of a copy's 6.8 and 1.27 PFLOP/s, between the cache's bytes and the chain of a
// tile; of 30 nodes 230 us, 6.0 TB/s; one tree of 16 nodes over 1024 keys 14 us, latency.
#include "attn_pairs.cuh"

namespace cp {
namespace {

using pairs::Item;

template <bool kPaged_, bool kLone_>  // units of one Q tile, or of two
struct TreeWork : pairs::WorkBase {
  static constexpr bool kPaged = kPaged_, kExpanded = false, kLone = kLone_;
  static constexpr int kQ = kLone ? 1 : 2;
  using Cursor = ShareCursor<TreeWork>;
  const int* past;
  int max_ctx, ctas;

  // A sequence within the call's bounds: its rows, positions before them, first row.
  __device__ __forceinline__ bool bounds(int s, int& r, int& p, int& row0) const {
    return seq_bounds(rows, past, total_rows, max_ctx, s, r, p, row0) && r <= CP_TREE_MAX;
  }
  __device__ __forceinline__ int q_units(int r) const { return (r - 1) / (kQ * tok_tile) + 1; }
  __device__ __forceinline__ int units(int s, bool report) const {
    int r, p, row0;
    if (bounds(s, r, p, row0)) return q_units(r) * hkv;
    if (report && status && r >= 1) atomicOr(status, CP_DEV_BOUNDS);
    return 0;
  }
  __device__ __forceinline__ int key_tiles(int s) const { return (past[s] + seq_rows(rows, s) - 1) / pairs::kKeys + 1; }
  // Unit u of a sequence: (KV head, Q tile or pair of them).
  __device__ __forceinline__ bool make(int s, int u, int k0, int n, Item& x) const {
    if (!bounds(s, x.rows, x.past, x.row0)) return false;
    const int np = q_units(x.rows);
    x.s = s;
    x.g = u / np;
    x.key0 = 0;
    x.t0 = (u - x.g * np) * kQ * tok_tile;
    x.q1 = !kLone && x.t0 + tok_tile < x.rows;
    x.j_begin = k0 * pairs::kKeys;
    const int seen = x.past + min(x.rows, x.t0 + kQ * tok_tile);  // by the item's last row
    x.ntiles = seen > x.j_begin ? min((seen - x.j_begin - 1) / pairs::kKeys + 1, n) : 0;
    x.all = x.past + (x.rows == 1 ? 1 : 0);
    return x.ntiles > 0;
  }
};

constexpr int kCombineRows = 8;
constexpr int kCombineCtas = 4 * kSms;

// Eight rows of a Q tile of a split sequence; lanes by row first, as the parts lie.
template <typename T, int NVB, typename Work>
__global__ void __launch_bounds__(kCombineRows * NVB * 16) tree_combine_kernel(const Work wk, const int groups,
                                                                                const bool by_share) {
  pdl_launch_dependents();
  pdl_look_ahead();
  const int group = blockIdx.x % groups, nth = blockIdx.x / groups;
  const MergedUnit<Work> x(wk, nth, by_share, wk.ctas);
  int r = 0, p = 0, row0 = 0;
  const bool found = x.s >= 0 && wk.bounds(x.s, r, p, row0);
  const int np = found ? wk.q_units(r) : 1, g = found ? x.unit / np : 0, t0 = found ? (x.unit - g * np) * Work::kQ * wk.tok_tile : 0;
  const int seen = found ? (p + min(r, t0 + Work::kQ * wk.tok_tile) - 1) / pairs::kKeys + 1 : 1;  // tiles of keys
  const UnitShares u(x.all, found ? x.first : 0, found ? x.n : 1, seen, wk.ctas);
  pdl_wait();  // on all paths: this kernel's end stands for the parts' kernel's
  if (!found || u.whole || (by_share && u.from != nth)) return;
  const int c4 = threadIdx.x / kCombineRows, per = wk.tok_tile * wk.group, rows = min(Work::kQ * wk.tok_tile, r - t0) * wk.group;
  for (int m = group * kCombineRows + threadIdx.x % kCombineRows; m < rows; m += groups * kCombineRows) {
    const int row = m < per ? m : 128 + m - per;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float mx = -INFINITY, l = 0.f;
    constexpr int kAhead = 8;
    for (int c0 = u.from; c0 <= u.to; c0 += kAhead) {
      float2 ml[kAhead];
      float4 x[kAhead];
      int n = 0;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (c0 + j > u.to) break;
        const int part = u.part(c0 + j);
        ml[j] = __ldcg(reinterpret_cast<const float2*>(wk.part_ml) + part * 256 + row);
        x[j] = __ldcg(reinterpret_cast<const float4*>(wk.part_o) + (part * (NVB * 16) + c4) * 256 + row);
        n = j + 1;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (j >= n) break;
        const float mn = fmaxf(mx, ml[j].x), z = mn == -INFINITY ? 0.f : mn;
        const float k0 = ex2_approx(mx - z), k1 = ex2_approx(ml[j].x - z);
        v.x = v.x * k0 + x[j].x * k1;
        v.y = v.y * k0 + x[j].y * k1;
        v.z = v.z * k0 + x[j].z * k1;
        v.w = v.w * k0 + x[j].w * k1;
        l = l * k0 + ml[j].y * k1;
        mx = mn;
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;  // a NaN stays
    const float o[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
    uint2 b;
    b.x = Pack<T>::store(o);
    b.y = Pack<T>::store(o + 2);
    const long long out = (long long)(row0 + t0 + m / wk.group) * wk.hq + g * wk.group + m % wk.group;
    *reinterpret_cast<uint2*>(static_cast<T*>(wk.out) + out * (NVB * 64) + 4 * c4) = b;
  }
}

template <typename T, int NB, bool kPaged, bool kLone>
cudaError_t launch_t(const RowsAttnArgs& a, int dtype, cudaStream_t st) {
  using Work = TreeWork<kPaged, kLone>;
  Work wk;
  wk.hq = a.hq;
  wk.hkv = a.hkv;
  wk.group = a.group;
  wk.tok_tile = a.tok_tile;
  wk.scale_log2 = a.scale_log2;
  wk.rows = a.rows;
  wk.total_rows = a.total_rows;
  wk.out = a.out;
  wk.status = a.status;
  wk.part_o = a.part_o;
  wk.part_ml = a.part_ml;
  wk.page_size = a.cache.page_size;
  wk.num_pages = a.cache.num_pages;
  wk.max_blocks = a.cache.max_blocks;
  wk.dn = a.dqk;
  wk.block_table = a.cache.block_table;
  wk.parents = a.parents;
  wk.past = a.past;
  wk.max_ctx = a.max_ctx;
  wk.ctas = a.ctas;
  pairs::Maps tm;
  const CacheView& c = a.cache;
  const uint64_t slots = kPaged ? c.page_size : c.capacity, planes = (uint64_t)(kPaged ? c.num_pages : a.rows.num_seqs) * a.hkv;
  const uint32_t box = kPaged ? c.page_size : pairs::kKeys;
  if (!encode_3d(&tm.q, dtype, a.q, a.dqk, a.hq, a.total_rows, 64, a.group, a.tok_tile) ||
      !encode_3d(&tm.k, dtype, a.k, a.dqk, slots, planes, 64, box, 1) ||
      !encode_3d(&tm.v, dtype, a.v, a.dv, slots, planes, 64, box, 1))
    return cudaErrorInvalidValue;
  tm.kr = tm.k;
  cudaError_t e = pairs::launch<T, NB, NB>(tm, wk, a.ctas, st);
  if (e != cudaSuccess || !a.split) return e;
  // A CTA takes several groups of rows of its unit, which it has to find but once (64 trees of 8 nodes 239 -> 203
  // us in all).
  const long long all = a.tiles * a.hkv, units = std::min<long long>(all, a.ctas);
  const int groups = (int)std::min<long long>(256 / kCombineRows, std::max<long long>(1, kCombineCtas / units));
  return launch_pdl(tree_combine_kernel<T, NB, Work>, dim3((unsigned)(units * groups)), dim3(kCombineRows * NB * 16), 0, st, wk,
                    groups, all > units);
}

template <typename T, int NB>
cudaError_t launch_dim(const RowsAttnArgs& a, int dtype, cudaStream_t st) {
  if (a.cache.kind == CP_CACHE_PAGED)
    return a.lone ? launch_t<T, NB, true, true>(a, dtype, st) : launch_t<T, NB, true, false>(a, dtype, st);
  return a.lone ? launch_t<T, NB, false, true>(a, dtype, st) : launch_t<T, NB, false, false>(a, dtype, st);
}

template <typename T>
cudaError_t launch_type(const RowsAttnArgs& a, int dtype, cudaStream_t st) {
  return a.dv == 64 ? launch_dim<T, 1>(a, dtype, st) : launch_dim<T, 2>(a, dtype, st);
}

}  // namespace

RowsPlan tree_plan(int hq, int hkv, int dv, bool uniform, long long num_seqs, long long total_rows, int max_ctx) {
  RowsPlan p{};
  const int group = hq / hkv, key_tiles = (max_ctx - 1) / pairs::kKeys + 1;
  p.tok_tile = 128 / group;
  const long long rows = std::min<long long>(uniform ? total_rows / num_seqs : total_rows, CP_TREE_MAX);
  const auto units = [&](int tokens) {  // of a KV head, at most
    const long long most = num_seqs * ((rows - 1) / tokens + 1);
    return uniform ? most : std::min(tiles_at_most(total_rows, num_seqs, tokens), most);
  };
  // Lone Q tiles where few have a second one beside them: both warpgroups have keys then (24 trees of 16 nodes, 32/8
  // heads x 64, over 4000 to 12000 keys: 101 -> 86 us; 64 of 8, x 128, over 2000 to 6000: 186 -> 180); else pairs, which
  // read the keys half as often.
  const long long lone = units(p.tok_tile), pairs = units(2 * p.tok_tile);
  p.lone = 4 * pairs > 3 * lone;
  p.tiles = p.lone ? lone : pairs;
  p.work = (double)p.tiles * hkv * (kStart + key_tiles);
  p.ctas = (int)std::min<double>(p.work, kSms);
  p.split = key_tiles > 1;
  p.part_floats = p.split ? 2LL * kSms * 256 * dv : 0;
  p.bytes = p.split ? 2LL * kSms * 256 * (dv + 2) * (long long)sizeof(float) : 0;
  return p;
}

cudaError_t launch_tree(const RowsAttnArgs& a, int dtype, cudaStream_t st) {
  return dtype == CP_BF16 ? launch_type<__nv_bfloat16>(a, dtype, st) : launch_type<__half>(a, dtype, st);
}

}  // namespace cp
