// attn_expanded.cu -- attention of prompt chunks over expanded keys and values of a
// latent cache, on the kernel of attn_pairs.cuh.
//
// Every head has keys and values of its own (and the rotated part of the keys in
// common), so a Q tile is 128 tokens of one head, and a score's product runs over
// nope_dim + rope_dim channels, the rotated part as 64 of which those past rope_dim
// are zeros.  The path is bound by the tensor cores.  Items are handed out with the
// most keys first, heads fastest.  8128 rows of 32 heads, 128 + 64 and 128 channels, after
// 8128 keys: 1.24 ms, 1.64 PFLOP/s, 0.86 of a large product's rate (call after call, under the
// power cap, 1.35 ms, 0.88 of what such a product sustains).
#include "attn_pairs.cuh"

namespace cp {
namespace {

using pairs::Item;

template <bool kLone_>  // items of one Q tile
struct ExpandedWork : pairs::WorkBase {
  static constexpr bool kPaged = false, kExpanded = true, kLone = kLone_;
  static constexpr int kItemRows = kLone ? 128 : 256;
  using Cursor = TurnCursor<ExpandedWork>;
  SeqRows keys;
  int total_keys;

  __device__ __forceinline__ int items(int r) const { return (r - 1) / kItemRows + 1; }
  __device__ __forceinline__ bool bounds(int s, int& r, int& row0, int& n, int& key0) const {
    r = seq_rows(rows, s);
    if (r < 1) return false;
    row0 = seq_row0(rows, s);
    n = keys.rows_uniform >= 0 ? keys.rows_uniform : keys.cu_rows[s + 1] - keys.cu_rows[s];
    key0 = keys.rows_uniform >= 0 ? s * keys.rows_uniform : keys.cu_rows[s];
    return row0 >= 0 && row0 <= total_rows - r && n >= 0 && key0 >= 0 && key0 <= total_keys - n;
  }
  __device__ __forceinline__ long long weight(int s, bool report) const {
    int r, row0, n, key0;
    if (!bounds(s, r, row0, n, key0)) {
      if (report && status && r >= 1) atomicOr(status, CP_DEV_BOUNDS);
      return 0;
    }
    return (long long)items(r) * hq;
  }
  __device__ __forceinline__ bool make(int s, long long idx, Item& x) const {
    int n;
    if (!bounds(s, x.rows, x.row0, n, x.key0)) return false;
    x.s = s;
    x.g = (int)(idx % hq);
    x.t0 = (items(x.rows) - 1 - (int)(idx / hq)) * kItemRows;
    x.q1 = !kLone && x.t0 + tok_tile < x.rows;
    x.past = n - x.rows;
    x.j_begin = 0;
    const int seen = x.past + min(x.rows, x.t0 + kItemRows);  // by the item's last row
    x.ntiles = seen > 0 ? (seen + pairs::kKeys - 1) / pairs::kKeys : 0;
    x.all = x.past + x.t0 + 1;
    x.whole = 1;
    x.part = 0;
    return true;
  }
};

// 3-D tensor of 16-bit elements with strides in elements, in 128-byte-swizzled boxes of 64 channels.
bool encode_strided(CUtensorMap* m, int dtype, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, int64_t s1, int64_t s2,
                    uint32_t b1, uint32_t b2) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {d0, d1, d2}, strides[2] = {(cuuint64_t)s1 * 2, (cuuint64_t)s2 * 2};
  const cuuint32_t box[3] = {64, b1, b2}, estr[3] = {1, 1, 1};
  return fn(m, dtype == CP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, bool kLone>
cudaError_t launch_t(const ExpandedArgs& a, int dtype, long long items, cudaStream_t st) {
  const int ctas = (int)std::min<long long>(items, kSms);
  ExpandedWork<kLone> wk;
  wk.hq = wk.hkv = a.heads;
  wk.group = 1;
  wk.tok_tile = 128;
  wk.scale_log2 = a.scale_log2;
  wk.rows = a.rows;
  wk.total_rows = a.total_rows;
  wk.out = a.out;
  wk.status = a.status;
  wk.part_o = wk.part_ml = nullptr;
  wk.page_size = wk.num_pages = wk.max_blocks = 0;
  wk.dn = a.dn;
  wk.block_table = wk.parents = nullptr;
  wk.keys = a.keys;
  if (a.keys.cu_rows) wk.keys.rows_uniform = -1;
  wk.total_keys = a.total_keys;
  pairs::Maps tm;
  const uint64_t H = a.heads, N = a.total_keys;
  if (!encode_3d(&tm.q, dtype, a.q, a.dn + a.r, H, a.total_rows, 64, 1, 128)) return cudaErrorInvalidValue;
  tm.k = tm.kr = tm.v = tm.q;  // without keys nothing is loaded
  if (N > 0) {
    if (!encode_strided(&tm.k, dtype, a.k_nope, a.dn, H, N, a.k_head, a.k_row, 1, 128) ||
        !encode_strided(&tm.v, dtype, a.v, a.dv, H, N, a.v_head, a.v_row, 1, 128) ||
        (a.r > 0 && !encode_strided(&tm.kr, dtype, a.k_rope, a.r, N, 1, a.r_row, a.r_row, 128, 1)))
      return cudaErrorInvalidValue;
  }
  const int nqb = a.dn / 64 + (a.r > 0 ? 1 : 0);
  if (a.dv == 64) {
    if (nqb == 1) return pairs::launch<T, 1, 1>(tm, wk, ctas, st);
    return nqb == 2 ? pairs::launch<T, 2, 1>(tm, wk, ctas, st) : pairs::launch<T, 3, 1>(tm, wk, ctas, st);
  }
  if (nqb == 1) return pairs::launch<T, 1, 2>(tm, wk, ctas, st);
  return nqb == 2 ? pairs::launch<T, 2, 2>(tm, wk, ctas, st) : pairs::launch<T, 3, 2>(tm, wk, ctas, st);
}

// Items of so many rows, at most.
long long items_of(const ExpandedArgs& a, int rows) {
  if (a.rows.rows_uniform > 0) return ((long long)(a.rows.rows_uniform - 1) / rows + 1) * a.rows.num_seqs * a.heads;
  return tiles_at_most(a.total_rows, a.rows.num_seqs, rows) * a.heads;
}

// Items are of one Q tile up to ten for each SM, or where few tiles have a second one beside them: the work is shared out
// more evenly, and both warpgroups have some (8 heads of 1000 rows after 4000: 76 us as pairs, 40; 20 heads of 2048 after
// 2000, 320 tiles: 88, 77; 1280 tiles: 474, 458; 512 prompts of 40 rows: 314, 272).  With more, pairs, which read K and V
// half as often (2048 tiles: 1.24 ms, lone 1.28).
template <typename T>
cudaError_t launch_type(const ExpandedArgs& a, int dtype, cudaStream_t st) {
  const long long lone = items_of(a, 128), pairs = items_of(a, 256);
  if (lone <= 10 * kSms || 4 * pairs > 3 * lone) return launch_t<T, true>(a, dtype, lone, st);
  return launch_t<T, false>(a, dtype, pairs, st);
}

}  // namespace

cudaError_t launch_expanded(const ExpandedArgs& a, int dtype, cudaStream_t st) {
  return dtype == CP_BF16 ? launch_type<__nv_bfloat16>(a, dtype, st) : launch_type<__half>(a, dtype, st);
}

}  // namespace cp
