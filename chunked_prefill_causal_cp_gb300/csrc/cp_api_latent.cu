// cp_api_latent.cu -- the C ABI of latent caches and drafted trees: argument
// checks and launches.  Every argument is checked before anything is enqueued.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "cp_host.h"
#include "cp_internal.h"
#include "cp_latent.h"

using namespace cp;

namespace {

// The description of a latent cache; *out is its cache as a layer of one KV head.
int latent_check(const cp_latent_desc* d, cp_layer_desc* out) {
  if (!d) return CP_ERR_INVALID_ARG;
  *out = cp_layer_desc{d->dtype, d->batch, d->num_heads, 1, 128, d->kind, d->capacity, d->page_size, d->num_pages,
                       d->max_blocks, d->scale};
  const int r = check_desc(out, false);
  if (r != CP_OK) return r;
  if (d->dtype == CP_F32 || d->kind == CP_CACHE_ROLLING) return CP_ERR_UNSUPPORTED;
  if (d->latent_dim <= 0 || d->rope_dim < 0 || d->nope_dim <= 0 || d->v_dim <= 0) return CP_ERR_INVALID_ARG;
  if (d->latent_dim % 128 != 0 || d->latent_dim > 512 || d->rope_dim % 16 != 0 || d->rope_dim > 64)
    return CP_ERR_UNSUPPORTED;
  if ((d->nope_dim != 64 && d->nope_dim != 128) || (d->v_dim != 64 && d->v_dim != 128)) return CP_ERR_UNSUPPORTED;
  return CP_OK;
}

float latent_scale_log2(const cp_latent_desc* d) {
  const double sc = d->scale > 0.f ? (double)d->scale : 1.0 / std::sqrt((double)(d->nope_dim + d->rope_dim));
  return (float)(sc * 1.4426950408889634);  // log2(e)
}

// Row and head strides of [rows, heads, width] in elements, dense where 0.
int strides_of(int64_t row, int64_t head, int64_t heads, int64_t width, int es, long long* row_out, long long* head_out) {
  int r = stride_of(head, width, es, head_out);
  if (r != CP_OK) return r;
  if (*head_out > (INT64_MAX >> 34) / heads) return CP_ERR_UNSUPPORTED;
  return stride_of(row, *head_out * heads, es, row_out);
}

// The checks and the launch of attention of few rows that both kinds of cache share.
int rows_attention(const cp_layer_desc* d, bool latent, int dqk, int dv, float scale, const void* q, const void* k,
                   const void* v, const int32_t* seqlens_k, const int32_t* block_table, const int32_t* parents,
                   const int32_t* cu_rows, int32_t num_seqs, int32_t total_rows, int32_t max_ctx, void* out,
                   void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream, SeqRows* rows) {
  int r = rows_of(cu_rows, num_seqs, total_rows, rows);
  if (r != CP_OK || total_rows == 0) return r;
  if (!q || !k || !v || !out || !seqlens_k || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
      !aligned4(seqlens_k, block_table, parents, cu_rows, dev_status))
    return CP_ERR_INVALID_ARG;
  r = cache_check(d, *rows, total_rows, block_table, max_ctx);
  if (r != CP_OK) return r;
  if (max_ctx > INT32_MAX - 4096) return CP_ERR_UNSUPPORTED;  // key indices run past the context by up to a tile
  if (parents && rows->rows_uniform > CP_TREE_MAX) return CP_ERR_UNSUPPORTED;
  if (d->num_q_heads > 65535 || (int64_t)total_rows * d->num_q_heads > INT32_MAX / 4) return CP_ERR_UNSUPPORTED;
  const int64_t pairs = (int64_t)total_rows * d->num_q_heads;
  if (overlap(out, pairs * dv * 2, q, pairs * dqk * 2)) return CP_ERR_INVALID_ARG;
  const bool uniform = cu_rows == nullptr;
  const RowsPlan p = latent ? latent_plan(d->num_q_heads, dv, uniform, num_seqs, total_rows, max_ctx)
                            : tree_plan(d->num_q_heads, d->num_kv_heads, dv, uniform, num_seqs, total_rows, max_ctx);
  if (p.tiles > INT32_MAX / 64 || p.work > 1e15) return CP_ERR_UNSUPPORTED;  // sums times CTAs stay within 64 bits
  if (p.bytes > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < (size_t)p.bytes)) return CP_ERR_WORKSPACE;
  RowsAttnArgs a;
  std::memset(&a, 0, sizeof(a));
  a.hq = d->num_q_heads;
  a.hkv = d->num_kv_heads;
  a.group = a.hq / a.hkv;
  a.dqk = dqk;
  a.dv = dv;
  a.scale_log2 = scale;
  a.rows = *rows;
  a.total_rows = total_rows;
  a.cache = make_cache(d, block_table);
  a.past = seqlens_k;
  a.parents = parents;
  a.max_ctx = max_ctx;
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.status = dev_status;
  a.ctas = p.ctas;
  a.q_rows = p.q_rows;
  a.tok_tile = p.tok_tile;
  a.tiles = p.tiles;
  a.lone = p.lone;
  a.split = p.split;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = a.part_o + p.part_floats;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launch_result(latent ? launch_latent(a, d->dtype, st) : launch_tree(a, d->dtype, st));
}

size_t rows_workspace(const cp_layer_desc* d, bool latent, int dv, int32_t total_rows, int32_t max_ctx, int32_t num_seqs) {
  if (total_rows <= 0 || max_ctx <= 0 || num_seqs <= 0) return 0;
  return (size_t)(latent ? latent_plan(d->num_q_heads, dv, false, num_seqs, total_rows, max_ctx).bytes
                         : tree_plan(d->num_q_heads, d->num_kv_heads, dv, false, num_seqs, total_rows, max_ctx).bytes);
}

int tree_check(const cp_layer_desc* d) {
  const int r = check_desc(d, false);
  if (r != CP_OK) return r;
  if (d->dtype == CP_F32 || d->kind == CP_CACHE_ROLLING) return CP_ERR_UNSUPPORTED;
  return d->num_q_heads / d->num_kv_heads > 64 ? CP_ERR_UNSUPPORTED : CP_OK;
}

// The checks and the launch of both commits; row_bytes: of a (position, head) row.
int commit_paths(const cp_layer_desc* d, int row_bytes, void* k, void* v, const int32_t* path, const int32_t* counts,
                 int32_t* seqlens_k, const int32_t* block_table, int32_t num_seqs, int32_t max_path, int32_t max_ctx,
                 int32_t commit, int32_t* dev_status, void* stream) {
  if (num_seqs < 0 || max_path < 0) return CP_ERR_INVALID_ARG;
  if (max_path > CP_TREE_MAX) return CP_ERR_UNSUPPORTED;
  if (num_seqs == 0 || max_path == 0) return CP_OK;
  if (!path || !counts || !seqlens_k || !aligned16(k) || !aligned16(v) ||
      !aligned4(path, counts, seqlens_k, block_table, dev_status))
    return CP_ERR_INVALID_ARG;
  const int r = cache_check(d, SeqRows{num_seqs, 1, nullptr}, num_seqs, block_table, max_ctx);
  if (r != CP_OK) return r;
  CommitArgs a;
  std::memset(&a, 0, sizeof(a));
  a.hkv = d->num_kv_heads;
  a.row_bytes = row_bytes;
  a.cache = make_cache(d, block_table);
  a.path = path;
  a.counts = counts;
  a.lens = seqlens_k;
  a.num_seqs = num_seqs;
  a.max_path = max_path;
  a.max_ctx = max_ctx;
  a.commit = commit != 0;
  a.k = k;
  a.v = v;
  a.status = dev_status;
  return launch_result(launch_tree_commit(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int cp_latent_append(const cp_latent_desc* desc, const cp_qk_prep* prep, const void* latent, int64_t latent_row_stride,
                     const void* k_rope, int64_t k_row_stride, const void* weight, const float* inv_freq,
                     const int32_t* positions, const void* q_rope, int64_t q_row_stride, int64_t q_head_stride,
                     void* q_out, int64_t out_row_stride, int64_t out_head_stride, const int32_t* cu_rows,
                     int32_t num_seqs, int32_t total_rows, void* cache, const int32_t* seqlens_k,
                     const int32_t* block_table, int32_t max_ctx, int32_t* dev_status, void* stream) {
  cp_layer_desc d;
  int r = latent_check(desc, &d);
  if (r != CP_OK) return r;
  if (!prep || !std::isfinite(prep->eps) || prep->eps < 0.f || (prep->interleaved != 0 && prep->interleaved != 1))
    return CP_ERR_INVALID_ARG;
  if (prep->rot_dim < 0 || prep->rot_dim > desc->rope_dim) return CP_ERR_INVALID_ARG;
  if (prep->rot_dim % 16 != 0 || d.num_q_heads > 65535) return CP_ERR_UNSUPPORTED;
  LatentAppendArgs a;
  std::memset(&a, 0, sizeof(a));
  r = rows_of(cu_rows, num_seqs, total_rows, &a.rows);
  if (r != CP_OK) return r;
  const int R = desc->rope_dim;
  r = stride_of(latent_row_stride, desc->latent_dim, 2, &a.latent_stride);
  if (r != CP_OK) return r;
  r = stride_of(k_row_stride, R, 2, &a.k_stride);
  if (r != CP_OK) return r;
  r = strides_of(q_row_stride, q_head_stride, d.num_q_heads, R, 2, &a.q_row, &a.q_head);
  if (r != CP_OK) return r;
  r = strides_of(out_row_stride, out_head_stride, d.num_q_heads, R, 2, &a.out_row, &a.out_head);
  if (r != CP_OK) return r;
  if ((q_rope != nullptr) != (q_out != nullptr)) return CP_ERR_INVALID_ARG;
  if (q_rope && q_rope == q_out && (a.q_row != a.out_row || a.q_head != a.out_head)) return CP_ERR_INVALID_ARG;
  if (total_rows == 0) return CP_OK;
  if (!latent || !cache || !seqlens_k || (R > 0 && !k_rope) || (prep->rot_dim > 0 && !inv_freq)) return CP_ERR_INVALID_ARG;
  if (!aligned16(latent) || !aligned16(k_rope) || !aligned16(weight) || !aligned16(q_rope) || !aligned16(q_out) ||
      !aligned16(cache) || !aligned4(inv_freq, positions, cu_rows, seqlens_k, block_table, dev_status))
    return CP_ERR_INVALID_ARG;
  r = cache_check(&d, a.rows, total_rows, block_table, max_ctx);
  if (r != CP_OK) return r;
  a.heads = q_rope && R > 0 ? d.num_q_heads : 0;
  a.c = desc->latent_dim;
  a.r = R;
  a.pairs = prep->rot_dim / 16;
  a.interleaved = prep->interleaved != 0;
  a.eps = prep->eps;
  a.total_rows = total_rows;
  a.latent = latent;
  a.k_rope = k_rope;
  a.weight = weight;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.q = q_rope;
  a.q_out = q_out;
  a.cache = make_cache(&d, block_table);
  a.dst = cache;
  a.past = seqlens_k;
  a.max_ctx = max_ctx;
  a.status = dev_status;
  return launch_result(launch_latent_append(a, d.dtype, static_cast<cudaStream_t>(stream)));
}

int cp_latent_attn(const cp_latent_desc* desc, const void* q, const void* cache, int32_t* seqlens_k,
                   const int32_t* block_table, const int32_t* parents, const int32_t* cu_rows, int32_t num_seqs,
                   int32_t total_rows, int32_t max_ctx, void* out, void* workspace, size_t workspace_bytes,
                   int32_t commit, int32_t* dev_status, void* stream) {
  cp_layer_desc d;
  int r = latent_check(desc, &d);
  if (r != CP_OK) return r;
  if (parents && commit) return CP_ERR_INVALID_ARG;
  SeqRows rows;
  r = rows_attention(&d, true, desc->latent_dim + desc->rope_dim, desc->latent_dim, latent_scale_log2(desc), q, cache,
                     cache, seqlens_k, block_table, parents, cu_rows, num_seqs, total_rows, max_ctx, out, workspace,
                     workspace_bytes, dev_status, stream, &rows);
  if (r != CP_OK || total_rows == 0 || !commit) return r;
  return launch_result(launch_latent_commit(seqlens_k, rows, total_rows, max_ctx, static_cast<cudaStream_t>(stream)));
}

size_t cp_workspace_size_latent(const cp_latent_desc* desc, int32_t total_rows, int32_t max_ctx, int32_t num_seqs) {
  cp_layer_desc d;
  if (latent_check(desc, &d) != CP_OK) return 0;
  return rows_workspace(&d, true, desc->latent_dim, total_rows, max_ctx, num_seqs);
}

int cp_latent_chunk_attn(const cp_latent_desc* desc, const void* q, const void* k_nope, int64_t k_row_stride,
                         int64_t k_head_stride, const void* k_rope, int64_t k_rope_stride, const void* v,
                         int64_t v_row_stride, int64_t v_head_stride, const int32_t* cu_rows, const int32_t* cu_keys,
                         int32_t num_seqs, int32_t total_rows, int32_t total_keys, void* out, int32_t* dev_status,
                         void* stream) {
  cp_layer_desc d;
  int r = latent_check(desc, &d);
  if (r != CP_OK) return r;
  if ((cu_rows != nullptr) != (cu_keys != nullptr)) return CP_ERR_INVALID_ARG;
  ExpandedArgs a;
  std::memset(&a, 0, sizeof(a));
  r = rows_of(cu_rows, num_seqs, total_rows, &a.rows);
  if (r != CP_OK) return r;
  r = rows_of(cu_keys, num_seqs, total_keys, &a.keys);
  if (r != CP_OK) return r;
  const int H = d.num_q_heads, N = desc->nope_dim, R = desc->rope_dim, V = desc->v_dim;
  r = strides_of(k_row_stride, k_head_stride, H, N, 2, &a.k_row, &a.k_head);
  if (r != CP_OK) return r;
  r = strides_of(v_row_stride, v_head_stride, H, V, 2, &a.v_row, &a.v_head);
  if (r != CP_OK) return r;
  r = stride_of(k_rope_stride, R, 2, &a.r_row);
  if (r != CP_OK) return r;
  if (total_rows == 0) return CP_OK;
  if (!q || !out || (total_keys > 0 && (!k_nope || !v || (R > 0 && !k_rope)))) return CP_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_nope) || !aligned16(k_rope) || !aligned16(v) || !aligned16(out) ||
      !aligned4(cu_rows, cu_keys, dev_status))
    return CP_ERR_INVALID_ARG;
  if (H > 65535 || (int64_t)total_rows * H > INT32_MAX / 4 || total_keys > INT32_MAX - 4096) return CP_ERR_UNSUPPORTED;
  const int64_t pairs = (int64_t)total_rows * H;
  if (overlap(out, pairs * V * 2, q, pairs * (N + R) * 2)) return CP_ERR_INVALID_ARG;
  a.heads = H;
  a.dn = N;
  a.r = R;
  a.dv = V;
  a.scale_log2 = latent_scale_log2(desc);
  a.total_rows = total_rows;
  a.total_keys = total_keys;
  a.q = q;
  a.k_nope = k_nope;
  a.k_rope = k_rope;
  a.v = v;
  a.out = out;
  a.status = dev_status;
  return launch_result(launch_expanded(a, d.dtype, static_cast<cudaStream_t>(stream)));
}

int cp_tree_attn(const cp_layer_desc* desc, const void* q, const void* k_cache, const void* v_cache,
                 const int32_t* seqlens_k, const int32_t* block_table, const int32_t* parents, const int32_t* cu_rows,
                 int32_t num_seqs, int32_t total_rows, int32_t max_ctx, void* out, void* workspace,
                 size_t workspace_bytes, int32_t* dev_status, void* stream) {
  const int r = tree_check(desc);
  if (r != CP_OK) return r;
  if (total_rows > 0 && !parents) return CP_ERR_INVALID_ARG;
  SeqRows rows;
  return rows_attention(desc, false, desc->head_dim, desc->head_dim, scale_log2(desc), q, k_cache, v_cache, seqlens_k,
                        block_table, parents, cu_rows, num_seqs, total_rows, max_ctx, out, workspace, workspace_bytes,
                        dev_status, stream, &rows);
}

size_t cp_workspace_size_tree(const cp_layer_desc* desc, int32_t total_rows, int32_t max_ctx, int32_t num_seqs) {
  if (tree_check(desc) != CP_OK) return 0;
  return rows_workspace(desc, false, desc->head_dim, total_rows, max_ctx, num_seqs);
}

int cp_tree_commit(const cp_layer_desc* desc, void* k_cache, void* v_cache, const int32_t* path, const int32_t* counts,
                   int32_t* seqlens_k, const int32_t* block_table, int32_t num_seqs, int32_t max_path, int32_t max_ctx,
                   int32_t commit, int32_t* dev_status, void* stream) {
  const int r = check_desc(desc, false);
  if (r != CP_OK) return r;
  if (desc->kind == CP_CACHE_ROLLING) return CP_ERR_UNSUPPORTED;
  if (num_seqs > 0 && max_path > 0 && (!k_cache || !v_cache)) return CP_ERR_INVALID_ARG;
  return commit_paths(desc, desc->head_dim * esize_of(desc->dtype), k_cache, v_cache, path, counts, seqlens_k,
                      block_table, num_seqs, max_path, max_ctx, commit, dev_status, stream);
}

int cp_latent_tree_commit(const cp_latent_desc* desc, void* cache, const int32_t* path, const int32_t* counts,
                          int32_t* seqlens_k, const int32_t* block_table, int32_t num_seqs, int32_t max_path,
                          int32_t max_ctx, int32_t commit, int32_t* dev_status, void* stream) {
  cp_layer_desc d;
  const int r = latent_check(desc, &d);
  if (r != CP_OK) return r;
  if (num_seqs > 0 && max_path > 0 && !cache) return CP_ERR_INVALID_ARG;
  return commit_paths(&d, (desc->latent_dim + desc->rope_dim) * 2, cache, nullptr, path, counts, seqlens_k, block_table,
                      num_seqs, max_path, max_ctx, commit, dev_status, stream);
}

}  // extern "C"
