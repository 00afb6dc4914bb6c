// cp_api_q4.cu -- the C ABI of the query/key preparation and of the 4-bit
// cache: argument checks and launches.  Every argument is checked before
// anything is enqueued.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "cp_host.h"
#include "cp_internal.h"
#include "cp_q4.h"

using namespace cp;

namespace {

// The rows of a call: cu_rows, or equal rows when that is NULL.
int rows_of(const int32_t* cu_rows, int32_t num_seqs, int32_t total_rows, SeqRows* out) {
  if (num_seqs <= 0 || total_rows < 0) return CP_ERR_INVALID_ARG;
  if (!cu_rows && total_rows % num_seqs != 0) return CP_ERR_INVALID_ARG;
  *out = SeqRows{num_seqs, cu_rows ? 0 : total_rows / num_seqs, cu_rows};
  return CP_OK;
}

// Most rows a sequence of the call can have (every listed one has at least one).
int64_t most_rows(const SeqRows& r, int32_t total_rows) {
  if (r.rows_uniform > 0) return r.rows_uniform;
  return total_rows >= r.num_seqs ? (int64_t)total_rows - r.num_seqs + 1 : total_rows;
}

// Whether every array of 32-bit numbers starts on its own boundary.
template <typename... P>
bool aligned4(const P*... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & 3u) == 0;
}

bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

// A row stride in elements: 0 = dense; else at least the row and whole 16-byte pieces.
int stride_of(int64_t given, int64_t dense, int es, long long* out) {
  if (given != 0 && (given < dense || given % (16 / es) != 0)) return CP_ERR_INVALID_ARG;
  if (given > (INT64_MAX >> 34)) return CP_ERR_UNSUPPORTED;  // stride * rows * bytes stays within 64 bits
  *out = given ? given : dense;
  return CP_OK;
}

// The checks that cp_qk_norm_rope and its append share; fills *a.
int rope_check(const cp_layer_desc* d, const cp_qk_prep* p, const void* q, int64_t q_stride, const void* k,
               int64_t k_stride, const void* q_weight, const void* k_weight, const float* inv_freq, void* q_out,
               RopeArgs* a, int32_t total_rows) {
  const int r = check_desc(d, false);
  if (r != CP_OK) return r;
  if (!p || !std::isfinite(p->eps) || p->eps < 0.f || (p->interleaved != 0 && p->interleaved != 1))
    return CP_ERR_INVALID_ARG;
  if (p->rot_dim < 0 || p->rot_dim > d->head_dim) return CP_ERR_INVALID_ARG;
  if (p->rot_dim % 16 != 0 || d->num_q_heads > 65535) return CP_ERR_UNSUPPORTED;
  const int es = esize_of(d->dtype);
  long long qs, ks;
  int e = stride_of(q_stride, (int64_t)d->num_q_heads * d->head_dim, es, &qs);
  if (e != CP_OK) return e;
  e = stride_of(k_stride, (int64_t)d->num_kv_heads * d->head_dim, es, &ks);
  if (e != CP_OK) return e;
  if ((q != nullptr) != (q_out != nullptr)) return CP_ERR_INVALID_ARG;
  if (total_rows > 0 && p->rot_dim > 0 && !inv_freq) return CP_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_weight) || !aligned16(k_weight) || !aligned16(q_out) ||
      !aligned4(inv_freq))
    return CP_ERR_INVALID_ARG;
  std::memset(a, 0, sizeof(*a));
  a->hq = q ? d->num_q_heads : 0;
  a->hkv = k ? d->num_kv_heads : 0;
  a->half = p->rot_dim / 2;
  a->interleaved = p->interleaved != 0;
  a->eps = p->eps;
  a->total_rows = total_rows;
  a->q = q;
  a->k = k;
  a->q_stride = qs;
  a->k_stride = ks;
  a->q_weight = q_weight;
  a->k_weight = k_weight;
  a->inv_freq = inv_freq;
  a->q_out = q_out;
  return CP_OK;
}

// Bytes that `rows` rows of `width` elements `stride` apart span.
int64_t span(int64_t rows, int64_t stride, int64_t width, int es) {
  return rows > 0 ? ((rows - 1) * stride + width) * es : 0;
}

// Where the call's rows may go: CONTIG, ROLLING and PAGED limits of a call with
// a host bound on positions.
int cache_check(const cp_layer_desc* d, const SeqRows& rows, int32_t total_rows, const int32_t* block_table,
                int32_t max_ctx) {
  if (max_ctx <= 0) return CP_ERR_INVALID_ARG;
  if (d->kind == CP_CACHE_PAGED) {
    if (!block_table) return CP_ERR_INVALID_ARG;
  } else if (rows.num_seqs > d->batch) {
    return CP_ERR_INVALID_ARG;
  }
  if (d->kind == CP_CACHE_ROLLING) {
    if (most_rows(rows, total_rows) > d->capacity) return CP_ERR_CAPACITY;
  } else if ((int64_t)max_ctx > layout_limit(d)) {
    return CP_ERR_CAPACITY;
  }
  return CP_OK;
}

// Layers and caches that may be held in 4 bits, and the cache's arrays.
int q4_check(const cp_layer_desc* d, const cp_q4_cache* c, int32_t total_rows) {
  const int r = check_desc(d, false);
  if (r != CP_OK) return r;
  if (d->dtype == CP_F32 || d->kind == CP_CACHE_ROLLING) return CP_ERR_UNSUPPORTED;
  if (total_rows > 0 && (int64_t)total_rows * d->num_kv_heads > INT32_MAX) return CP_ERR_UNSUPPORTED;
  if (!c || !c->k_codes || !c->v_codes || !c->k_params || !c->v_params) return CP_ERR_INVALID_ARG;
  if (!aligned16(c->k_codes) || !aligned16(c->v_codes) || !aligned16(c->k_params) || !aligned16(c->v_params))
    return CP_ERR_INVALID_ARG;
  return CP_OK;
}

Q4Args q4_args(const cp_layer_desc* d, const cp_q4_cache* c, const SeqRows& rows, int32_t total_rows,
               const int32_t* past, const int32_t* block_table, int32_t max_ctx, int32_t* dev_status) {
  Q4Args a;
  std::memset(&a, 0, sizeof(a));
  a.hkv = d->num_kv_heads;
  a.rows = rows;
  a.total_rows = total_rows;
  a.cache = make_cache(d, block_table);
  a.past = past;
  a.max_ctx = max_ctx;
  a.k_codes = static_cast<uint8_t*>(c->k_codes);
  a.v_codes = static_cast<uint8_t*>(c->v_codes);
  a.k_params = static_cast<uint32_t*>(c->k_params);
  a.v_params = static_cast<uint32_t*>(c->v_params);
  a.status = dev_status;
  return a;
}

// How an attention call over a 4-bit cache runs: the rows per sequence that take
// the split path, and where its workspace goes -- a copy of the lengths in
// whole 256-byte blocks (cp_mixed_step_q4), then the split path's parts when a
// context may need more than one split.
struct Q4Plan {
  int dec_rows;            // rows of a sequence on the split path
  bool split, tensor;      // which paths have sequences
  bool by_row;             // ragged, no more rows than sequences: the split path takes every row, as single rows
  int max_splits;
  int64_t pairs;           // pairs of Q tiles on the tensor-core path, at most
  int64_t parts;           // (row, head, split) parts, 0 when every context fits one split
  int64_t lens_bytes;
  double bytes;            // in floating point: absurd sizes must not wrap
};

Q4Plan q4_plan(const cp_layer_desc* d, bool ragged, int32_t num_seqs, int32_t total_rows, int32_t max_ctx) {
  Q4Plan p;
  const int64_t most = decode_max_rows(d->num_q_heads / d->num_kv_heads);
  const int64_t uniform = total_rows / num_seqs;
  p.dec_rows = !ragged && uniform >= 1 && uniform <= most ? (int)uniform : 1;
  p.split = ragged || uniform == p.dec_rows;
  // With a row in every sequence no more rows than sequences means one each; with a
  // sequence without rows others may have several, which the split path then takes.
  p.by_row = ragged && total_rows <= num_seqs;
  p.tensor = ragged ? !p.by_row : !p.split;
  p.max_splits = q4_max_splits(max_ctx);
  const int64_t ppt = 2 * (kTcBlockM / std::max(d->num_q_heads / d->num_kv_heads, 1));  // tokens of a pair
  p.pairs = !p.tensor ? 0 : ragged ? (total_rows + ppt - 1) / ppt + num_seqs : num_seqs * ((uniform + ppt - 1) / ppt);
  p.lens_bytes = ((int64_t)num_seqs * 4 + 255) / 256 * 256;
  const double parts = !p.split || p.max_splits == 1
                           ? 0.0
                           : (double)num_seqs * p.dec_rows * d->num_q_heads * p.max_splits;
  p.bytes = (double)p.lens_bytes + parts * (d->head_dim + 2) * sizeof(float);
  p.parts = p.bytes < 4e18 ? (int64_t)parts : 0;
  return p;
}

// The checks of cp_chunk_attn_q4 and cp_mixed_step_q4, but for the new rows.
int q4_attn_check(const cp_layer_desc* d, const void* q, const cp_q4_cache* c, const int32_t* seqlens_k,
                  const int32_t* block_table, const int32_t* cu_rows, int32_t num_seqs, int32_t total_rows,
                  int32_t max_ctx, const void* out, const void* workspace, size_t workspace_bytes, const int32_t* dev_status,
                  SeqRows* rows, Q4Plan* plan) {
  int r = q4_check(d, c, total_rows);
  if (r != CP_OK) return r;
  r = rows_of(cu_rows, num_seqs, total_rows, rows);
  if (r != CP_OK) return r;
  const int G = d->num_q_heads / d->num_kv_heads;
  if (G > 16 || (G & (G - 1))) return CP_ERR_UNSUPPORTED;
  if (total_rows == 0) return CP_OK;
  if (!q || !out || !seqlens_k || !aligned16(q) || !aligned16(out) ||
      !aligned4(seqlens_k, cu_rows, block_table, dev_status))
    return CP_ERR_INVALID_ARG;
  r = cache_check(d, *rows, total_rows, block_table, max_ctx);
  if (r != CP_OK) return r;
  if (max_ctx > INT32_MAX - 4096) return CP_ERR_UNSUPPORTED;  // key indices run past the context by up to a split
  *plan = q4_plan(d, cu_rows != nullptr, num_seqs, total_rows, max_ctx);
  if (d->num_q_heads > 65535 || (int64_t)num_seqs * plan->max_splits > INT32_MAX ||
      (double)num_seqs * plan->dec_rows * d->num_q_heads > INT32_MAX || 2 * plan->pairs > INT32_MAX)
    return CP_ERR_UNSUPPORTED;
  if (!workspace || !aligned16(workspace) || (double)workspace_bytes < plan->bytes) return CP_ERR_WORKSPACE;
  return CP_OK;
}

// The attention itself; `commit` (may be NULL): the lengths to advance, of which `past` is then a copy.
int q4_attention(const cp_layer_desc* d, const Q4Plan& p, const void* q, const cp_q4_cache* c, const int32_t* past,
                 int32_t* commit, const int32_t* block_table, const SeqRows& rows, int32_t total_rows, int32_t max_ctx,
                 void* out, void* workspace, int32_t* dev_status, cudaStream_t st) {
  Q4AttnArgs a;
  std::memset(&a, 0, sizeof(a));
  a.hq = d->num_q_heads;
  a.hkv = d->num_kv_heads;
  a.group = a.hq / a.hkv;
  a.scale_log2 = scale_log2(d);
  a.rows = rows;
  a.total_rows = total_rows;
  a.cache = make_cache(d, block_table);
  a.past = past;
  a.max_ctx = max_ctx;
  a.q = q;
  a.k_codes = static_cast<const uint8_t*>(c->k_codes);
  a.v_codes = static_cast<const uint8_t*>(c->v_codes);
  a.k_params = static_cast<const uint32_t*>(c->k_params);
  a.v_params = static_cast<const uint32_t*>(c->v_params);
  a.out = out;
  a.status = dev_status;
  a.dec_rows = p.dec_rows;
  a.by_row = p.by_row;
  a.min_rows = p.split ? p.dec_rows + 1 : 1;
  a.max_splits = p.max_splits;
  a.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.lens_bytes);
  a.part_ml = a.part_o + p.parts * d->head_dim;
  if (p.split) {
    a.commit_lens = commit;
    const int r = launch_result(launch_q4_decode(a, d->dtype, d->head_dim, st));
    if (r != CP_OK || !p.tensor) return r;
    a.commit_lens = nullptr;
  } else {
    a.commit_lens = commit;
  }
  return launch_result(launch_q4_tc(a, d->dtype, d->head_dim, (int)p.pairs, st));
}

}  // namespace

extern "C" {

int cp_qk_norm_rope(const cp_layer_desc* desc, const cp_qk_prep* prep, const void* q, int64_t q_row_stride,
                    const void* k, int64_t k_row_stride, const void* q_weight, const void* k_weight,
                    const float* inv_freq, const int32_t* positions, const int32_t* seqlens_k,
                    const int32_t* cu_rows, int32_t num_seqs, int32_t total_rows, void* q_out, void* k_out,
                    void* stream) {
  RopeArgs a;
  int r = rope_check(desc, prep, q, q_row_stride, k, k_row_stride, q_weight, k_weight, inv_freq, q_out, &a, total_rows);
  if (r != CP_OK) return r;
  if ((k != nullptr) != (k_out != nullptr) || !aligned16(k_out)) return CP_ERR_INVALID_ARG;
  if (!aligned4(positions, seqlens_k, cu_rows)) return CP_ERR_INVALID_ARG;
  if (positions) {
    if (total_rows < 0) return CP_ERR_INVALID_ARG;
    a.rows = SeqRows{1, total_rows, nullptr};
  } else {
    r = rows_of(cu_rows, num_seqs, total_rows, &a.rows);
    if (r != CP_OK) return r;
    if (total_rows > 0 && !seqlens_k) return CP_ERR_INVALID_ARG;
  }
  if (total_rows == 0 || (!q && !k)) return CP_OK;
  // Outputs may be their own dense inputs and overlap nothing else.
  const int es = esize_of(desc->dtype);
  const int64_t wq = (int64_t)desc->num_q_heads * desc->head_dim, wk = (int64_t)desc->num_kv_heads * desc->head_dim;
  const int64_t nq = q ? span(total_rows, a.q_stride, wq, es) : 0, nk = k ? span(total_rows, a.k_stride, wk, es) : 0;
  const int64_t oq = q ? span(total_rows, wq, wq, es) : 0, ok = k ? span(total_rows, wk, wk, es) : 0;
  if (q && overlap(q_out, oq, q, nq) && !(q_out == q && a.q_stride == wq)) return CP_ERR_INVALID_ARG;
  if (k && overlap(k_out, ok, k, nk) && !(k_out == k && a.k_stride == wk)) return CP_ERR_INVALID_ARG;
  if (q && k && (overlap(q_out, oq, k, nk) || overlap(k_out, ok, q, nq) || overlap(q_out, oq, k_out, ok)))
    return CP_ERR_INVALID_ARG;
  a.positions = positions;
  a.past = seqlens_k;
  a.k_out = k_out;
  return launch_result(launch_qk_rope(a, desc->dtype, desc->head_dim, static_cast<cudaStream_t>(stream)));
}

int cp_qk_norm_rope_append(const cp_layer_desc* desc, const cp_qk_prep* prep, const void* q, int64_t q_row_stride,
                           const void* k_new, int64_t k_row_stride, const void* v_new, int64_t v_row_stride,
                           const void* q_weight, const void* k_weight, const float* inv_freq,
                           const int32_t* positions, const int32_t* cu_rows, int32_t num_seqs, int32_t total_rows,
                           void* q_out, void* k_cache, void* v_cache, const int32_t* seqlens_k,
                           const int32_t* block_table, int32_t max_ctx, int32_t* dev_status, void* stream) {
  RopeArgs a;
  int r = rope_check(desc, prep, q, q_row_stride, k_new, k_row_stride, q_weight, k_weight, inv_freq, q_out, &a,
                     total_rows);
  if (r != CP_OK) return r;
  r = rows_of(cu_rows, num_seqs, total_rows, &a.rows);
  if (r != CP_OK) return r;
  const int es = esize_of(desc->dtype);
  const int64_t wq = (int64_t)desc->num_q_heads * desc->head_dim, wk = (int64_t)desc->num_kv_heads * desc->head_dim;
  r = stride_of(v_row_stride, wk, es, &a.v_stride);
  if (r != CP_OK) return r;
  if (total_rows == 0) return CP_OK;
  if (!q || !k_new || !v_new || !k_cache || !v_cache || !seqlens_k) return CP_ERR_INVALID_ARG;
  if (!aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned4(positions, seqlens_k, cu_rows, block_table, dev_status))
    return CP_ERR_INVALID_ARG;
  r = cache_check(desc, a.rows, total_rows, block_table, max_ctx);
  if (r != CP_OK) return r;
  const int64_t nq = span(total_rows, a.q_stride, wq, es), oq = span(total_rows, wq, wq, es);
  if (overlap(q_out, oq, q, nq) && !(q_out == q && a.q_stride == wq)) return CP_ERR_INVALID_ARG;
  if (overlap(q_out, oq, k_new, span(total_rows, a.k_stride, wk, es)) ||
      overlap(q_out, oq, v_new, span(total_rows, a.v_stride, wk, es)))
    return CP_ERR_INVALID_ARG;
  a.positions = positions;
  a.past = seqlens_k;
  a.v = v_new;
  a.cache = make_cache(desc, block_table);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.max_ctx = max_ctx;
  a.status = dev_status;
  return launch_result(launch_qk_rope(a, desc->dtype, desc->head_dim, static_cast<cudaStream_t>(stream)));
}

int cp_kv_append_q4(const cp_layer_desc* desc, const void* k_new, const void* v_new, const int32_t* cu_rows,
                    int32_t num_seqs, int32_t total_rows, const cp_q4_cache* cache, const int32_t* seqlens_k,
                    const int32_t* block_table, int32_t max_ctx, int32_t* dev_status, void* stream) {
  int r = q4_check(desc, cache, total_rows);
  if (r != CP_OK) return r;
  SeqRows rows;
  r = rows_of(cu_rows, num_seqs, total_rows, &rows);
  if (r != CP_OK || total_rows == 0) return r;
  if (!k_new || !v_new || !seqlens_k || !aligned16(k_new) || !aligned16(v_new) ||
      !aligned4(seqlens_k, cu_rows, block_table, dev_status))
    return CP_ERR_INVALID_ARG;
  r = cache_check(desc, rows, total_rows, block_table, max_ctx);
  if (r != CP_OK) return r;
  Q4Args a = q4_args(desc, cache, rows, total_rows, seqlens_k, block_table, max_ctx, dev_status);
  a.k_new = k_new;
  a.v_new = v_new;
  return launch_result(launch_q4_append(a, desc->dtype, desc->head_dim, static_cast<cudaStream_t>(stream)));
}

int cp_kv_read_q4(const cp_layer_desc* desc, const cp_q4_cache* cache, const int32_t* starts,
                  const int32_t* block_table, const int32_t* cu_rows, int32_t num_seqs, int32_t total_rows,
                  int32_t max_ctx, void* k_out, void* v_out, int32_t* dev_status, void* stream) {
  int r = q4_check(desc, cache, total_rows);
  if (r != CP_OK) return r;
  SeqRows rows;
  r = rows_of(cu_rows, num_seqs, total_rows, &rows);
  if (r != CP_OK || total_rows == 0) return r;
  if (!starts || !aligned16(k_out) || !aligned16(v_out) || !aligned4(starts, cu_rows, block_table, dev_status))
    return CP_ERR_INVALID_ARG;
  r = cache_check(desc, rows, total_rows, block_table, max_ctx);
  if (r != CP_OK) return r;
  if (!k_out && !v_out) return CP_OK;
  Q4Args a = q4_args(desc, cache, rows, total_rows, starts, block_table, max_ctx, dev_status);
  a.k_out = k_out;
  a.v_out = v_out;
  return launch_result(launch_q4_read(a, desc->dtype, desc->head_dim, static_cast<cudaStream_t>(stream)));
}

size_t cp_workspace_size_q4(const cp_layer_desc* desc, int32_t total_rows, int32_t max_ctx, int32_t num_seqs) {
  if (check_desc(desc, false) != CP_OK || total_rows <= 0 || max_ctx <= 0 || num_seqs <= 0) return 0;
  const int G = desc->num_q_heads / desc->num_kv_heads;
  if (G > 16 || (G & (G - 1)) || desc->dtype == CP_F32 || desc->kind == CP_CACHE_ROLLING) return 0;
  // The split path's rows of any call within these bounds: one of every sequence,
  // or up to 16 / G of each in a call of equal rows.
  const int64_t rows = std::max<int64_t>(num_seqs, std::min<int64_t>(total_rows, (int64_t)num_seqs * decode_max_rows(G)));
  const int splits = q4_max_splits(max_ctx);
  const double parts = splits > 1 ? (double)rows * desc->num_q_heads * splits : 0.0;
  const double bytes = (double)(((int64_t)num_seqs * 4 + 255) / 256 * 256) + parts * (desc->head_dim + 2) * sizeof(float);
  return bytes < 4e18 ? (size_t)bytes : SIZE_MAX;
}

int cp_chunk_attn_q4(const cp_layer_desc* desc, const void* q, const cp_q4_cache* cache, int32_t* seqlens_k,
                     const int32_t* block_table, const int32_t* cu_rows, int32_t num_seqs, int32_t total_rows,
                     int32_t max_ctx, void* out, void* workspace, size_t workspace_bytes, int32_t commit,
                     int32_t* dev_status, void* stream) {
  SeqRows rows;
  Q4Plan plan;
  int r = q4_attn_check(desc, q, cache, seqlens_k, block_table, cu_rows, num_seqs, total_rows, max_ctx, out, workspace,
                        workspace_bytes, dev_status, &rows, &plan);
  if (r != CP_OK || total_rows == 0) return r;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  r = q4_attention(desc, plan, q, cache, seqlens_k, nullptr, block_table, rows, total_rows, max_ctx, out, workspace,
                   dev_status, st);
  if (r != CP_OK || !commit) return r;
  return launch_result(launch_commit(seqlens_k, rows, rows.rows_uniform > 0 ? rows.rows_uniform : -1, nullptr, st));
}

int cp_mixed_step_q4(const cp_layer_desc* desc, const void* q, const void* k_new, const void* v_new,
                     const cp_q4_cache* cache, const int32_t* block_table, const int32_t* cu_rows,
                     int32_t* seqlens_k, int32_t num_seqs, int32_t total_rows, int32_t max_ctx, void* out,
                     void* workspace, size_t workspace_bytes, int32_t commit, int32_t* dev_status, void* stream) {
  SeqRows rows;
  Q4Plan plan;
  int r = q4_attn_check(desc, q, cache, seqlens_k, block_table, cu_rows, num_seqs, total_rows, max_ctx, out, workspace,
                        workspace_bytes, dev_status, &rows, &plan);
  if (r != CP_OK || total_rows == 0) return r;
  if (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new)) return CP_ERR_INVALID_ARG;
  // The append keeps a copy of the lengths for the attention to read, so that
  // the attention's first kernel may advance the lengths themselves.
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Q4Args ap = q4_args(desc, cache, rows, total_rows, seqlens_k, block_table, max_ctx, dev_status);
  ap.k_new = k_new;
  ap.v_new = v_new;
  ap.past_snapshot = static_cast<int*>(workspace);
  r = launch_result(launch_q4_append(ap, desc->dtype, desc->head_dim, st));
  if (r != CP_OK) return r;
  return q4_attention(desc, plan, q, cache, ap.past_snapshot, commit ? seqlens_k : nullptr, block_table, rows,
                      total_rows, max_ctx, out, workspace, dev_status, st);
}

}  // extern "C"
