// cp_latent.h -- argument blocks and launchers of the latent cache's calls and
// of drafted trees.  Every pointer is a device pointer.
#pragma once

#include "cp_internal.h"

namespace cp {

// Norm and rotation of rows into a latent cache, rotation of the queries' part
// (cp_latent_append).
struct LatentAppendArgs {
  int heads, c, r;         // H (0: no queries), channels of the latent and of the rotated part
  int pairs;               // 16-byte chunks that hold the first channels of the rotated pairs (rot_dim / 16)
  bool interleaved;
  float eps;
  SeqRows rows;
  int total_rows;
  const void* latent;
  const void* k_rope;
  long long latent_stride, k_stride;         // elements from a row to the next
  const void* weight;      // [C] or nullptr
  const float* inv_freq;
  const int* positions;    // [total_rows] or nullptr: past + row within the sequence
  const void* q;
  void* q_out;
  long long q_row, q_head, out_row, out_head;  // elements
  CacheView cache;
  void* dst;               // the cache
  const int* past;
  int max_ctx;
  int* status;
};

// Splits of a sequence of n positions whose (row, head) pairs make nt tiles, over a latent
// cache: few keys a split for a short context, where the wait for one CTA's walk is what
// counts, more for a long one, whose parts cost less then, and no more than kRowsItems
// (tile, split) items.  By the sequence's own sizes alone, so a row's result never
// depends on what shares the launch.
constexpr int kRowsItems = 304;  // twice the SMs
__host__ __device__ inline int rows_split_base(int n) { return n <= 2048 ? 128 : n <= 8192 ? 256 : n <= 16384 ? 512 : 1024; }
__host__ __device__ inline int rows_splits(int n, int nt) {
  const int cap = kRowsItems / nt, k = (n - 1) / rows_split_base(n) + 1;
  return cap <= 1 ? 1 : k < cap ? k : cap;
}
// Keys of each split: whole tiles of 64.
__host__ __device__ inline int rows_split_keys(int n, int splits) { return ((n - 1) / splits + 64) & ~63; }
// Most splits of a sequence of up to ctx positions and nt tiles.
inline int rows_max_splits(int ctx, int nt) {
  int m = rows_splits(ctx, nt);
  const int steps[3] = {2048, 8192, 16384};
  for (int s : steps)
    if (ctx > s && rows_splits(s, nt) > m) m = rows_splits(s, nt);
  return m;
}

// The same for a drafted tree over a K/V cache, nt pairs of Q tiles times KV heads, in
// whole tiles of 128 keys.
constexpr int kTreeItems = 152;  // (pair, KV head, split) items of a split sequence, at most: the SMs
__host__ __device__ inline int tree_split_base(int n) { return n <= 2048 ? 128 : n <= 4096 ? 256 : n <= 8192 ? 512 : n <= 16384 ? 1024 : 2048; }
__host__ __device__ inline int tree_splits(int n, int nt) {
  const int cap = kTreeItems / nt, k = (n - 1) / tree_split_base(n) + 1;
  return cap <= 1 ? 1 : k < cap ? k : cap;
}
__host__ __device__ inline int tree_split_keys(int n, int splits) { return ((n - 1) / splits + 128) & ~127; }
inline int tree_max_splits(int ctx, int nt) {
  int m = tree_splits(ctx, nt);
  const int steps[4] = {2048, 4096, 8192, 16384};
  for (int s : steps)
    if (ctx > s && tree_splits(s, nt) > m) m = tree_splits(s, nt);
  return m;
}

// Attention of few rows over a long cache (cp_latent_attn, cp_tree_attn).  A
// latent cache is one KV head whose group is all heads and whose values are its
// keys' first dv channels.
struct RowsAttnArgs {
  int hq, hkv, group;
  int dqk, dv;             // channels of a score's product, of an output row
  float scale_log2;        // softmax scale * log2(e)
  SeqRows rows;
  int total_rows;
  CacheView cache;
  const int* past;
  const int* parents;      // [total_rows] or nullptr: rows follow one another
  int max_ctx;
  const void* q;           // [total_rows, hq, dqk]
  const void* k;           // the cache (latent: both)
  const void* v;
  void* out;               // [total_rows, hq, dv]
  int* status;
  // A latent cache's (cp_latent_attn):
  int q_rows;              // pairs of a tile that the call can have, at most
  int tiles_bound;         // tiles of the call, at most
  int max_splits;          // of any sequence
  int part_slots;          // parts that the workspace has room for
  float* part_o;           // [part_slots, 64, dv] unnormalised parts
  float* part_ml;          // [part_slots, 64, 2] their maximum (log2 domain) and sum
};

// How such a call runs, from its host bounds.
struct RowsPlan {
  int q_rows;
  long long tiles;         // at most
  int max_splits;
  long long slots;         // parts, at most
  double part_floats;      // of their outputs
  double bytes;            // of workspace; in floating point: absurd sizes must not wrap
};
// How a call of drafted trees over a K/V cache runs.
struct TreePlan {
  int tok_tile;            // tokens of a Q tile
  long long tiles, items;  // Q tiles, items, at most
  int max_splits;
  long long slots;         // parts, at most
  double bytes;
};
TreePlan tree_plan(int hq, int hkv, int dv, bool uniform, long long num_seqs, long long total_rows, int max_ctx);
cudaError_t launch_tree(const RowsAttnArgs& a, const TreePlan& p, int dtype, cudaStream_t st);

RowsPlan rows_plan(int heads, int dv, bool uniform, long long num_seqs, long long total_rows, int max_ctx);

// Attention of chunks over expanded keys and values (cp_latent_chunk_attn).
struct ExpandedArgs {
  int heads, dn, r, dv;
  float scale_log2;
  SeqRows rows, keys;
  int total_rows, total_keys;
  const void* q;           // [total_rows, H, dn + r]
  const void* k_nope;
  const void* k_rope;
  const void* v;
  long long k_row, k_head, r_row, v_row, v_head;  // elements
  void* out;               // [total_rows, H, dv]
  int* status;
};

// The rows of accepted paths to their places (cp_tree_commit).
struct CommitArgs {
  int hkv, row_bytes;      // KV heads, bytes of a (position, head) row
  CacheView cache;
  const int* path;         // [num_seqs, max_path]
  const int* counts;
  int* lens;
  int num_seqs, max_path, max_ctx;
  bool commit;
  void* k;
  void* v;                 // nullptr: a latent cache
  int* status;
};

cudaError_t launch_latent_append(const LatentAppendArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_rows_attn(const RowsAttnArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_expanded(const ExpandedArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_tree_commit(const CommitArgs& a, cudaStream_t st);

}  // namespace cp
