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
};

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
