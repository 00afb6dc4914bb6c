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

// How the work of cp_latent_attn and cp_tree_attn is shared out: units -- a tile of pairs, or
// pair of Q tiles, of a sequence (and KV head), with all its tiles of keys -- lie in a row,
// which is cut into a share for each CTA, wherever in a unit that is.
// All CTAs have as much to do, within a tile, whatever the sequences' lengths; a unit
// that does not end where it began leaves parts, of which a CTA has two at most: of
// the unit it starts in the middle of, and of the one it does not finish.  (Splits of
// fixed length, of a sequence's own or by the number of sequences, left the last CTA with
// 14 to 30% more than the mean, or had as much again in starts, ends and parts.)
constexpr int kSms = 152;
// Tiles of so many rows that num_seqs sequences of total_rows rows in all can have.
inline long long tiles_at_most(long long total_rows, long long num_seqs, long long rows) {
  return (total_rows + num_seqs * (rows - 1)) / rows;
}
constexpr int kStart = 4;  // what the start and end of a unit cost, in tiles (2 to 6 are within 3%, 1 is up to a fifth slower)
// The shares of `all` tiles: each CTA's, the first `more` of them one tile longer.
struct Shares {
  int ctas;         // that have one: of a grid, at most a CTA for each tile
  long long least;  // tiles of a share
  int more;
  __host__ __device__ Shares(long long all, int grid)
      : ctas(all < grid ? (all > 1 ? (int)all : 1) : grid), least(quotient(all, ctas)), more((int)(all - least * ctas)) {}
  __host__ __device__ static long long quotient(long long x, long long y) {  // in 32 bits where they do
    return ((unsigned long long)(x | y) >> 32) == 0 ? (long long)((unsigned)x / (unsigned)y) : x / y;
  }
  __host__ __device__ long long begin(int c) const { return least * c + (c < more ? c : more); }
  __host__ __device__ int of(long long tile) const {
    const long long longer = (least + 1) * more;
    return (int)(tile < longer ? quotient(tile, least + 1) : more + quotient(tile - longer, least));
  }
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
  // By the host's bounds:
  int ctas;                // that share the work
  int q_rows;              // a latent cache's: pairs of a tile that the call can have, at most
  int tok_tile;            // a tree's: tokens of a Q tile
  long long tiles;         // of pairs, or (pairs of) Q tiles, at most
  bool lone;               // a tree's units are of one Q tile
  bool split;              // whether units may be shared by CTAs
  float* part_o;           // parts: unnormalised outputs,
  float* part_ml;          // their maximum (log2 domain) and sum
};

// How such a call runs, from its host bounds.
struct RowsPlan {
  int ctas, q_rows, tok_tile;
  long long tiles;
  bool lone, split;
  double work;             // tiles of keys of all units, at most
  long long part_floats;   // of all parts' outputs
  long long bytes;         // of workspace
};
RowsPlan latent_plan(int heads, int dv, bool uniform, long long num_seqs, long long total_rows, int max_ctx);
RowsPlan tree_plan(int hq, int hkv, int dv, bool uniform, long long num_seqs, long long total_rows, int max_ctx);

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
cudaError_t launch_latent(const RowsAttnArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_latent_commit(int* lens, const SeqRows& rows, int total_rows, int max_ctx, cudaStream_t st);
cudaError_t launch_tree(const RowsAttnArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_expanded(const ExpandedArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_tree_commit(const CommitArgs& a, cudaStream_t st);

}  // namespace cp
