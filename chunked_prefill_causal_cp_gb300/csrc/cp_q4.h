// cp_q4.h -- argument blocks and launchers of the query/key preparation and of
// the 4-bit cache.  Every pointer is a device pointer.
#pragma once

#include "cp_internal.h"

namespace cp {

// Keys per split of a sequence of n keys on the split path: few for a short
// context, where the wait for one CTA's walk is what counts (one row over 1025
// keys: 6.6 us with 256, 8.2 with 512; over 8001 keys: 8.9 with 512, 12.1 with 1024),
// more for a long one, whose set-up and parts cost less then (4 x 100001 keys: 121
// us with 1024 against 132 with 512; 64 rows over 512 to 8191 keys would gain 3% from
// 1024 beyond 4096).  By the sequence's own length alone, so a row's result never
// depends on what shares the launch.
__host__ __device__ inline int q4_split_keys(int n) { return n <= 2048 ? 256 : n <= 16384 ? 512 : 1024; }
__host__ __device__ inline int q4_splits(int n) { return (n - 1) / q4_split_keys(n) + 1; }
// Most splits of any sequence of up to `ctx` keys.
inline int q4_max_splits(int ctx) {
  int m = q4_splits(ctx);
  if (ctx > 2048) m = m > q4_splits(2048) ? m : q4_splits(2048);
  if (ctx > 16384) m = m > q4_splits(16384) ? m : q4_splits(16384);
  return m;
}

// Norm and rotation of the query and key heads (cp_qk_norm_rope), and, when
// k_cache is set, the keys and values into their cache slots.
struct RopeArgs {
  int hq, hkv;             // 0: that tensor is skipped
  int pairs;               // lanes of a head row that rotate (see qk_rope.cu)
  int half;                // first channel of the second half (rot_dim / 2), half-split pairs
  bool interleaved;
  float eps;
  SeqRows rows;
  int total_rows;
  const void* q;
  const void* k;
  const void* v;           // append only
  long long q_stride, k_stride, v_stride;  // elements from a row to the next
  const void* q_weight;    // [D] or nullptr
  const void* k_weight;
  const float* inv_freq;
  const int* positions;    // [total_rows] or nullptr: past + row within the sequence
  const int* past;
  void* q_out;
  void* k_out;             // dense rows, without an append
  CacheView cache;
  void* k_cache;
  void* v_cache;
  int max_ctx;
  int* status;
};

// Rows into or out of a 4-bit cache.
struct Q4Args {
  int hkv;
  SeqRows rows;
  int total_rows;
  CacheView cache;
  const int* past;         // position of each sequence's first row
  int max_ctx;
  uint8_t* k_codes;        // [..., D / 2]
  uint8_t* v_codes;
  uint32_t* k_params;      // [..., D / 32]: scale in the low half, smallest value in the high half
  uint32_t* v_params;
  const void* k_new;       // append: rows in
  const void* v_new;
  void* k_out;             // read: rows out (either may be nullptr)
  void* v_out;
  int* past_snapshot;      // optional [num_seqs]: CTA 0 copies past[] here
  int* status;
};

// Attention over a 4-bit cache.
struct Q4AttnArgs {
  int hq, hkv, group;
  float scale_log2;        // softmax scale * log2(e)
  SeqRows rows;
  int total_rows;
  CacheView cache;
  const int* past;
  int max_ctx;
  const void* q;           // [total_rows, hq, D]
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const uint32_t* k_params;
  const uint32_t* v_params;
  void* out;
  int* status;
  int min_rows;            // tensor-core kernel: sequences with fewer rows are skipped (the split path has them)
  int dec_rows;            // split path: takes the sequences of exactly this many rows (dec_rows * group <= 16)
  bool by_row;             // split path, dec_rows 1: takes every row of the call (no more than num_seqs), one by one
  int max_splits;
  float* part_o;           // [num_seqs * dec_rows, hq, max_splits, D] unnormalised parts
  float* part_ml;          // [num_seqs * dec_rows, hq, max_splits, 2] their maximum (log2 domain) and sum
  int* commit_lens;        // optional: CTA (0, 0) advances these lengths by each sequence's rows (`past` is a copy)
};

cudaError_t launch_qk_rope(const RopeArgs& a, int dtype, int d, cudaStream_t st);
cudaError_t launch_q4_append(const Q4Args& a, int dtype, int d, cudaStream_t st);
cudaError_t launch_q4_read(const Q4Args& a, int dtype, int d, cudaStream_t st);
// Split path: the sequences of exactly a.dec_rows rows, parts and their merge.
cudaError_t launch_q4_decode(const Q4AttnArgs& a, int dtype, int d, cudaStream_t st);
// Tensor-core path: the sequences of at least a.min_rows rows; pairs_bound: pairs of 128-row Q tiles to cover.
cudaError_t launch_q4_tc(const Q4AttnArgs& a, int dtype, int d, int pairs_bound, cudaStream_t st);

}  // namespace cp
