// tree_commit.cu -- the accepted path of a drafted tree, moved to its places.
//
// A path's places ascend, so place j of it is at j or behind: a row never moves
// onto the source of a later one, but may move onto that of an earlier one.  Each
// thread therefore moves its own 16-byte piece of all the path's rows in order, eight
// at a time -- the eight loads, then the eight stores -- and threads need not wait for
// one another.  One CTA a sequence, so that it may advance the length itself.  Bound by
// latency (a path's places, their pages, the rows): 64 paths of 8 of 61 rows, 8 heads x 128 in
// pages of 16, 3.3 us, one path of 5 rows 2.4 us, launch included.
#include <cstdint>

#include "cp_latent.h"
#include "cp_rows.cuh"

namespace cp {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;

__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const CommitArgs a) {
  __shared__ long long src[CP_TREE_MAX], dst[CP_TREE_MAX];  // rows of KV head 0
  pdl_launch_dependents();
  pdl_wait();
  const int s = blockIdx.x, j = threadIdx.x;
  const int count = a.counts[s], len = a.lens[s];
  const int* path = a.path + (long long)s * a.max_path;
  bool bad = count < 0 || count > a.max_path || len < 0 || len > a.max_ctx;
  if (!bad && j < count) {
    const int p = path[j];
    src[j] = p < 0 ? -1 : cache_row(a.cache, a.hkv, s, 0, (long long)len + p, a.max_ctx);
    dst[j] = cache_row(a.cache, a.hkv, s, 0, (long long)len + j, a.max_ctx);
    bad = src[j] < 0 || dst[j] < 0 || (j > 0 && path[j - 1] >= p);
  }
  if (__syncthreads_or(bad)) {
    if (j == 0 && a.status) atomicOr(a.status, CP_DEV_BOUNDS);
    return;
  }
  if (j == 0 && a.commit) a.lens[s] = len + count;
  const int pieces = a.row_bytes / 16, per = pieces * a.hkv;  // 16-byte pieces of a position in one array
  const long long head = a.cache.kind == CP_CACHE_PAGED ? a.cache.page_size : a.cache.capacity;  // rows between KV heads
  for (int i = threadIdx.x; i < (a.v ? 2 : 1) * per; i += kThreads) {
    uint4* x = static_cast<uint4*>(i < per ? a.k : a.v);
    const int e = i < per ? i : i - per;
    const long long at = (long long)(e / pieces) * head;
    const int piece = e % pieces;
    for (int j0 = 0; j0 < count; j0 += kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (j0 + u < count) v[u] = x[(src[j0 + u] + at) * pieces + piece];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (j0 + u < count && src[j0 + u] != dst[j0 + u]) x[(dst[j0 + u] + at) * pieces + piece] = v[u];
    }
  }
}

}  // namespace

cudaError_t launch_tree_commit(const CommitArgs& a, cudaStream_t st) {
  return launch_pdl(tree_commit_kernel, dim3(a.num_seqs), dim3(kThreads), 0, st, a);
}

}  // namespace cp
