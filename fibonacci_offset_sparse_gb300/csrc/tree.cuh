// Device pieces that the two tree decodes share: a sequence's state and its tree in shared
// memory.
#pragma once
#include "cache.cuh"
#include "tc_common.cuh"

namespace fibattn {

// The tree of one sequence.  anc[s][j]: the ancestor j levels above node s (anc[s][0] = s).
struct TreeSmem {
  int n, len;
  int depth[kMaxDrafts];
  int parent[kMaxDrafts];
  unsigned char anc[kMaxDrafts][kMaxDrafts];
};

// Reads the sequence and builds its tree; every thread of the block calls it (at least
// kMaxDrafts of them).  False (for the whole block) where a value is out of its range: nothing
// may be read or written for this sequence then.  Ends with the block synchronised.
__device__ __forceinline__ bool load_tree(const TreeArgs& a, int b, TreeSmem* ts) {
  const int tid = threadIdx.x;
  const int n = a.nodes == nullptr ? a.T : a.nodes[b];
  const int len = a.lens[b];
  bool bad = n < 0 || n > a.T || len < 0 || len > (static_cast<long long>(a.max_pages) << a.page_shift);
  if (!bad && tid < n) {
    const int p = a.parent == nullptr ? tid - 1 : a.parent[static_cast<size_t>(b) * a.T + tid];
    bad = p < -1 || p >= tid;
    ts->parent[tid] = p;
  }
  if (tid == 0) {
    ts->n = n;
    ts->len = len;
  }
  bad = __syncthreads_or(bad);
  if (!bad && tid < n) {
    int d = 0;
    for (int u = tid; u >= 0; u = ts->parent[u]) ts->anc[tid][d++] = static_cast<unsigned char>(u);
    ts->depth[tid] = d - 1;
    bad = static_cast<long long>(len) + d > a.N;
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) atomicExch(a.status, kStatusDeviceAssert);
  return !bad;
}

// Offset (in elements) of cache row x of sequence b, key head h, in the layer's pools; -1 where the
// page id lies outside the pool.
__device__ __forceinline__ long long cache_row(const TreeArgs& a, int b, int h, int x) {
  const int page = __ldg(a.table + static_cast<size_t>(b) * a.max_pages + (x >> a.page_shift));
  if (page < 0 || page >= a.n_pages) return -1;
  return (((static_cast<long long>(page) * a.H + h) << a.page_shift) + (x & ((1 << a.page_shift) - 1))) * kD;
}

}  // namespace fibattn
