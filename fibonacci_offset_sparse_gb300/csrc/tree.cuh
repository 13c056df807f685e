// Device pieces that the two tree decodes share: a sequence's tree, in registers of a warp.
#pragma once
#include "cache.cuh"
#include "tc_common.cuh"

namespace fibattn {

// The nodes of one sequence's tree over the lanes of a warp: lane x holds nodes x and x + 32.
// above[i]: bit u is set where node u is the node itself or one of its ancestors; since a parent has
// a smaller number than its child, ancestors lie nearer the higher their bit.
struct WarpTree {
  int depth[2];
  uint64_t above[2];
};

__device__ __forceinline__ uint64_t pick64(const uint64_t (&x)[2], int s) {
  const uint64_t a = __shfl_sync(0xffffffffu, x[0], s & 31), b = __shfl_sync(0xffffffffu, x[1], s & 31);
  return s & 32 ? b : a;
}
__device__ __forceinline__ int pick32(const int (&x)[2], int s) {
  const int a = __shfl_sync(0xffffffffu, x[0], s & 31), b = __shfl_sync(0xffffffffu, x[1], s & 31);
  return s & 32 ? b : a;
}

// The tree of sequence b with n nodes; a whole warp calls it.  Ancestors by doubling: after i
// rounds a node knows those up to 2^i levels above it.  *ok turns false (in every lane) where a
// parent is out of its range; the nodes are then taken as roots, so that nothing is read out
// of bounds.
__device__ __forceinline__ WarpTree warp_tree(const int32_t* parent, int n, bool* ok) {
  const int lane = threadIdx.x & 31;
  WarpTree t;
  int up[2];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = lane + 32 * i;
    up[i] = -1;
    if (s < n) {
      up[i] = parent == nullptr ? s - 1 : parent[s];
      if (up[i] < -1 || up[i] >= s) {
        bad = true;
        up[i] = -1;
      }
    }
    t.above[i] = 1ull << s;
  }
  if (__any_sync(0xffffffffu, bad)) {
    *ok = false;
    up[0] = up[1] = -1;
  }
  while (__any_sync(0xffffffffu, up[0] >= 0 || up[1] >= 0)) {
    uint64_t m[2];
    int v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[i] = pick64(t.above, up[i] & 63);
      v[i] = pick32(up, up[i] & 63);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (up[i] >= 0) {
        t.above[i] |= m[i];
        up[i] = v[i];
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) t.depth[i] = __popcll(t.above[i]) - 1;
  return t;
}

// Nodes and cached rows of sequence b; false where one is out of its range.
__device__ __forceinline__ bool sequence_of(const TreeArgs& a, int b, int* n, int* len) {
  *n = a.nodes == nullptr ? a.T : a.nodes[b];
  *len = a.lens[b];
  return *n >= 0 && *n <= a.T && *len >= 0 && *len <= (static_cast<long long>(a.max_pages) << a.page_shift) &&
         static_cast<long long>(*len) + (*n > 0) <= a.N;
}

// Offset (in elements) of cache row x of sequence b, key head h, in the layer's pools; -1 where the
// page id lies outside the pool.
__device__ __forceinline__ long long cache_row(const TreeArgs& a, int b, int h, int x) {
  const int page = __ldg(a.table + static_cast<size_t>(b) * a.max_pages + (x >> a.page_shift));
  if (page < 0 || page >= a.n_pages) return -1;
  return (((static_cast<long long>(page) * a.H + h) << a.page_shift) + (x & ((1 << a.page_shift) - 1))) * kD;
}

}  // namespace fibattn
