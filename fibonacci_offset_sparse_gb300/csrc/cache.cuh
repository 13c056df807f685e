// Launch interface of the paged cache's kernels (cache.cu) and of the decodes over it
// (tree.cu, tree_dense.cu).
#pragma once
#include "../../include/fib_attn.h"
#include "common.cuh"

namespace fibattn {

constexpr int kMaxDrafts = FIB_MAX_DRAFTS;
constexpr int kMaxSeqs = FIB_MAX_SEQS;
constexpr int kStatusNoPages = 8;  // FIB_ERR_NO_PAGES

// state words of a cache
constexpr int kStateCursor = 0, kStateStatus = 1, kStateLive = 2;

size_t cache_workspace_bytes(const fib_attn_cache& c);
cudaError_t launch_cache_commit(const fib_attn_cache& c, int B, int T, int n_max, const int32_t* n_new,
                                const int32_t* path, const void* k_new, const void* v_new, const float2* lo_tab,
                                const float2* hi_tab, void* ws, cudaStream_t stream);
cudaError_t launch_cache_fork(const fib_attn_cache& c, const int32_t* src, void* ws, cudaStream_t stream);
cudaError_t launch_cache_compact(const fib_attn_cache& c, int32_t* remap, void* ws, cudaStream_t stream);

// What the decodes share.  kc, vc: the layer's pools.
struct TreeArgs {
  LayerTable t;  // sparse only
  int N;         // positions are below it
  int B, Hq, H, G, T;
  int n_pages, max_pages, page_shift;
  const void* q;
  const void* kn;
  const void* vn;
  const void* kc;
  const void* vc;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* parent;
  const int32_t* nodes;
  void* o;
  float* lse;
  const float2* rope_lo;
  const float2* rope_hi;
  int* status;
};
cudaError_t launch_tree(const TreeArgs& a, int dtype, cudaStream_t stream);
size_t dense_tree_workspace_bytes(int Hq, int H, int T, int dtype);
cudaError_t launch_dense_tree(const TreeArgs& a, int dtype, unsigned long long wait_ns, int skip_copy, void* ws, cudaStream_t stream);

inline int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// Block-wide exclusive prefix sum of `x` over 1024 threads; *total gets the sum.  `sums`: 33
// ints of shared memory.  Ends with the block synchronised.
__device__ __forceinline__ int block_scan_1024(int x, int* sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int s = sums[lane];
    int si = s;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, si, d);
      if (lane >= d) si += y;
    }
    sums[lane] = si - s;
    if (lane == 31) sums[32] = si;
  }
  __syncthreads();
  const int out = sums[warp] + inc - x;
  *total = sums[32];
  __syncthreads();
  return out;
}

}  // namespace fibattn
