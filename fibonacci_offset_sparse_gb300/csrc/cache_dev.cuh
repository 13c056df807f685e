// What the paged cache's own operators share on the device (cache.cu, evict.cu): the cache as kernels see it, launches in
// a chain, counts of pages and the search for free ones.
#pragma once
#include "cache.cuh"
#include "tc_common.cuh"

namespace fibattn {

constexpr int kPlanThreads = 1024;

struct CacheDev {
  int L, H, P, shift, n_pages, S, max_pages;
  void* k;
  void* v;
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  int32_t* state;
};

inline CacheDev device_view(const fib_attn_cache& c) {
  CacheDev d;
  d.L = c.n_layers;
  d.H = c.heads;
  d.P = c.page_rows;
  d.shift = log2_of(c.page_rows);
  d.n_pages = c.n_pages;
  d.S = c.max_seqs;
  d.max_pages = c.max_pages;
  d.k = c.k;
  d.v = c.v;
  d.table = c.table;
  d.lens = c.lens;
  d.refs = c.refs;
  d.state = c.state;
  return d;
}

__device__ __forceinline__ void wait_for_first() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void let_second_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// A kernel, in clusters of `cluster` blocks and with `shared` bytes of dynamic shared memory, as a programmatic dependent of the one before it on
// the stream.
template <typename... Params, typename... Args>
inline cudaError_t launch_second_in_clusters(void (*kernel)(Params...), dim3 grid, unsigned cluster, int threads, size_t shared, cudaStream_t stream,
                                             Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = shared;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename... Params, typename... Args>
inline cudaError_t launch_second(void (*kernel)(Params...), dim3 grid, int threads, size_t shared, cudaStream_t stream, Args... args) {
  return launch_second_in_clusters(kernel, grid, 1, threads, shared, stream, args...);
}

// The counts of four pages from `id` (a multiple of 4) on; 0 behind the last page.
__device__ __forceinline__ void load_counts(const CacheDev& c, int id, int (&r)[4]) {
  r[0] = r[1] = r[2] = r[3] = 0;
  if (id + 3 < c.n_pages) {
    const int4 x = *reinterpret_cast<const int4*>(c.refs + id);
    r[0] = x.x; r[1] = x.y; r[2] = x.z; r[3] = x.w;
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (id + u < c.n_pages) r[u] = c.refs[id + u];
  }
}
// ... 1 (in use) for those outside [from, n_pages).
__device__ __forceinline__ void load_refs(const CacheDev& c, int id, int from, int (&r)[4]) {
  load_counts(c, id, r);
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (id + u < from || id + u >= c.n_pages) r[u] = 1;
}

// The ids of free pages from `from` on, ascending, into list[0 .. want); returns how many there
// are up to `want`.  4096 counts a step (r: those of the first, loaded by the caller ahead of its other reads);
// stops as soon as enough are found.
__device__ inline int find_free(const CacheDev& c, int from, int (&r)[4], int want, int32_t* list, int* sums) {
  int found = 0;
  for (int base = from & ~3; base < c.n_pages && found < want; base += 4 * kPlanThreads) {
    const int id = base + 4 * static_cast<int>(threadIdx.x);
    if (base > from) load_refs(c, id, from, r);
    const int n = (r[0] == 0) + (r[1] == 0) + (r[2] == 0) + (r[3] == 0);
    int total;
    int at = found + block_scan_1024(n, sums, &total);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (r[u] == 0) {
        if (at < want) list[at] = id + u;
        ++at;
      }
    found += total;
  }
  __syncthreads();
  return min(found, want);
}

__device__ __forceinline__ int pages_of(const CacheDev& c, int len) { return (len + c.P - 1) >> c.shift; }

inline size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace fibattn
