// Sparse decode of a tree of drafted tokens over the paged cache (sm_103a).
//
// Node s of a sequence sits at position p = len + depth(s); its key at distance d is the
// ancestor d levels up where d <= depth(s) and cache row p - d otherwise, so that it attends
// exactly what row p of the forward attends in the sequence of the cached rows and its line of
// ancestors ("Depth-Staggered Fibonacci Spacing for Sparse Attention", Methodology >
// "Attended set", "Scaling", "Implementation").  Cached K rows are rotated already; the query
// and the drafted K rows are rotated here, in float32, at their own positions.
//
// Row by row (this file): a row is a node and a query head.  What bounds it is latency: lengths and
// parents, then pages and tables, then the rows themselves, one after the other; everything of a step is on its
// way at once.  A quad of threads takes a key (lane t the dims D_t of common.cuh), a warp or four
// a row, and quads and warps merge their running maxima and sums in a fixed order.  One token of one sequence takes 3.8 us
// in a graph, 32768 float32 rows of 35 interpolated keys 91 us (97 where alpha is on the device), of 35 rows 79.  No shared memory but
// the key table of a device alpha and the merge of four warps.
#include "tree.cuh"

namespace fibattn {

namespace {

constexpr int kTreeWarps = 4;

// PER: warps a row (1 or 4).  128 registers, so that an SM holds 16 warps: 64 sequences of 8 heads and 64 float32 nodes take
// 99 us, with 134 registers and 12 warps 113, with 96 and 20 (they spill) 113; one node each 6.0, 8.2 and 6.4.
template <typename DT, int PER>
__global__ void __launch_bounds__(32 * kTreeWarps, 4) tree_kernel(const __grid_constant__ TreeArgs a, int blocks_per_head) {
  __shared__ KeySmem ks;
  __shared__ RowMerge<PER> merge;
  const int head = blockIdx.x / blocks_per_head, b = head / a.H, h = head % a.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the key table: from the launch parameters where the host knows the distances, else from the device alpha
  const bool host_keys = a.t.mode == 0 || a.t.alpha_dev == nullptr;
  if (!host_keys) {
    build_keys(a.t, a.N, &ks);
    __syncthreads();
  }
  int n, len;
  bool ok = sequence_of(a, b, &n, &len);
  if (!ok) {
    if (threadIdx.x == 0) atomicExch(a.status, kStatusDeviceAssert);
    return;
  }
  const int r = (blockIdx.x % blocks_per_head) * (kTreeWarps / PER) + (PER == 1 ? warp : 0);
  if (r >= n * a.G) return;  // (of the whole block where four warps share a row)
  const int g = r / n, s = r - g * n;
  const WarpTree tree = warp_tree(a, b, n, &ok);
  const int depth = pick32(tree.depth, s), pos = len + depth;
  const uint64_t above = pick64(tree.above, s);
  if (pos >= a.N) ok = false;
  if (!ok) {  // (the same in all warps of a row)
    if (lane == 0) atomicExch(a.status, kStatusDeviceAssert);
    return;
  }
  const size_t row = (static_cast<size_t>(b) * a.Hq + h * a.G + g) * a.T + s;
  attend_row<DT, PER>(a, host_keys ? nullptr : &ks, b, h, row, depth, pos, above, PER == 1 ? 0 : warp, &merge);
}

template <typename DT>
cudaError_t launch_rows(const TreeArgs& a, cudaStream_t stream) {
  const int heads = a.B * a.H, rows = a.G * a.T;
  // Four warps a row while that leaves SMs idle otherwise: a row then waits for its keys once, not three times.  Of 8 rows in
  // all 4.7 us with four warps and 6.2 with one, 256 rows 5.1 and 6.3, 512 rows 6.0 and 6.5, 1024 rows 10.0 and 7.1.
  if (static_cast<long long>(heads) * rows <= 152 * 4) {
    tree_kernel<DT, 4><<<heads * rows, 32 * kTreeWarps, 0, stream>>>(a, rows);
  } else {
    const int per = (rows + kTreeWarps - 1) / kTreeWarps;
    const long long blocks = static_cast<long long>(heads) * per;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    tree_kernel<DT, 1><<<static_cast<unsigned>(blocks), 32 * kTreeWarps, 0, stream>>>(a, per);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree(const TreeArgs& a, int dtype, cudaStream_t stream) {
  if (dtype == FIB_DTYPE_F32) return launch_rows<float>(a, stream);
  return tree_tc_serves(a) ? launch_tree_tc(a, stream) : launch_rows<__nv_bfloat16>(a, stream);
}

}  // namespace fibattn
