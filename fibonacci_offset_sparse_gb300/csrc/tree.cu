// Sparse decode of a tree of drafted tokens over the paged cache (sm_103a).
//
// Node s of a sequence sits at position p = len + depth(s); its key at distance d is the
// ancestor d levels up where d <= depth(s) and cache row p - d otherwise, so that it attends
// exactly what row p of the forward attends in the sequence of the cached rows and its line of
// ancestors ("Depth-Staggered Fibonacci Spacing for Sparse Attention", Methodology >
// "Attended set", "Scaling", "Implementation").  Cached K rows are rotated already; the query
// and the drafted K rows are rotated here, in float32, at their own positions.
#include "tree.cuh"

namespace fibattn {

namespace {

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

constexpr int kTreeThreads = 128;
constexpr int kTreeWarps = kTreeThreads / 32;

// A warp a row (node and query head): its 8 quads take keys c, c + 8, ...; a quad keeps an
// online softmax over its keys (lane t holds the dims D_t of common.cuh), and the quads merge
// with shuffles.
template <typename DT>
__global__ void __launch_bounds__(kTreeThreads) tree_kernel(const __grid_constant__ TreeArgs a, int rows_per_block) {
  __shared__ TreeSmem ts;
  __shared__ KeySmem ks;
  __shared__ __align__(16) float s_kd[kMaxDrafts][kD];
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int tid = threadIdx.x, warp = tid >> 5, quad = (tid & 31) >> 2, t = tid & 3;
  build_keys(a.t, a.N, &ks);
  if (!load_tree(a, b, &ts)) return;
  const int n = ts.n, len = ts.len;
  const int r0 = blockIdx.y * rows_per_block, r1 = min(r0 + rows_per_block, n * a.G);
  if (r0 >= r1) return;
  const DT* kn = static_cast<const DT*>(a.kn) + (static_cast<size_t>(b) * a.H + h) * a.T * kD;
  const DT* vn = static_cast<const DT*>(a.vn) + (static_cast<size_t>(b) * a.H + h) * a.T * kD;
  const DT* kc = static_cast<const DT*>(a.kc);
  const DT* vc = static_cast<const DT*>(a.vc);
  for (int u = tid >> 2; u < n; u += kTreeThreads / 4) {
    float x[16];
    float2 e[8];
    load_part(kn + static_cast<size_t>(u) * kD, t, x);
    rope_row(a.rope_lo, a.rope_hi, len + ts.depth[u], t, e);
    rotate_part(x, e, false);
    store_part(s_kd[u], t, x);
  }
  __syncthreads();
  for (int r = r0 + warp; r < r1; r += kTreeWarps) {
    const int g = r / n, s = r % n;
    const int depth = ts.depth[s], pos = len + depth;
    const size_t row = (static_cast<size_t>(b) * a.Hq + h * a.G + g) * a.T + s;
    float q[16];
    load_part(static_cast<const DT*>(a.q) + row * kD, t, q);
    {
      float2 e[8];
      rope_row(a.rope_lo, a.rope_hi, pos, t, e);
      rotate_part(q, e, false);
    }
#pragma unroll
    for (int u = 0; u < 16; ++u) q[u] *= kLog2e / 8.0f;
    // row at distance d: its K part into k, its V part into v
    auto fetch = [&](int d, float (&k)[16], float (&v)[16]) {
      if (d <= depth) {
        const int u = ts.anc[s][d];
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          k[w] = s_kd[u][8 * t + w];
          k[8 + w] = s_kd[u][kFreq + 8 * t + w];
        }
        load_part(vn + static_cast<size_t>(u) * kD, t, v);
        return;
      }
      long long at = cache_row(a, b, h, pos - d);
      if (at < 0) {
        atomicExch(a.status, kStatusDeviceAssert);
        at = 0;
      }
      load_part(kc + at, t, k);
      load_part(vc + at, t, v);
    };
    float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) o[u] = 0.f;
    for (int c0 = 0; c0 < ks.nv; c0 += 8) {  // the same trip count in every quad
      const int c = c0 + quad;
      const bool ok = c < ks.nv && pos >= ks.need[c];
      const float w = ok ? ks.w[c] : 0.f;
      float k[16], v[16], sc = 0.f;
      if (ok) {
        fetch(ks.lo[c], k, v);
        if (w > 0.f) {
          float k1[16], v1[16];
          fetch(ks.lo[c] + 1, k1, v1);
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            k[u] = (1.f - w) * k[u] + w * k1[u];
            v[u] = (1.f - w) * v[u] + w * v1[u];
          }
        }
#pragma unroll
        for (int u = 0; u < 16; ++u) sc = fmaf(q[u], k[u], sc);
      }
      sc = quad_sum(sc);
      if (!ok) continue;  // after the shuffles; no further warp-wide operation in this trip
      if (sc == -INFINITY) continue;  // weight 0 (a NaN goes on)
      const float mn = fmaxf(m, sc);
      const float corr = exp2f(m - mn), p = exp2f(sc - mn);
      l = l * corr + p;
#pragma unroll
      for (int u = 0; u < 16; ++u) o[u] = fmaf(p, v[u], o[u] * corr);
      m = mn;
    }
    __syncwarp();
    float all = m;
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, x));
    const float f = m == -INFINITY ? 0.f : exp2f(m - all);  // a quad that saw no key
    l *= f;
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    const float inv = 1.f / l;
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      o[u] *= f;
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) o[u] += __shfl_xor_sync(0xffffffffu, o[u], x);
      o[u] *= inv;
    }
    if (quad == 0) {
      store_part(static_cast<DT*>(a.o) + row * kD, t, o);
      if (t == 0 && a.lse != nullptr) a.lse[row] = (all + log2f(l)) * kLn2;
    }
  }
}

}  // namespace

cudaError_t launch_tree(const TreeArgs& a, int dtype, cudaStream_t stream) {
  const int rows = a.G * a.T, per = rows < 16 ? rows : 16;
  const dim3 grid(static_cast<unsigned>(a.B) * a.H, (rows + per - 1) / per);
  if (dtype == FIB_DTYPE_F32)
    tree_kernel<float><<<grid, kTreeThreads, 0, stream>>>(a, per);
  else
    tree_kernel<__nv_bfloat16><<<grid, kTreeThreads, 0, stream>>>(a, per);
  return cudaGetLastError();
}

}  // namespace fibattn
