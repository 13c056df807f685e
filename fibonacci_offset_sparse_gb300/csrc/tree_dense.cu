// Dense decode of a tree of drafted tokens over the paged cache (sm_103a): the dense control's
// form of tree.cu.  Node s attends every cached row, its ancestors and itself.
#include "tree.cuh"

namespace fibattn {

namespace {

constexpr int kDtThreads = 128;
constexpr int kDtQuads = kDtThreads / 4;

// A block a row (node and query head): its 32 quads take keys c, c + 32, ... of the cached rows
// and then the ancestors; the quads merge through shared memory in a fixed order.
template <typename DT>
__global__ void __launch_bounds__(kDtThreads) dense_tree_kernel(const __grid_constant__ TreeArgs a) {
  __shared__ TreeSmem ts;
  __shared__ float s_m[kDtQuads], s_l[kDtQuads], s_o[kDtQuads][kD];
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int tid = threadIdx.x, quad = tid >> 2, t = tid & 3;
  if (!load_tree(a, b, &ts)) return;
  const int n = ts.n, len = ts.len, r = blockIdx.y;
  if (r >= n * a.G) return;
  const int g = r / n, s = r % n, depth = ts.depth[s];
  const size_t fresh = (static_cast<size_t>(b) * a.H + h) * a.T * kD;
  const size_t row = (static_cast<size_t>(b) * a.Hq + h * a.G + g) * a.T + s;
  float q[16];
  float2 e[8];
  load_part(static_cast<const DT*>(a.q) + row * kD, t, q);
  rope_row(a.rope_lo, a.rope_hi, len + depth, t, e);
  rotate_part(q, e, false);
#pragma unroll
  for (int u = 0; u < 16; ++u) q[u] *= kLog2e / 8.0f;
  float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
  for (int u = 0; u < 16; ++u) o[u] = 0.f;
  for (int c0 = 0; c0 < len + depth + 1; c0 += kDtQuads) {  // the same trip count in every quad
    const int c = c0 + quad;
    const bool ok = c < len + depth + 1;
    float k[16], v[16], sc = 0.f;
    if (ok && c < len) {
      long long at = cache_row(a, b, h, c);
      if (at < 0) {
        atomicExch(a.status, kStatusDeviceAssert);
        at = 0;
      }
      load_part(static_cast<const DT*>(a.kc) + at, t, k);
      load_part(static_cast<const DT*>(a.vc) + at, t, v);
    } else if (ok) {
      const int u = ts.anc[s][c - len];
      load_part(static_cast<const DT*>(a.kn) + fresh + static_cast<size_t>(u) * kD, t, k);
      load_part(static_cast<const DT*>(a.vn) + fresh + static_cast<size_t>(u) * kD, t, v);
      rope_row(a.rope_lo, a.rope_hi, len + ts.depth[u], t, e);
      rotate_part(k, e, false);
    }
    if (ok) {
#pragma unroll
      for (int u = 0; u < 16; ++u) sc = fmaf(q[u], k[u], sc);
    }
    sc = quad_sum(sc);
    if (!ok) continue;  // after the shuffles
    if (sc == -INFINITY) continue;  // weight 0 (a NaN goes on)
    const float mn = fmaxf(m, sc);
    const float corr = exp2f(m - mn), p = exp2f(sc - mn);
    l = l * corr + p;
#pragma unroll
    for (int u = 0; u < 16; ++u) o[u] = fmaf(p, v[u], o[u] * corr);
    m = mn;
  }
  if (t == 0) s_m[quad] = m;
  __syncthreads();
  float all = -INFINITY;
  for (int x = 0; x < kDtQuads; ++x) all = fmaxf(all, s_m[x]);
  const float f = m == -INFINITY ? 0.f : exp2f(m - all);  // a quad that saw no key
  if (t == 0) s_l[quad] = l * f;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    s_o[quad][8 * t + u] = o[u] * f;
    s_o[quad][kFreq + 8 * t + u] = o[8 + u] * f;
  }
  __syncthreads();
  if (tid < kD) {
    float acc = 0.f, sum = 0.f;
    for (int x = 0; x < kDtQuads; ++x) {
      acc += s_o[x][tid];
      sum += s_l[x];
    }
    const float out = acc / sum;
    if constexpr (sizeof(DT) == 4)
      static_cast<float*>(a.o)[row * kD + tid] = out;
    else
      static_cast<__nv_bfloat16*>(a.o)[row * kD + tid] = __float2bfloat16_rn(out);
    if (tid == 0 && a.lse != nullptr) a.lse[row] = (all + log2f(sum)) * kLn2;
  }
}

}  // namespace

size_t dense_tree_workspace_bytes(int, int, int, int, int) { return 256; }

cudaError_t launch_dense_tree(const TreeArgs& a, int dtype, void*, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.H, static_cast<unsigned>(a.G * a.T));
  if (dtype == FIB_DTYPE_F32)
    dense_tree_kernel<float><<<grid, kDtThreads, 0, stream>>>(a);
  else
    dense_tree_kernel<__nv_bfloat16><<<grid, kDtThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fibattn
