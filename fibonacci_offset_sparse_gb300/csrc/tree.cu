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
// a row, and quads and warps merge their running maxima and sums in a fixed order.  No shared memory but
// the key table of a device alpha and the merge of four warps.
#include "tree.cuh"

namespace fibattn {

namespace {

constexpr int kTreeWarps = 4;

// The ancestor d levels above the node whose line is `above`: the d-th set bit from the top.
__device__ __forceinline__ int ancestor_at(uint64_t above, int d) {
  int u = 0;
#pragma unroll
  for (int step = 32; step > 0; step >>= 1)
    if (__popcll(above >> (u + step)) > d) u += step;
  return u;
}

// PER: warps a row (1 or 4).
template <typename DT, int PER>
__global__ void __launch_bounds__(32 * kTreeWarps) tree_kernel(const __grid_constant__ TreeArgs a, int blocks_per_head) {
  __shared__ KeySmem ks;
  __shared__ __align__(16) float s_o[kTreeWarps][kD];
  __shared__ float s_m[kTreeWarps], s_l[kTreeWarps];
  const int head = blockIdx.x / blocks_per_head, b = head / a.H, h = head % a.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3;
  const int quad = (PER == 1 ? 0 : 8 * warp) + (lane >> 2);
  constexpr int kQuads = 8 * PER;
  // the key table: from the launch parameters where the host knows the distances, else from the device alpha
  const bool host_keys = a.t.mode == 0 || a.t.alpha_dev == nullptr;
  if (!host_keys) {
    build_keys(a.t, a.N, &ks);
    __syncthreads();
  }
  const int nv = host_keys ? a.t.W + a.t.n : ks.nv;
  int n, len;
  bool ok = sequence_of(a, b, &n, &len);
  if (!ok) {
    if (threadIdx.x == 0) atomicExch(a.status, kStatusDeviceAssert);
    return;
  }
  const int r = (blockIdx.x % blocks_per_head) * (kTreeWarps / PER) + (PER == 1 ? warp : 0);
  if (r >= n * a.G) return;  // (of the whole block where four warps share a row)
  const int g = r / n, s = r - g * n;
  const WarpTree tree = warp_tree(a.parent == nullptr ? nullptr : a.parent + static_cast<size_t>(b) * a.T, n, &ok);
  const int depth = pick32(tree.depth, s), pos = len + depth;
  const uint64_t above = pick64(tree.above, s);
  if (pos >= a.N) ok = false;
  if (!ok) {  // (the same in all warps of a row)
    if (lane == 0) atomicExch(a.status, kStatusDeviceAssert);
    return;
  }
  const size_t row = (static_cast<size_t>(b) * a.Hq + h * a.G + g) * a.T + s;
  const DT* kn = static_cast<const DT*>(a.kn) + (static_cast<size_t>(b) * a.H + h) * a.T * kD;
  const DT* vn = static_cast<const DT*>(a.vn) + (static_cast<size_t>(b) * a.H + h) * a.T * kD;
  float q[16];
  load_part(static_cast<const DT*>(a.q) + row * kD, t, q);
  {
    float2 e[8];
    rope_row(a.rope_lo, a.rope_hi, pos, t, e);
    rotate_part(q, e, false);
  }
#pragma unroll
  for (int u = 0; u < 16; ++u) q[u] *= kLog2e / 8.0f;
  // the row at distance d: its K part into k, its V part into v
  auto fetch = [&](int d, float (&k)[16], float (&v)[16]) {
    if (d <= depth) {
      const int u = ancestor_at(above, d);
      float2 e[8];
      load_part(kn + static_cast<size_t>(u) * kD, t, k);
      load_part(vn + static_cast<size_t>(u) * kD, t, v);
      rope_row(a.rope_lo, a.rope_hi, pos - d, t, e);
      rotate_part(k, e, false);
      return;
    }
    long long at = cache_row(a, b, h, pos - d);
    if (at < 0) {
      atomicExch(a.status, kStatusDeviceAssert);
      at = 0;
    }
    load_part(static_cast<const DT*>(a.kc) + at, t, k);
    load_part(static_cast<const DT*>(a.vc) + at, t, v);
  };
  float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
  for (int u = 0; u < 16; ++u) o[u] = 0.f;
  for (int c0 = 0; c0 < nv; c0 += kQuads) {  // the same trip count in every quad
    const int c = c0 + quad;
    int lo = 0, need = pos + 1;
    float w = 0.f;
    if (c < nv) {
      if (!host_keys) {
        lo = ks.lo[c];
        w = ks.w[c];
      } else if (c < a.t.W) {
        lo = c;
      } else {
        lo = a.t.lo[c - a.t.W];
        w = a.t.mode == 1 ? a.t.w[c - a.t.W] : 0.f;
      }
      need = lo + (w > 0.f ? 1 : 0);
    }
    const bool in = pos >= need;
    float k[16], v[16], sc = 0.f;
    if (in) {
      fetch(lo, k, v);
      if (w > 0.f) {
        float k1[16], v1[16];
        fetch(lo + 1, k1, v1);
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
    if (!in) continue;             // after the shuffles; no further warp-wide operation in this trip
    if (sc == -INFINITY) continue;  // weight 0 (a NaN goes on)
    const float mn = fmaxf(m, sc);
    const float corr = exp2f(m - mn), p = exp2f(sc - mn);
    l = l * corr + p;
#pragma unroll
    for (int u = 0; u < 16; ++u) o[u] = fmaf(p, v[u], o[u] * corr);
    m = mn;
  }
  __syncwarp();
  // merge the quads of the warp; a quad without a finite score counts nothing, unless a NaN is in it
  auto weight = [](float m, float l, float all) { return m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : exp2f(m - all); };
  float all = m;
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, x));
  const float f = weight(m, l, all);
  l *= f;
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    o[u] *= f;
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) o[u] += __shfl_xor_sync(0xffffffffu, o[u], x);
  }
  if constexpr (PER == 1) {
    const float inv = 1.f / l;
#pragma unroll
    for (int u = 0; u < 16; ++u) o[u] *= inv;
    if (lane < 4) {
      store_part(static_cast<DT*>(a.o) + row * kD, t, o);
      if (t == 0 && a.lse != nullptr) a.lse[row] = (all + log2f(l)) * kLn2;
    }
  } else {
    if (lane < 4) store_part(s_o[warp], t, o);
    if (lane == 0) {
      s_m[warp] = all;
      s_l[warp] = l;
    }
    __syncthreads();
    if (warp == 0 && lane < 16) {
      float top = -INFINITY, sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int y = 0; y < kTreeWarps; ++y) top = fmaxf(top, s_m[y]);
#pragma unroll
      for (int y = 0; y < kTreeWarps; ++y) {
        const float fy = weight(s_m[y], s_l[y], top);
        sum += s_l[y] * fy;
        const float4 z = *reinterpret_cast<const float4*>(&s_o[y][4 * lane]);
        x[0] += z.x * fy;
        x[1] += z.y * fy;
        x[2] += z.z * fy;
        x[3] += z.w * fy;
      }
      const float inv = 1.f / sum;
      if constexpr (sizeof(DT) == 4)
        *reinterpret_cast<float4*>(static_cast<float*>(a.o) + row * kD + 4 * lane) = make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
      else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + row * kD + 4 * lane) =
            make_uint2(pack_bf2(x[0] * inv, x[1] * inv), pack_bf2(x[2] * inv, x[3] * inv));
      if (lane == 0 && a.lse != nullptr) a.lse[row] = (top + log2f(sum)) * kLn2;
    }
  }
}

template <typename DT>
cudaError_t launch_rows(const TreeArgs& a, cudaStream_t stream) {
  const int heads = a.B * a.H, rows = a.G * a.T;
  // four warps a row while that leaves SMs idle otherwise: a row then waits for its keys once, not three times
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
  return dtype == FIB_DTYPE_F32 ? launch_rows<float>(a, stream) : launch_rows<__nv_bfloat16>(a, stream);
}

}  // namespace fibattn
