// Device pieces that the two tree decodes share: a sequence's tree, in registers of a warp.
#pragma once
#include "cache.cuh"
#include "tc_common.cuh"

namespace fibattn {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

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
__device__ __forceinline__ WarpTree warp_tree(const TreeArgs& a, int b, int n, bool* ok) {
  const int lane = threadIdx.x & 31;
  WarpTree t;
  int up[2];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = lane + 32 * i;
    up[i] = s - 1;  // (the row of parents is read whole, so that the load does not wait for n)
    if (a.parent != nullptr && s < a.T) up[i] = a.parent[static_cast<size_t>(b) * a.T + s];
    t.above[i] = 1ull << s;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = lane + 32 * i;
    if (s >= n) {
      up[i] = -1;
    } else if (up[i] < -1 || up[i] >= s) {
      bad = true;
      up[i] = -1;
    }
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

// The ancestor d levels above the node whose line is `above`: the d-th set bit from the top.
__device__ __forceinline__ int ancestor_at(uint64_t above, int d) {
  int u = 0;
#pragma unroll
  for (int step = 32; step > 0; step >>= 1)
    if (__popcll(above >> (u + step)) > d) u += step;
  return u;
}

// Shared memory in which four warps that share a row meet.
template <int PER>
struct RowMerge {
  float4 o[PER][kD / 4];
  float m[PER], l[PER];
};

// One row (node s at position pos = len + depth, of query row `row`) by PER warps (1 or 4), each calling it with its number.
// Keys: from `ks`, or from the launch parameters where the host knows the distances (ks null).
template <typename DT, int PER>
__device__ __forceinline__ void attend_row(const TreeArgs& a, const KeySmem* ks, int b, int h, size_t row, int depth, int pos, uint64_t above,
                                           int warp, RowMerge<PER>* merge) {
  const int lane = threadIdx.x & 31, t = lane & 3;
  const int quad = 8 * warp + (lane >> 2), nv = ks == nullptr ? a.t.W + a.t.n : ks->nv;
  constexpr int kQuads = 8 * PER;
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
      if (ks != nullptr) {
        lo = ks->lo[c];
        w = ks->w[c];
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
    if (lane < 4) store_part(reinterpret_cast<float*>(merge->o[warp]), t, o);
    if (lane == 0) {
      merge->m[warp] = all;
      merge->l[warp] = l;
    }
    __syncthreads();
    if (warp == 0 && lane < 16) {
      float top = -INFINITY, sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int y = 0; y < PER; ++y) top = fmaxf(top, merge->m[y]);
#pragma unroll
      for (int y = 0; y < PER; ++y) {
        const float fy = weight(merge->m[y], merge->l[y], top);
        sum += merge->l[y] * fy;
        const float4 z = merge->o[y][lane];
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

// tree_tc.cu: bf16, many rows a key head
bool tree_tc_serves(const TreeArgs& a);
cudaError_t launch_tree_tc(const TreeArgs& a, cudaStream_t stream);

}  // namespace fibattn
