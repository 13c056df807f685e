// Sparse decode of a tree of drafted tokens, bf16 with many query rows a key head (sm_103a): what tree.cu does row
// by row, on tensor cores.
//
// The nodes of a tree share most of their keys: at a rung of distance d the nodes of depths 0 .. D read the D + 1
// cached rows from len - d on, whatever their number, and the window's rows and the drafted ones are common.  A
// block (a sequence and key head, up to 64 query rows) therefore stages the union of the keys once, a few hundred
// rows, and forms S = Q' K'^T of all its rows against all of them: most products are not used, but a matrix
// product of 64 x 176 x 64 costs less than the row-by-row fetch, conversion and sum of 64 x 35 keys.  Each row then picks its
// scores (and blends an interpolated key's two: scores are linear in the key), and its weights go
// into a matrix of mostly zeros for O = P V.
//
//   mma.sync m16n8k16, keys (then dims) as the 16 rows, 8 query rows as the columns, as in tree_dense.cu; the query
//   and the drafted keys, rotated here, are split in three bf16 (24 bits: lse is float32, 1.3e-7 off; 16 bits left 1.9e-6), the
//   weights in two (O is rounded to 8 bits).
// A weight 0 times an infinity or NaN is NaN, so rows of which some value is not finite take the block to the
// row-by-row path, as do trees so deep that the union does not fit even for 8 rows at a time.
//
// What bounds it: the latency of a block's steps (lengths and tree; tables; pages; rows; products, weights, products), two
// blocks an SM by shared memory and registers: 64 sequences of 8 heads and 64 nodes are 512 blocks and take two rounds, 33.6
// us for a floor of 4.4 (issue slots 38% busy, tensor pipes 24%); 30.5 with query and drafts in two parts.
#include <algorithm>

#include "tree.cuh"

namespace fibattn {

namespace {

constexpr int kTtThreads = 256, kTtWarps = kTtThreads / 32;
constexpr int kTtRows = 8 * kTtWarps;   // query rows of a block: 8 a warp
constexpr int kTtMost = 304;            // staged rows a block may have

// Sizes of a call and byte offsets in dynamic shared memory (its base is 128-byte aligned).  So many staged rows that
// two blocks share an SM: the fewer query rows, the less room their scores take.
struct TtShape {
  int keys;    // staged rows, a multiple of 16
  int stride;  // 4-byte words of a row of S or P, 4 modulo 16: writes of a fragment meet no bank twice
  int v, lo, s, key, key_stride, bytes;
};
TtShape shape_of(int rows, int T, int keys) {
  TtShape p;
  const int r8 = rows < kTtRows ? (rows + 7) / 8 * 8 : kTtRows;
  p.keys = r8 <= 16 ? 304 : r8 <= 32 ? 240 : 176;
  p.stride = p.keys + 4;
  p.v = p.keys * 128;                         // K [keys][64], then V, 16-byte words swizzled by row
  p.lo = 2 * p.v;                             // the drafted keys' middle parts
  p.s = p.lo + (T + 15) / 16 * 16 * 128;      // [row][stride]: S, then P as hi | lo << 16, then O as bf16
  p.key = p.s + r8 * p.stride * 4;            // the drafted keys' lowest parts, then [row][key_stride]: weights by key
  p.key_stride = keys + 1;
  p.bytes = p.key + std::max(r8 * p.key_stride * 4, (T + 15) / 16 * 16 * 128);
  return p;
}

struct TtSmem {
  int4 key[kMaxKeys];  // distance, position it needs, weight of the second row, place (below)
  union {
    KeySmem ks;        // as built; again for the row-by-row path
    int from[kTtMost];  // of a staged cached row: which of the pools' rows it is
  };
  unsigned char line[kMaxDrafts][kMaxDrafts];  // [s][d]: the ancestor d levels above node s
  unsigned char by_distance[kMaxDrafts];       // first key that reads the row at a distance
  int first[kMaxR + 1], at[kMaxR + 2];         // of the window's run (0) and the rungs': first cached row, place among the staged
  int step;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf2_rn(x0, x1);
  lo = pack_bf2_rn(x0 - bf_lo(hi), x1 - bf_hi(hi));
}
// ... as hi + mid + lo
__device__ __forceinline__ void split3(float x0, float x1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_bf2_rn(x0, x1);
  split2(x0 - bf_lo(hi), x1 - bf_hi(hi), mid, lo);
}
// x as hi | lo << 16
__device__ __forceinline__ uint32_t split1(float x) {
  const __nv_bfloat16 hi = __float2bfloat16_rn(x), lo = __float2bfloat16_rn(x - __bfloat162float(hi));
  return static_cast<uint32_t>(__bfloat16_as_ushort(hi)) | static_cast<uint32_t>(__bfloat16_as_ushort(lo)) << 16;
}
// Whether a bf16 of the two is infinite or NaN.
__device__ __forceinline__ bool not_finite(uint32_t x) { return (~x & 0x7f80u) == 0 || (~x & 0x7f800000u) == 0; }
__device__ __forceinline__ bool not_finite(const uint4& x) { return not_finite(x.x) | not_finite(x.y) | not_finite(x.z) | not_finite(x.w); }

__global__ void __launch_bounds__(kTtThreads, 2) tree_tc_kernel(const __grid_constant__ TreeArgs a, int blocks_per_head,
                                                                     const __grid_constant__ TtShape shape) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(16) TtSmem ts;
  const int head = blockIdx.x / blocks_per_head, b = head / a.H, h = head % a.H;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  build_keys(a.t, a.N, &ts.ks);
  int n, len;
  bool ok = sequence_of(a, b, &n, &len);
  if (!ok) {
    if (tid == 0) atomicExch(a.status, kStatusDeviceAssert);
    return;
  }
  const int r0 = (blockIdx.x % blocks_per_head) * kTtRows, rows = min(kTtRows, n * a.G - r0);
  if (rows <= 0) return;
  const WarpTree tree = warp_tree(a, b, n, &ok);
  const int deepest = __reduce_max_sync(0xffffffffu, max(lane < n ? tree.depth[0] : 0, lane + 32 < n ? tree.depth[1] : 0));
  if (static_cast<long long>(len) + deepest >= a.N) ok = false;
  if (!ok) {  // (the same in all warps)
    if (tid == 0) atomicExch(a.status, kStatusDeviceAssert);
    return;
  }
  __syncthreads();
  const int W = a.t.W, nr = ts.ks.nr, nv = ts.ks.nv, drafts = (n + 15) & ~15;
  const uint32_t base = smem_addr(smem);
  bool bad = false;  // something staged is not finite

  // ---- on their way while the runs are planned: the query's words of row 8 warp + g, and a drafted row's 16 dims
  const int qr = 8 * warp + g;
  const int q_head = qr < rows ? (r0 + qr) / n : 0, q_node = qr < rows ? (r0 + qr) - q_head * n : 0;
  const size_t q_row = (static_cast<size_t>(b) * a.Hq + h * a.G + q_head) * a.T + q_node;
  const int depth = pick32(tree.depth, q_node), pos = len + depth;  // of this lane's row, here and below
  uint32_t qx[2][2], qy[2][2];
  {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) + q_row * kD) + t;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        qx[k][f] = __ldg(q + 8 * k + 4 * f);
        qy[k][f] = __ldg(q + 8 * k + 4 * f + kFreq / 2);
      }
  }
  const int du = tid >> 2;  // 64 quads: every drafted row at once
  const int d_pos = len + pick32(tree.depth, du);
  uint4 dk[2], dv[2];
  dk[0] = dk[1] = dv[0] = dv[1] = make_uint4(0, 0, 0, 0);
  if (du < n) {
    const size_t at = ((static_cast<size_t>(b) * a.H + h) * a.T + du) * kD;
    const uint4* kr = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.kn) + at);
    const uint4* vr = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.vn) + at);
    dk[0] = __ldg(kr + t);
    dk[1] = __ldg(kr + t + 4);
    dv[0] = __ldg(vr + t);
    dv[1] = __ldg(vr + t + 4);
  }

  // The union of the cached rows of `step` query rows from `from` on: its runs' places; returns the number of staged
  // rows.  By one warp: lane c has run c (0: the window, c: rung c - 1).  key(c): distance and weight of key c.
  auto plan_runs = [&](int from, int step, auto&& key) {
    int lowest = 64, highest = 0;
    for (int x = from; x < min(from + step, rows); x += 32) {
      const int r = min(x + lane, rows - 1), d = pick32(tree.depth, (r0 + r) % n);
      if (x + lane < min(from + step, rows)) {
        lowest = min(lowest, d);
        highest = max(highest, d);
      }
    }
    lowest = __reduce_min_sync(0xffffffffu, lowest);
    highest = __reduce_max_sync(0xffffffffu, highest);
    int total = drafts;
    for (int c0 = 0; c0 <= nr; c0 += 32) {
      const int c = c0 + lane;
      int first = 0, count = 0;
      if (c == 0) {
        first = max(0, len + lowest - (W - 1));
        count = max(0, len - first);
      } else if (c <= nr) {
        float w;
        const int lo = key(W + c - 1, w), two = w > 0.f ? 1 : 0;
        first = max(0, len + lowest - lo - two);
        count = max(0, min(len - 1, len + highest - lo) - first + 1);
      }
      int at = count;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, at, x);
        if (lane >= x) at += y;
      }
      if (c <= nr) {
        ts.first[c] = first;
        ts.at[c] = total + at - count;
      }
      total += __shfl_sync(0xffffffffu, at, 31);
    }
    if (lane == 0) ts.at[nr + 1] = total;
    return total;
  };
  // the tables, a warp or two each: nodes, runs, distances, keys
  if (warp < 2) {  // node `tid`
    if (tid < n) {
      uint64_t left = tree.above[warp];
      for (int d = 0; left != 0; ++d) {
        const int u = 63 - __clzll(static_cast<long long>(left));
        ts.line[tid][d] = static_cast<unsigned char>(u);
        left &= ~(1ull << u);
      }
    }
  } else if (warp == 2) {  // the most rows at a time whose union fits, in two steps at most (more leave most warps idle too long)
    int step = kTtRows;
    for (; step >= 8 && 2 * step >= rows; step >>= 1) {
      bool fits = true;
      for (int from = 0; from < rows && fits; from += step) fits = plan_runs(from, step, [&](int c, float& w) {
          w = ts.ks.w[c];
          return ts.ks.lo[c];
        }) <= shape.keys;
      if (fits) break;
    }
    if (lane == 0) ts.step = step >= 8 && 2 * step >= rows ? step : 0;
  } else if (warp < 5) {  // the first key that reads the row at distance d: keys are in the order of lo, and read lo and lo + 1
    const int d = tid - 96;
    int c = 0, end = nv;
    while (c < end) {
      const int mid = (c + end) >> 1;
      if (ts.ks.lo[mid] + 1 < d)
        c = mid + 1;
      else
        end = mid;
    }
    ts.by_distance[d] = static_cast<unsigned char>(c);
  } else {
    for (int c = tid - 160; c < nv; c += kTtThreads - 160) ts.key[c] = make_int4(ts.ks.lo[c], ts.ks.need[c], __float_as_int(ts.ks.w[c]), 0);
  }

  // ---- query fragments (hi, mid, lo) of the warp's 8 rows, in registers
  uint32_t qh[4][2], qm[4][2], ql[4][2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int d = 16 * k + 8 * f + 2 * t;
      const float2 e0 = rope_factor(a.rope_lo, a.rope_hi, pos, d), e1 = rope_factor(a.rope_lo, a.rope_hi, pos, d + 1);
      const float sc = kLog2e / 8.0f;
      const float x0 = bf_lo(qx[k][f]) * sc, x1 = bf_hi(qx[k][f]) * sc, y0 = bf_lo(qy[k][f]) * sc, y1 = bf_hi(qy[k][f]) * sc;
      split3(x0 * e0.x - y0 * e0.y, x1 * e1.x - y1 * e1.y, qh[k][f], qm[k][f], ql[k][f]);
      split3(x0 * e0.y + y0 * e0.x, x1 * e1.y + y1 * e1.x, qh[k + 2][f], qm[k + 2][f], ql[k + 2][f]);
    }
  // ---- drafted rows: K rotated, hi in the K tile, mid and lo apart; zeros behind the last
  auto stage_draft = [&](const uint4 (&kr)[2], bool again) {  // (again: lo alone, whose room the weights have taken)
    uint32_t hi[8], mid[8], lo[8];
    float x[16];
    float2 e[8];
    const uint32_t w[8] = {kr[0].x, kr[0].y, kr[0].z, kr[0].w, kr[1].x, kr[1].y, kr[1].z, kr[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = bf_lo(w[i]);
      x[2 * i + 1] = bf_hi(w[i]);
    }
    rope_row(a.rope_lo, a.rope_hi, du < n ? d_pos : 0, t, e);
    rotate_part(x, e, false);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      split3(x[2 * i], x[2 * i + 1], hi[i], mid[i], lo[i]);
      bad |= not_finite(hi[i]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = du * 128 + (((t + 4 * i) ^ (du & 7)) << 4);
      *reinterpret_cast<uint4*>(smem + shape.key + at) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
      if (again) continue;
      *reinterpret_cast<uint4*>(smem + at) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
      *reinterpret_cast<uint4*>(smem + shape.lo + at) = make_uint4(mid[4 * i], mid[4 * i + 1], mid[4 * i + 2], mid[4 * i + 3]);
    }
  };
  if (du < drafts) {
    stage_draft(dk, false);
    bad |= not_finite(dv[0]) | not_finite(dv[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<uint4*>(smem + shape.v + du * 128 + (((t + 4 * i) ^ (du & 7)) << 4)) = dv[i];
  }
  __syncthreads();
  const int step = ts.step;

  int from = 0;
  for (; from < rows && step > 0; from += step) {
    if (step < rows) {  // (else the plan of the only step stands)
      __syncthreads();
      if (warp == 0)
        plan_runs(from, step, [&](int c, float& w) {
          w = __int_as_float(ts.key[c].z);
          return ts.key[c].x;
        });
      if (from > 0 && du < drafts) {
        uint4 kr[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (du < n) {
          const size_t at = ((static_cast<size_t>(b) * a.H + h) * a.T + du) * kD;
          const uint4* row = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.kn) + at);
          kr[0] = __ldg(row + t);
          kr[1] = __ldg(row + t + 4);
        }
        stage_draft(kr, true);
      }
      __syncthreads();
    }
    const int total = ts.at[nr + 1], padded = (total + 15) & ~15;
    // ---- where the staged rows lie; the keys as the rows below read them: at position p, key c's row lies at place + p
    // among the staged (its second one in front of that)
    for (int x = drafts + tid; x < total; x += kTtThreads) {
      int c = 0, end = nr + 1;  // the run: at[c] <= x < at[c + 1]
      while (end - c > 1) {
        const int mid = (c + end) >> 1;
        if (ts.at[mid] <= x)
          c = mid;
        else
          end = mid;
      }
      long long at = cache_row(a, b, h, ts.first[c] + x - ts.at[c]);
      if (at < 0) {
        atomicExch(a.status, kStatusDeviceAssert);
        at = 0;
      }
      ts.from[x] = static_cast<int>(at / kD);
    }
    if (tid < nv) {
      const int run = tid < W ? 0 : tid - W + 1;
      ts.key[tid].w = ts.at[run] - ts.first[run] - ts.key[tid].x;
    }
    __syncthreads();
    // ---- the cached rows, 192 on their way at once
    for (int x0 = drafts; x0 < padded; x0 += 6 * (kTtThreads / 8)) {
      uint4 k[6], v[6];
#pragma unroll
      for (int j = 0; j < 6; ++j) {
        const int x = x0 + j * (kTtThreads / 8) + (tid >> 3), ch = tid & 7;
        k[j] = v[j] = make_uint4(0, 0, 0, 0);
        if (x < total) {
          const size_t at = static_cast<size_t>(ts.from[x]) * kD;
          k[j] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.kc) + at) + ch);
          v[j] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.vc) + at) + ch);
        }
      }
#pragma unroll
      for (int j = 0; j < 6; ++j) {
        const int x = x0 + j * (kTtThreads / 8) + (tid >> 3), ch = tid & 7;
        bad |= not_finite(k[j]) | not_finite(v[j]);
        if (x < padded) {
          const int to = x * 128 + ((ch ^ (x & 7)) << 4);
          *reinterpret_cast<uint4*>(smem + to) = k[j];
          *reinterpret_cast<uint4*>(smem + shape.v + to) = v[j];
        }
      }
    }
    if (__syncthreads_or(bad)) break;  // the rows from here on one by one

    // ---- 8 query rows a warp
    const bool takes = 8 * warp >= from && 8 * warp < min(from + step, rows);
    const int mi = lane >> 3, rl = lane & 7, stride = shape.stride;
    uint32_t* S = reinterpret_cast<uint32_t*>(smem + shape.s) + 8 * warp * stride;
    if (takes) {
#pragma unroll 2
      for (int x0 = 0; x0 < padded; x0 += 16) {
        float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}}, d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const uint32_t row = base + (x0 + (mi & 1) * 8 + rl) * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t ka[4];
          const uint32_t word = ((2 * k + (mi >> 1)) ^ rl) << 4;
          ldsm4(ka, row + word);
          mma16(c[k & 1], ka, qh[k][0], qh[k][1]);
          mma16(d[k & 1], ka, ql[k][0], ql[k][1]);
          mma16(d[k & 1], ka, qm[k][0], qm[k][1]);
        }
        if (x0 < drafts) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t ka[4];
            const uint32_t word = ((2 * k + (mi >> 1)) ^ rl) << 4;
            ldsm4(ka, row + shape.key + word);
            mma16(d[k & 1], ka, qh[k][0], qh[k][1]);
            ldsm4(ka, row + shape.lo + word);
            mma16(d[k & 1], ka, qm[k][0], qm[k][1]);
            mma16(d[k & 1], ka, qh[k][0], qh[k][1]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          S[(2 * t + (e & 1)) * stride + x0 + g + 8 * (e >> 1)] = __float_as_uint((c[0][e] + c[1][e]) + (d[0][e] + d[1][e]));
      }
    }
    __syncthreads();  // the drafted keys' lowest parts are read; from here on a warp keeps to its own rows
    if (takes) {
      // weights: 4 lanes a row (this lane's: g), keys t, t + 4, ...
      const bool in = qr < rows;
      uint32_t* row = S + g * stride;
      float* key = reinterpret_cast<float*>(smem + shape.key) + qr * shape.key_stride;
      const unsigned char* line = ts.line[q_node];
      float m = -INFINITY;
      for (int c0 = t; c0 < nv; c0 += 16) {  // scores by key, four at a time: every read before a write
        float x[4], y[4], w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // (no branches: both rows' places are looked up for every key, in bounds where it is none)
          const int4 kk = ts.key[min(c0 + 4 * j, nv - 1)];
          const bool on = in && c0 + 4 * j < nv && pos >= kk.y;
          const int above0 = line[min(kk.x, kMaxDrafts - 1)], above1 = line[min(kk.x + 1, kMaxDrafts - 1)];
          const int at0 = kk.x <= depth ? above0 : kk.w + pos, at1 = kk.x < depth ? above1 : kk.w + pos - 1;
          w[j] = on ? __int_as_float(kk.z) : 0.f;
          x[j] = __uint_as_float(row[on ? at0 : 0]);
          y[j] = __uint_as_float(row[w[j] > 0.f ? at1 : 0]);
          if (!on) x[j] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (w[j] > 0.f) x[j] = (1.f - w[j]) * x[j] + w[j] * y[j];
          if (c0 + 4 * j < nv) key[c0 + 4 * j] = x[j];
          m = fmaxf(m, x[j]);
        }
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      __syncwarp();
      for (int x = t; x < padded / 4; x += 4) reinterpret_cast<uint4*>(row)[x] = make_uint4(0, 0, 0, 0);
      __syncwarp();
      float l = 0.f;
      for (int c0 = t; c0 < nv; c0 += 16) {
        float p[4];
        int4 kk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          kk[j] = ts.key[min(c0 + 4 * j, nv - 1)];
          p[j] = c0 + 4 * j < nv ? ex2(key[min(c0 + 4 * j, nv - 1)] - m) : 0.f;  // (of a row that is none NaN, which nobody reads)
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float w = __int_as_float(kk[j].z);
          l += p[j];
          if (c0 + 4 * j >= nv) continue;
          key[c0 + 4 * j] = p[j];
          // a cached row of a run is this key's alone
          if (in && pos >= kk[j].y) {
            if (kk[j].x > depth) row[kk[j].w + pos] = split1(p[j] * (1.f - w));
            if (w > 0.f && kk[j].x >= depth) row[kk[j].w + pos - 1] = split1(p[j] * w);
          }
        }
      }
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      __syncwarp();
      // a drafted row may be several keys': their sum in the order of the keys
      if (in)
        for (int d = t; d <= depth; d += 4) {
          float x = 0.f;
          for (int c = ts.by_distance[d], more = 1; more; c += 3) {  // seldom more than two: three at a time
#pragma unroll
            for (int j = 0; j < 3; ++j) {
              const int at = min(c + j, nv - 1);
              const int4 kk = ts.key[at];
              const float w = __int_as_float(kk.z), p = key[at] * (kk.x == d ? 1.f - w : w);
              more = c + j < nv && kk.x <= d;
              if (more) x += p;
            }
          }
          row[line[d]] = split1(x);
        }
      const float inv = 1.f / l;
      if (in && t == 0 && a.lse != nullptr) a.lse[q_row] = (m + log2f(l)) * kLn2;
      __syncwarp();
      // O^T = V^T P^T, 16 dims at a time
      float c[4][4], d[4][4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[x][e] = d[x][e] = 0.f;
#pragma unroll 2
      for (int x0 = 0; x0 < padded; x0 += 16) {
        const uint2 p = *reinterpret_cast<const uint2*>(row + x0 + 2 * t), q = *reinterpret_cast<const uint2*>(row + x0 + 2 * t + 8);
        const uint32_t h0 = __byte_perm(p.x, p.y, 0x5410), h1 = __byte_perm(q.x, q.y, 0x5410);
        const uint32_t l0 = __byte_perm(p.x, p.y, 0x7632), l1 = __byte_perm(q.x, q.y, 0x7632);
        const uint32_t vr = base + shape.v + (x0 + (mi >> 1) * 8 + rl) * 128;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t va[4];
          ldsm4_t(va, vr + (((2 * x + (mi & 1)) ^ rl) << 4));
          mma16(c[x], va, h0, h1);
          mma16(d[x], va, l0, l1);
        }
      }
      __syncwarp();
      // rows 2t, 2t + 1 of the fragments; their 1 / l from the lanes that have them
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(S);
      const float inv0 = __shfl_sync(0xffffffffu, inv, 8 * t), inv1 = __shfl_sync(0xffffffffu, inv, 8 * t + 4);
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          out[(2 * t + (e & 1)) * 72 + 16 * x + g + 8 * (e >> 1)] = __float2bfloat16_rn((c[x][e] + d[x][e]) * (e & 1 ? inv1 : inv0));
      __syncwarp();
      if (in) {
        uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + q_row * kD);
        to[t] = *reinterpret_cast<const uint4*>(out + g * 72 + 8 * t);
        to[t + 4] = *reinterpret_cast<const uint4*>(out + g * 72 + 8 * t + 32);
      }
    }
  }
  if (from >= rows) return;
  // ---- what is left, row by row
  __syncthreads();
  build_keys(a.t, a.N, &ts.ks);
  const WarpTree again = warp_tree(a, b, n, &ok);
  __syncthreads();
  for (int r = from + warp; r < rows; r += kTtWarps) {
    const int hq = (r0 + r) / n, s = (r0 + r) - hq * n, d = pick32(again.depth, s);
    attend_row<__nv_bfloat16, 1>(a, &ts.ks, b, h, (static_cast<size_t>(b) * a.Hq + h * a.G + hq) * a.T + s, d, len + d, pick64(again.above, s), 0,
                                 nullptr);
  }
}

}  // namespace

// A round of 304 blocks takes some 8 us at least, whatever their rows; row by row takes 4.5 us and 2.5 ns a row of the whole
// batch (interpolated; 2.1 where the keys are rows).  Measured on such keys (us here, row by row): 512 blocks of 64 rows 31 and 72, of
// 16 rows 17.7 and 21.0, of 12 rows 17.5 and 16.2, of 8 rows 16.6 and 11.7; 256 blocks of 16 rows 9.9 and 12.1; 128 blocks of 32 rows
// 9.0 and 12.1, of 16 rows 8.4 and 7.0; 64 blocks of 64 rows 11.6 and 12.3; 32 blocks of 64 rows 11.4 and 7.1.
// A chain's union grows with its length: it fits for 12 nodes of the Fibonacci base's distances, more are served row by
// row.  (Deep trees that are given by their parents are found on the device only; they take 1.3 times the time then.)
bool tree_tc_serves(const TreeArgs& a) {
  if (a.parent == nullptr && a.T > 12) return false;
  const long long heads = static_cast<long long>(a.B) * a.H, blocks = heads * ((a.G * a.T + kTtRows - 1) / kTtRows);
  return heads * a.G * a.T > 2800 * ((blocks + 303) / 304) - 400;
}

cudaError_t launch_tree_tc(const TreeArgs& a, cudaStream_t stream) {
  const int per = (a.G * a.T + kTtRows - 1) / kTtRows;
  const TtShape shape = shape_of(a.G * a.T, a.T, a.t.W + a.t.n);
  const cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (e != cudaSuccess) return e;
  const long long blocks = static_cast<long long>(a.B) * a.H * per;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  tree_tc_kernel<<<static_cast<unsigned>(blocks), kTtThreads, shape.bytes, stream>>>(a, per, shape);
  return cudaGetLastError();
}

}  // namespace fibattn
