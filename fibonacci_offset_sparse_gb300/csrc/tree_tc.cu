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
//   mma.sync m16n8k16, keys (then dims) as the 16 rows, 8 query rows as the columns, as in tree_dense.cu; the query,
//   the weights and the drafted keys (rotated here) are split in two bf16, hi + lo.
// A weight 0 times an infinity or NaN is NaN, so rows of which some value is not finite take the block to the
// row-by-row path, as do trees so deep that the union does not fit even for 8 rows at a time.
//
// What bounds it: the latency of a block's steps (lengths and tree; pages; rows; three phases between barriers), two
// blocks an SM; the tensor work is a quarter of that.
#include "tree.cuh"

namespace fibattn {

namespace {

constexpr int kTtThreads = 256, kTtWarps = kTtThreads / 32;
constexpr int kTtRows = 64;                // query rows of a block
constexpr int kTtPass = 32;                // ... of a pass between barriers
constexpr int kTtKeys = 192;               // staged rows, a multiple of 16
constexpr int kTtStride = kTtKeys + 4;     // 4-byte words of a row of S or P: writes of a fragment meet no bank twice
constexpr int kTtLow = 64;                 // rows of the drafted keys' lower parts

// byte offsets in dynamic shared memory (its base is 128-byte aligned)
constexpr int kTtK = 0;
constexpr int kTtV = kTtK + kTtKeys * 128;
constexpr int kTtLo = kTtV + kTtKeys * 128;
constexpr int kTtQ = kTtLo + kTtLow * 128;                 // fragments: [8 rows][k-step][lane] hi, hi, lo, lo
constexpr int kTtS = kTtQ + kTtRows / 8 * 2048;            // [kTtPass][kTtStride]: S, then P as hi | lo << 16
constexpr int kTtOut = kTtS + kTtPass * kTtStride * 4;     // [kTtPass][72] bf16
constexpr int kTtKey = kTtOut + kTtPass * 144;             // [kTtPass][keys + 1]: weights by key
size_t tt_bytes(int keys) { return kTtKey + static_cast<size_t>(kTtPass) * (keys + 1) * 4; }

struct TtSmem {
  KeySmem ks;
  int depth[kMaxDrafts];
  uint64_t above[kMaxDrafts];
  int first[kMaxR + 1], at[kMaxR + 2];  // of the window's run (0) and the rungs': first cached row, place among the staged
  int by_distance[kMaxDrafts];          // first key that reads the row at a distance
  int lowest, highest;                  // depths of a step's nodes
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
// x as hi | lo << 16
__device__ __forceinline__ uint32_t split1(float x) {
  const __nv_bfloat16 hi = __float2bfloat16_rn(x), lo = __float2bfloat16_rn(x - __bfloat162float(hi));
  return static_cast<uint32_t>(__bfloat16_as_ushort(hi)) | static_cast<uint32_t>(__bfloat16_as_ushort(lo)) << 16;
}
// Whether a bf16 of the two is infinite or NaN.
__device__ __forceinline__ bool not_finite(uint32_t x) { return (~x & 0x7f80u) == 0 || (~x & 0x7f800000u) == 0; }
__device__ __forceinline__ bool not_finite(const uint4& x) { return not_finite(x.x) | not_finite(x.y) | not_finite(x.z) | not_finite(x.w); }

__global__ void __launch_bounds__(kTtThreads, 2) tree_tc_kernel(const __grid_constant__ TreeArgs a, int blocks_per_head, int key_stride) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ TtSmem ts;
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
  const WarpTree tree = warp_tree(a.parent == nullptr ? nullptr : a.parent + static_cast<size_t>(b) * a.T, n, &ok);
  const int deepest = __reduce_max_sync(0xffffffffu, max(lane < n ? tree.depth[0] : 0, lane + 32 < n ? tree.depth[1] : 0));
  if (static_cast<long long>(len) + deepest >= a.N) ok = false;
  if (!ok) {  // (the same in all warps)
    if (tid == 0) atomicExch(a.status, kStatusDeviceAssert);
    return;
  }
  if (warp == 0)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ts.depth[lane + 32 * i] = tree.depth[i];
      ts.above[lane + 32 * i] = tree.above[i];
    }
  __syncthreads();
  const int W = a.t.W, nr = ts.ks.nr, nv = ts.ks.nv, drafts = (n + 15) & ~15;
  const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(a.kc);
  const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(a.vc);
  const uint32_t base = smem_addr(smem);
  float* s_key = reinterpret_cast<float*>(smem + kTtKey);
  bool bad = false;  // something staged is not finite

  // ---- query fragments of all rows: lane (g, t) of warp w the row 8 w + g
  if (8 * warp < rows) {
    const int r = 8 * warp + g;
    uint4* at = reinterpret_cast<uint4*>(smem + kTtQ) + warp * 128 + lane;
    if (r < rows) {
      const int hq = (r0 + r) / n, s = (r0 + r) - hq * n, pos = len + ts.depth[s];
      const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                            ((static_cast<size_t>(b) * a.Hq + h * a.G + hq) * a.T + s) * kD);
      uint32_t qh[4][2], ql[4][2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int d = 16 * k + 8 * f + 2 * t;
          const uint32_t x = __ldg(q + d / 2), y = __ldg(q + d / 2 + kFreq / 2);
          const float2 e0 = rope_factor(a.rope_lo, a.rope_hi, pos, d), e1 = rope_factor(a.rope_lo, a.rope_hi, pos, d + 1);
          const float sc = kLog2e / 8.0f;
          const float x0 = bf_lo(x) * sc, x1 = bf_hi(x) * sc, y0 = bf_lo(y) * sc, y1 = bf_hi(y) * sc;
          split2(x0 * e0.x - y0 * e0.y, x1 * e1.x - y1 * e1.y, qh[k][f], ql[k][f]);
          split2(x0 * e0.y + y0 * e0.x, x1 * e1.y + y1 * e1.x, qh[k + 2][f], ql[k + 2][f]);
        }
#pragma unroll
      for (int k = 0; k < 4; ++k) at[32 * k] = make_uint4(qh[k][0], qh[k][1], ql[k][0], ql[k][1]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) at[32 * k] = make_uint4(0, 0, 0, 0);
    }
  }
  // ---- drafted rows: K rotated, hi in the K tile and lo apart; a quad a row, zeros behind the last
  for (int u = tid >> 2; u < drafts; u += kTtThreads / 4) {
    uint32_t hi[8], lo[8];
    uint4 v[2];
    if (u < n) {
      const size_t from = ((static_cast<size_t>(b) * a.H + h) * a.T + u) * kD;
      float x[16];
      float2 e[8];
      load_part(static_cast<const __nv_bfloat16*>(a.kn) + from, t, x);
      const uint4* vr = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.vn) + from);
      v[0] = __ldg(vr + t);
      v[1] = __ldg(vr + t + 4);
      rope_row(a.rope_lo, a.rope_hi, len + ts.depth[u], t, e);
      rotate_part(x, e, false);
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        split2(x[2 * w], x[2 * w + 1], hi[w], lo[w]);
        bad |= not_finite(hi[w]);
      }
      bad |= not_finite(v[0]) | not_finite(v[1]);
    } else {
      v[0] = v[1] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < 8; ++w) hi[w] = lo[w] = 0;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int at = u * 128 + (((t + 4 * x) ^ (u & 7)) << 4);
      *reinterpret_cast<uint4*>(smem + kTtK + at) = make_uint4(hi[4 * x], hi[4 * x + 1], hi[4 * x + 2], hi[4 * x + 3]);
      *reinterpret_cast<uint4*>(smem + kTtLo + at) = make_uint4(lo[4 * x], lo[4 * x + 1], lo[4 * x + 2], lo[4 * x + 3]);
      *reinterpret_cast<uint4*>(smem + kTtV + at) = v[x];
    }
  }
  // ---- the first key that reads the row at distance d: keys are in the order of lo, and read lo and lo + 1
  if (tid < kMaxDrafts) {
    int c = 0;
    while (c < nv && ts.ks.lo[c] + 1 < tid) ++c;
    ts.by_distance[tid] = c;
  }

  // The union of the cached rows of `step` query rows from `from` on: its runs' places (thread c < nr + 1 of warp 0 holds
  // run c); the number of staged rows.  By warp 0.
  auto plan_runs = [&](int from, int step) {
    int lowest = 64, highest = 0;
    for (int r = from + lane; r < min(from + step, rows); r += 32) {
      const int d = ts.depth[(r0 + r) % n];
      lowest = min(lowest, d);
      highest = max(highest, d);
    }
    lowest = __reduce_min_sync(0xffffffffu, lowest);
    highest = __reduce_max_sync(0xffffffffu, highest);
    int total = drafts;
    for (int c0 = 0; c0 <= nr; c0 += 32) {  // run 0: the window; run c: rung c - 1
      const int c = c0 + lane;
      int first = 0, count = 0;
      if (c == 0) {
        first = max(0, len + lowest - (W - 1));
        count = max(0, len - first);
      } else if (c <= nr) {
        const int lo = ts.ks.lo[W + c - 1], two = ts.ks.w[W + c - 1] > 0.f ? 1 : 0;
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
  // The most rows at a time whose union fits
  __shared__ int s_step;
  if (warp == 0) {
    int step = kTtRows;
    for (; step >= 8; step >>= 1) {
      bool fits = true;
      for (int from = 0; from < rows && fits; from += step) fits = plan_runs(from, step) <= kTtKeys;
      if (fits) break;
    }
    if (lane == 0) s_step = step;
  }
  __syncthreads();
  const int step = s_step;

  int from = 0;
  for (; from < rows && step >= 8; from += step) {
    if (step < rows) {  // (else the plan of the only step stands)
      __syncthreads();
      if (warp == 0) plan_runs(from, step);
      __syncthreads();
    }
    const int total = ts.at[nr + 1], padded = (total + 15) & ~15;
    // ---- the cached rows, eight 16-byte words of K and of V each
    for (int i = drafts * 8 + tid; i < padded * 8; i += kTtThreads) {
      const int x = i >> 3, ch = i & 7;
      uint4 k = make_uint4(0, 0, 0, 0), v = k;
      if (x < total) {
        int c = 0;  // its run
        while (ts.at[c + 1] <= x) ++c;
        long long at = cache_row(a, b, h, ts.first[c] + x - ts.at[c]);
        if (at < 0) {
          atomicExch(a.status, kStatusDeviceAssert);
          at = 0;
        }
        k = __ldg(reinterpret_cast<const uint4*>(kc + at) + ch);
        v = __ldg(reinterpret_cast<const uint4*>(vc + at) + ch);
        bad |= not_finite(k) | not_finite(v);
      }
      const int to = x * 128 + ((ch ^ (x & 7)) << 4);
      *reinterpret_cast<uint4*>(smem + kTtK + to) = k;
      *reinterpret_cast<uint4*>(smem + kTtV + to) = v;
    }
    if (__syncthreads_or(bad)) break;  // the rows from here on one by one

    for (int p0 = from; p0 < min(from + step, rows); p0 += kTtPass) {
      const int p1 = min(min(p0 + kTtPass, from + step), rows);  // a pass: rows [p0, p1)
      const int tiles = (p1 - p0 + 7) >> 3, mi = lane >> 3, rl = lane & 7;
      uint32_t* S = reinterpret_cast<uint32_t*>(smem + kTtS);
      // ---- scores: an item is 16 keys against 16 query rows
      for (int item = warp; item < padded / 16 * 2; item += kTtWarps) {
        const int x0 = (item >> 1) * 16, n0 = (item & 1) * 2;
        if (n0 >= tiles) continue;
        float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}}, d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const uint32_t row = (x0 + (mi & 1) * 8 + rl) * 128;
        const uint4* qs = reinterpret_cast<const uint4*>(smem + kTtQ) + ((p0 >> 3) + n0) * 128 + lane;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t ka[4];
          const uint32_t word = ((2 * k + (mi >> 1)) ^ rl) << 4;
          ldsm4(ka, base + kTtK + row + word);
          const uint4 q0 = qs[32 * k], q1 = qs[128 + 32 * k];  // (tiles behind the last are not used)
          mma16(c[0], ka, q0.x, q0.y);
          mma16(c[1], ka, q1.x, q1.y);
          mma16(d[0], ka, q0.z, q0.w);
          mma16(d[1], ka, q1.z, q1.w);
          if (x0 < drafts) {
            ldsm4(ka, base + kTtLo + row + word);
            mma16(d[0], ka, q0.x, q0.y);
            mma16(d[1], ka, q1.x, q1.y);
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            S[(8 * (n0 + j) + 2 * t + (e & 1)) * kTtStride + x0 + g + 8 * (e >> 1)] = __float_as_uint(c[j][e] + d[j][e]);
      }
      __syncthreads();
      // ---- weights: 8 lanes a row
      {
        const int pr = tid >> 3, l8 = tid & 7, r = p0 + pr;
        const bool in = r < p1;
        const int hq = in ? (r0 + r) / n : 0, s = in ? (r0 + r) - hq * n : 0, depth = ts.depth[s], pos = len + depth;
        uint32_t* row = S + pr * kTtStride;
        // where the row at distance dist lies among the staged, read by key c
        auto place = [&](int c, int dist) {
          if (dist <= depth) return ancestor_at(ts.above[s], dist);
          const int run = c < W ? 0 : c - W + 1;
          return ts.at[run] + pos - dist - ts.first[run];
        };
        float sc[kMaxKeys / 8], m = -INFINITY;
#pragma unroll
        for (int j = 0; j < kMaxKeys / 8; ++j) {
          const int c = 8 * j + l8;
          sc[j] = -INFINITY;
          if (8 * j >= nv) continue;  // (uniform, as below)
          if (in && c < nv && pos >= ts.ks.need[c]) {
            const int lo = ts.ks.lo[c];
            const float w = ts.ks.w[c];
            sc[j] = __uint_as_float(row[place(c, lo)]);
            if (w > 0.f) sc[j] = (1.f - w) * sc[j] + w * __uint_as_float(row[place(c, lo + 1)]);
          }
          m = fmaxf(m, sc[j]);
        }
#pragma unroll
        for (int x = 1; x < 8; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        float l = 0.f;
#pragma unroll
        for (int j = 0; j < kMaxKeys / 8; ++j) {
          if (8 * j >= nv) break;
          sc[j] = exp2f(sc[j] - m);  // (a row has its own key at least; of a row that is none, NaN that nobody reads)
          l += sc[j];
        }
#pragma unroll
        for (int x = 1; x < 8; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        const float inv = 1.f / l;
        __syncwarp();
        for (int x = l8; x < padded / 4; x += 8) reinterpret_cast<uint4*>(row)[x] = make_uint4(0, 0, 0, 0);
        __syncwarp();
        float* key = s_key + pr * key_stride;
#pragma unroll
        for (int j = 0; j < kMaxKeys / 8; ++j) {
          if (8 * j >= nv) break;
          const int c = 8 * j + l8;
          if (in && c < nv) {
            const bool on = pos >= ts.ks.need[c];
            const float p = on ? sc[j] * inv : 0.f, w = ts.ks.w[c];
            const int lo = ts.ks.lo[c];
            key[c] = p;
            // a cached row of a run is this key's alone
            if (on && lo > depth) row[place(c, lo)] = split1(p * (1.f - w));
            if (on && w > 0.f && lo + 1 > depth) row[place(c, lo + 1)] = split1(p * w);
          }
        }
        __syncwarp();
        // a drafted row may be several keys': their sum in the order of the keys
        if (in)
          for (int d = l8; d <= depth; d += 8) {
            float x = 0.f;
            for (int c = ts.by_distance[d]; c < nv && ts.ks.lo[c] <= d; ++c) {
              const float w = ts.ks.w[c];
              x += key[c] * (ts.ks.lo[c] == d ? 1.f - w : w);
            }
            row[ancestor_at(ts.above[s], d)] = split1(x);
          }
        if (in && l8 == 0 && a.lse != nullptr)
          a.lse[(static_cast<size_t>(b) * a.Hq + h * a.G + hq) * a.T + s] = (m + log2f(l)) * kLn2;
      }
      __syncthreads();
      // ---- O^T = V^T P^T: warp w the dims 16 (w % 4) .. and the query rows 16 (w / 4) ..
      {
        const int d0 = 16 * (warp & 3), n0 = (warp >> 2) * 2;
        float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}}, d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        if (n0 < tiles) {
          for (int x0 = 0; x0 < padded; x0 += 16) {
            uint32_t va[4];
            ldsm4_t(va, base + kTtV + (x0 + (mi >> 1) * 8 + rl) * 128 + (((d0 / 8 + (mi & 1)) ^ rl) << 4));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t* row = S + (8 * (n0 + j) + g) * kTtStride + x0 + 2 * t;
              const uint2 p = *reinterpret_cast<const uint2*>(row), q = *reinterpret_cast<const uint2*>(row + 8);
              mma16(c[j], va, __byte_perm(p.x, p.y, 0x5410), __byte_perm(q.x, q.y, 0x5410));
              mma16(d[j], va, __byte_perm(p.x, p.y, 0x7632), __byte_perm(q.x, q.y, 0x7632));
            }
          }
          __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(smem + kTtOut);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              out[(8 * (n0 + j) + 2 * t + (e & 1)) * 72 + d0 + g + 8 * (e >> 1)] = __float2bfloat16_rn(c[j][e] + d[j][e]);
        }
      }
      __syncthreads();
      {
        const int pr = tid >> 3, ch = tid & 7, r = p0 + pr;
        if (r < p1) {
          const int hq = (r0 + r) / n, s = (r0 + r) - hq * n;
          reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + ((static_cast<size_t>(b) * a.Hq + h * a.G + hq) * a.T + s) * kD)[ch] =
              *reinterpret_cast<const uint4*>(smem + kTtOut + pr * 144 + ch * 16);
        }
      }
    }
  }
  // ---- what is left, row by row
  for (int r = from + warp; r < rows; r += kTtWarps) {
    const int hq = (r0 + r) / n, s = (r0 + r) - hq * n, depth = ts.depth[s];
    attend_row<__nv_bfloat16, 1>(a, &ts.ks, b, h, (static_cast<size_t>(b) * a.Hq + h * a.G + hq) * a.T + s, depth, len + depth, ts.above[s], 0,
                                 nullptr);
  }
}

}  // namespace

// From 16 query rows a key head on (measured, 512 heads of a batch: 8 rows 00 us here and 00 row by row, 16 rows 00 and 00).
bool tree_tc_serves(const TreeArgs& a) { return a.G * a.T >= 16; }

cudaError_t launch_tree_tc(const TreeArgs& a, cudaStream_t stream) {
  const int per = (a.G * a.T + kTtRows - 1) / kTtRows, keys = a.t.W + a.t.n;
  const size_t smem = tt_bytes(keys);
  const cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(tt_bytes(kMaxKeys)));
  if (e != cudaSuccess) return e;
  const long long blocks = static_cast<long long>(a.B) * a.H * per;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  tree_tc_kernel<<<static_cast<unsigned>(blocks), kTtThreads, smem, stream>>>(a, per, keys + 1);
  return cudaGetLastError();
}

}  // namespace fibattn
