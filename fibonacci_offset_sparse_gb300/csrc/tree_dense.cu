// Dense decode of a tree of drafted tokens over the paged cache (sm_103a): the dense control's
// form of tree.cu.  Node s of a sequence attends every cached row, its ancestors and itself:
// O_s = sum_j p_sj v_j, p = softmax(q'_s . k'_j / 8).
//
// What bounds it: every cached row is read once for all nodes and query heads of its key head, so up to some
// 64 rows of queries a key the read of the cache from HBM is the floor.  16 sequences of 4096, 8192 .. 65536 rows, 8 heads (1.14
// GB), one query: 175 us, 6.5 TB/s (96% of a measured copy).  float32, 8 sequences of 8192 .. 65536 rows (1.21 GB): 233 us, 5.2
// TB/s, what three blocks' rings hold in flight.  A call of one sequence is 9 us of launches, lengths, query, first copies and join.
//
// Work: a unit is kUnit consecutive cached rows of one task; a task is a (sequence, key head, block of
// ROWS query rows) and costs its units and kTaskCost more, what a block spends before and after
// its rows.  The costs of all tasks, in that order, are cut into one equal run a block (split of the
// long axis), whatever the lengths are: lengths live on the device, so every block computes the
// cut from them.  A block that holds a whole task writes its outputs; else it leaves a
// partial (max, sum, unnormalised O) in the workspace and join_kernel adds the partials of a
// task in a fixed order.
//
// Block: 4 warps that compute and one that feeds them.  The feeder copies K and V rows of a unit by
// TMA (128-byte swizzle) into a slot of a ring, a page at a time.  The computing warps are TILES row
// tiles (2 where float32 has more than 16 query rows) times 4 / TILES groups; the groups take the units in turn, and each warp keeps an online
// softmax (running maximum and sum, O in registers) over its units; the groups merge at the end of the run.
//   bf16: mma.sync m16n8k16 with the keys (then the dimensions of V) as the 16 rows of a tile and 8
//   query rows as its columns, so that a single query pays for 8 rows and not for 16.  K and V enter as
//   they are stored; the rotated query is split in three bf16 (24 bits of significand: lse is float32; with two, 16 bits,
//   lse was 1.3e-6 off where it is 1.6e-7) and the softmax weights in two (O is rounded to 8 bits).
//   float32: mma.sync m16n8k8 on tf32 with both operands split (hi, lo): hi*hi + hi*lo + lo*hi, 21 bits;
//   16 query rows a tile, whose weights are in place for the second product as the first leaves them.
// The tensor pipes round each sum toward zero (measured: 3.6e-8 of it a product in the mean, all to one side), so that a chain of
// products over a whole run would lose 1e-4 of O over 8 x 8 heads of 65536 rows.  Here each unit's products have a sum of their own, the
// smaller ones first, and O is added up from those in float32, rounded to nearest.  float32: the query and the weights are split to
// nearest and a score is two chains of four products, for the same reason: over 8191 rows O is 4.4e-7 off the 64-bit result (a
// float32 evaluation 2.3e-7), 9.9e-7 with all operands cut off and one chain, in 236 and 230 us for the 8 sequences above.  K and V
// are cut: to split them to nearest would leave 3.7e-7 and take, with 32 query rows, 389 us instead of 377.
// The drafted keys (at most 64, each seen by its own descendants only) are added by the block that holds a
// task's last unit, on CUDA cores in float32: a quad a query row, over the row's ancestors
// alone, so that another branch's values, NaN included, never meet a product.
#include <algorithm>

#include "tree_dense.cuh"

namespace fibattn {

namespace {

// bf16: up to so many query rows here, more in tree_dense_tc.cu.  8 rows over the 16 sequences above take 174 us here and
// 176 there, over 32 sequences of up to 1024 rows 17 and 23; one query over 4096 9.9 and 15.2; 16 rows over the 16 sequences took 283
// here (two tiles of 8) where they took 173 there.
constexpr int kMmaRows = 8;
constexpr int kSlotBytes = 8192;  // K and V of a unit
constexpr int kHalf = kSlotBytes / 2;
template <typename DT>
constexpr int kUnitRows = kHalf / (kD * static_cast<int>(sizeof(DT)));  // cached rows of a unit: 32 (bf16), 16 (float32)

// ------------------------------------------------------------------------------ products --
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ float lds_f32(uint32_t addr) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(x) : "r"(addr));
  return x;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x as tf32 hi (the upper 10 bits of the fraction) + the rest (exact in float32; the product takes
// its upper 10 bits).  An infinity or NaN stays in hi; its rest is NaN, as is the product's sum then.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}

// The same with the upper part rounded to nearest, so that the rest has either sign: products of two rests are left out, and
// would else all err to one side.  For |x| < 2^127 (an infinity or NaN stays as above).
__device__ __forceinline__ void split_tf32_near(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + (isfinite(x) ? 0x1000u : 0u)) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}

// What a computing warp holds and does, by type.  kRows: query rows of its tile.  load_query: a row of
// the query, rotated and times log2(e)/8, into the fragments of its tile in shared memory, where the groups'
// warps share them (registers are left for O and the scores).  unit: one unit's keys; rows of it from `valid` on
// were not filled for this sequence and count as absent, whatever lies there (`zero`: 128 bytes of 0,
// read in their place).  each(f): f(row, dim, pair of values) over O, dims d and d + step.
template <typename DT>
struct Core;

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}

// bf16, 8 query rows.  Lane (g, t): of the scores keys g and g + 8 of each 16, rows 2t and 2t + 1;
// of O dims g and g + 8 of each 16, the same rows.
template <>
struct Core<__nv_bfloat16> {
  static constexpr int kRows = 8, UNIT = kUnitRows<__nv_bfloat16>;
  static constexpr int kQueryBytes = 4 * 768;  // [k-step of 16 dims][lane]: hi, hi, mid, mid; then lo, lo
  float o[4][4];  // [16 dims][fragment]
  float m[2], l[2];

  // the row of the query that this lane loads
  static constexpr int kLoads = 1;
  __device__ __forceinline__ static int load_row(int) { return (threadIdx.x & 31) >> 2; }
  __device__ __forceinline__ static void load_query(const TreeArgs& a, uint4* qs, int, bool in, size_t row, int pos) {
    uint4* at = qs + (threadIdx.x & 31);
    uint2* low = reinterpret_cast<uint2*>(qs + 128) + (threadIdx.x & 31);
    if (!in) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        at[32 * s] = make_uint4(0, 0, 0, 0);
        low[32 * s] = make_uint2(0, 0);
      }
      return;
    }
    uint32_t qh[4][2], qm[4][2], ql[4][2];
    const int t = threadIdx.x & 3;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) + row * kD);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int d = 16 * s + 8 * f + 2 * t;
        const uint32_t x = __ldg(q + d / 2), y = __ldg(q + d / 2 + kFreq / 2);
        const float2 e0 = rope_factor(a.rope_lo, a.rope_hi, pos, d), e1 = rope_factor(a.rope_lo, a.rope_hi, pos, d + 1);
        const float sc = kLog2e / 8.0f;
        const float x0 = bf_lo(x) * sc, x1 = bf_hi(x) * sc, y0 = bf_lo(y) * sc, y1 = bf_hi(y) * sc;
        split_bf16(x0 * e0.x - y0 * e0.y, x1 * e1.x - y1 * e1.y, qh[s][f], qm[s][f], ql[s][f]);
        split_bf16(x0 * e0.y + y0 * e0.x, x1 * e1.y + y1 * e1.x, qh[s + 2][f], qm[s + 2][f], ql[s + 2][f]);
      }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      at[32 * s] = make_uint4(qh[s][0], qh[s][1], qm[s][0], qm[s][1]);
      low[32 * s] = make_uint2(ql[s][0], ql[s][1]);
    }
  }
  __device__ __forceinline__ void clear() {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
  }
  // Bits that are there only when every product with V is, and so every load of K and V by any lane.
  __device__ __forceinline__ uint32_t touched() const {
    return __float_as_uint(o[0][0]) | __float_as_uint(o[1][0]) | __float_as_uint(o[2][0]) | __float_as_uint(o[3][0]);
  }
  __device__ __forceinline__ static void scores(uint32_t kt, const uint4* qs, float (&s)[2][4]) {
    const int mi = (threadIdx.x & 31) >> 3, rl = threadIdx.x & 7;
    const uint32_t row = kt + ((mi & 1) * 8 + rl) * 128;
    const uint2* low = reinterpret_cast<const uint2*>(qs + 128);
    float c[2][4];  // the small products apart
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[x][e] = c[x][e] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t a[2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x) ldsm_x4(a[x], row + x * 2048 + (((2 * k + (mi >> 1)) ^ rl) << 4));
      const uint4 q = qs[k * 32 + (threadIdx.x & 31)];
      const uint2 l = low[k * 32 + (threadIdx.x & 31)];
#pragma unroll
      for (int x = 0; x < 2; ++x) mma_bf16(s[x], a[x], q.x, q.y);
#pragma unroll
      for (int x = 0; x < 2; ++x) mma_bf16(c[x], a[x], l.x, l.y);
#pragma unroll
      for (int x = 0; x < 2; ++x) mma_bf16(c[x], a[x], q.z, q.w);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[x][e] += c[x][e];
  }
  // Where a score came out NaN, the upper parts' product alone: an infinite key keeps its sign there, where
  // the parts' sum may add two infinities of opposite signs.
  __device__ __forceinline__ static void mend(uint32_t kt, const uint4* qs, float (&s)[2][4]) {
    const int mi = (threadIdx.x & 31) >> 3, rl = threadIdx.x & 7;
    const uint32_t row = kt + ((mi & 1) * 8 + rl) * 128;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        uint32_t a[4];
        ldsm_x4(a, row + x * 2048 + (((2 * k + (mi >> 1)) ^ rl) << 4));
        const uint4 q = qs[k * 32 + (threadIdx.x & 31)];
        mma_bf16(c, a, q.x, q.y);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (isnan(s[x][e])) s[x][e] = c[e];
    }
  }
  __device__ __forceinline__ void unit(uint32_t slot, const uint4* qs, uint32_t zero, int valid) {
    const int lane = threadIdx.x & 31, g = lane >> 2, mi = lane >> 3, rl = lane & 7;
    float s[2][4], sum[2];
    for (bool again = false;;) {  // a second time only where an infinite key made a NaN of the parts' sum
      scores(slot, qs, s);
      if (again) mend(slot, qs, s);
      if (valid < UNIT) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * x + g + 8 * (e >> 1) >= valid) s[x][e] = -INFINITY;
      }
      // the reference moves only when a score passes it by more than 8 (weights <= 256 until then), so
      // that the lanes of a row need not agree on a maximum for each unit
      float mx[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) mx[e] = fmaxf(fmaxf(s[0][e], s[0][2 + e]), fmaxf(s[1][e], s[1][2 + e]));
      if (__any_sync(0xffffffffu, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = mx[e];
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          x = fmaxf(x, m[e]);
          const float corr = m[e] == -INFINITY ? 1.f : ex2(m[e] - x);  // (nothing but zeros or a NaN yet)
          m[e] = x;
          l[e] *= corr;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            o[d][e] *= corr;
            o[d][2 + e] *= corr;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ref = m[e] == -INFINITY ? 0.f : m[e];  // no key yet: every weight is 0
        sum[e] = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            s[x][2 * h + e] = ex2(s[x][2 * h + e] - ref);
            sum[e] += s[x][2 * h + e];
          }
      }
      if (again || !__any_sync(0xffffffffu, isnan(sum[0]) || isnan(sum[1]))) break;
      again = true;
    }
    l[0] += sum[0];
    l[1] += sum[1];
    // O += V^T P: the weights turned from (key, row) to (row, key) 8 x 8 at a time
    const uint32_t vt = slot + kHalf;
    float c[4][4];  // the unit's own sum
#pragma unroll
    for (int d = 0; d < 4; ++d) c[d][0] = c[d][1] = c[d][2] = c[d][3] = 0.f;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t ph[2], pl[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t hi, lo;
        split_bf16(s[x][2 * h], s[x][2 * h + 1], hi, lo);
        ph[h] = transpose8x8(hi);
        pl[h] = transpose8x8(lo);
      }
      const int key = 16 * x + (mi >> 1) * 8 + rl;
      const uint32_t row = key < valid ? vt + key * 128 : zero;
      uint32_t a[4][4];
#pragma unroll
      for (int d = 0; d < 4; ++d) ldsm_x4_t(a[d], row + (((2 * d + (mi & 1)) ^ rl) << 4));
#pragma unroll
      for (int d = 0; d < 4; ++d) mma_bf16(c[d], a[d], pl[0], pl[1]);
#pragma unroll
      for (int d = 0; d < 4; ++d) mma_bf16(c[d], a[d], ph[0], ph[1]);
    }
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] += c[d][e];
  }
  // the rows' sums over the lanes
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
    }
  }
  __device__ __forceinline__ static bool leader() { return (threadIdx.x & 31) < 4; }
  __device__ __forceinline__ static int own_row(int i) { return 2 * (threadIdx.x & 3) + i; }  // the row of m[i], l[i]
  // O of own value i into row `acc`: f times O, and `old` times what is there where `keep`; the loads of a
  // row first, so that they do not wait for one another's stores
  __device__ __forceinline__ void add_to(int i, float* acc, float old, bool keep, float f) const {
    const int g = (threadIdx.x & 31) >> 2;
    float x[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) x[d] = keep ? acc[8 * d + g] : 0.f;
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      const float y = o[d >> 1][2 * (d & 1) + i] * f;
      acc[8 * d + g] = keep ? fmaf(x[d], old, y) : y;
    }
  }
};

// float32, 16 query rows.  Lane (g, t): rows g and g + 8; of the scores keys 2t and 2t + 1 of each 8, of
// O dims 2t and 2t + 1 of each 8.
template <>
struct Core<float> {
  static constexpr int kRows = 16, UNIT = kUnitRows<float>, NT = UNIT / 8;
  static constexpr int kQueryBytes = 8 * 2 * 512;  // [k-step of 8 dims][hi, lo][lane]
  float o[8][4], m[2], l[2];

  static constexpr int kLoads = 2;
  __device__ __forceinline__ static int load_row(int i) { return 8 * i + ((threadIdx.x & 31) >> 2); }
  __device__ __forceinline__ static void load_query(const TreeArgs& a, uint4* qs, int i, bool in, size_t row, int pos) {
    const int t = threadIdx.x & 3;
    uint32_t* at = reinterpret_cast<uint32_t*>(qs + (threadIdx.x & 31)) + i;  // fragment 2f + i of k-step s: 256 s + 2 f
    const float* q = static_cast<const float*>(a.q) + row * kD;
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int d = 8 * s + 4 * f + t;
        float x = 0.f, y = 0.f;
        float2 e = make_float2(1.f, 0.f);
        if (in) {
          e = rope_factor(a.rope_lo, a.rope_hi, pos, d);
          x = __ldg(q + d) * (kLog2e / 8.0f);
          y = __ldg(q + d + kFreq) * (kLog2e / 8.0f);
        }
        split_tf32_near(x * e.x - y * e.y, at[256 * s + 2 * f], at[256 * s + 128 + 2 * f]);
        split_tf32_near(x * e.y + y * e.x, at[256 * (s + 4) + 2 * f], at[256 * (s + 4) + 128 + 2 * f]);
      }
  }
  __device__ __forceinline__ void clear() {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int n = 0; n < 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  }
  __device__ __forceinline__ uint32_t touched() const {  // as above
    uint32_t x = 0;
#pragma unroll
    for (int n = 0; n < 8; ++n) x |= __float_as_uint(o[n][0]);
    return x;
  }
  __device__ __forceinline__ static void scores(uint32_t kt, const uint4* qs, float (&s)[NT][4]) {
    const int mi = (threadIdx.x & 31) >> 3, rl = threadIdx.x & 7;
    const uint32_t row = kt + rl * 128;  // dims 0..31, then 32..63 a half tile further
    float c[3][NT][4];                   // half of the large products and the small ones apart: four short chains a tile
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = c[0][n][e] = c[1][n][e] = c[2][n][e] = 0.f;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      uint32_t h[2][4], lo[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        *reinterpret_cast<uint4*>(h[k]) = qs[(2 * p + k) * 64 + (threadIdx.x & 31)];
        *reinterpret_cast<uint4*>(lo[k]) = qs[(2 * p + k) * 64 + 32 + (threadIdx.x & 31)];
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t b[4];
        ldsm_x4(b, row + n * 1024 + (p >> 1) * (kHalf / 2) + (((4 * (p & 1) + mi) ^ rl) << 4));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t h0, l0, h1, l1;
          split_tf32(__uint_as_float(b[2 * k]), h0, l0);
          split_tf32(__uint_as_float(b[2 * k + 1]), h1, l1);
          mma_tf32(p < 2 ? c[2][n] : s[n], h[k], h0, h1);
          mma_tf32(c[0][n], lo[k], h0, h1);
          mma_tf32(c[1][n], h[k], l0, l1);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = (s[n][e] + c[2][n][e]) + (c[0][n][e] + c[1][n][e]);
  }
  __device__ __forceinline__ static void mend(uint32_t kt, const uint4* qs, float (&s)[NT][4]) {  // as above
    const int mi = (threadIdx.x & 31) >> 3, rl = threadIdx.x & 7;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int p = 0; p < 4; ++p) {
        uint32_t b[4], h[4];
        ldsm_x4(b, kt + rl * 128 + n * 1024 + (p >> 1) * (kHalf / 2) + (((4 * (p & 1) + mi) ^ rl) << 4));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          *reinterpret_cast<uint4*>(h) = qs[(2 * p + k) * 64 + (threadIdx.x & 31)];
          mma_tf32(c, h, b[2 * k], b[2 * k + 1]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (isnan(s[n][e])) s[n][e] = c[e];
    }
  }
  __device__ __forceinline__ void unit(uint32_t slot, const uint4* qs, uint32_t zero, int valid) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float s[NT][4], sum[2];
    for (bool again = false;;) {  // a second time only where an infinite key made a NaN of the parts
      scores(slot, qs, s);
      if (again) mend(slot, qs, s);
      if (valid < UNIT) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (8 * n + 2 * t + (e & 1) >= valid) s[n][e] = -INFINITY;
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
      if (__any_sync(0xffffffffu, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {  // as above
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x = mx[h];
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          x = fmaxf(x, m[h]);
          const float corr = m[h] == -INFINITY ? 1.f : ex2(m[h] - x);
          m[h] = x;
          l[h] *= corr;
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            o[n][2 * h] *= corr;
            o[n][2 * h + 1] *= corr;
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float ref = m[h] == -INFINITY ? 0.f : m[h];
        sum[h] = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[n][2 * h + e] = ex2(s[n][2 * h + e] - ref);
            sum[h] += s[n][2 * h + e];
          }
      }
      if (again || !__any_sync(0xffffffffu, isnan(sum[0]) || isnan(sum[1]))) break;
      again = true;
    }
    l[0] += sum[0];
    l[1] += sum[1];
    // k index t of the product is key 2t, t + 4 is key 2t + 1: what a lane holds of the scores
    const uint32_t vt = slot + kHalf;
    uint32_t hi[NT][4], lo[NT][4], row[NT][2], half[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      split_tf32_near(s[n][0], hi[n][0], lo[n][0]);
      split_tf32_near(s[n][2], hi[n][1], lo[n][1]);
      split_tf32_near(s[n][1], hi[n][2], lo[n][2]);
      split_tf32_near(s[n][3], hi[n][3], lo[n][3]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int k = 8 * n + 2 * t + x;
        row[n][x] = k < valid ? vt + k * 128 : zero;
        half[n][x] = k < valid ? kHalf / 2 : 0;
      }
    }
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      const int ch = 2 * (d & 3) + (g >> 2);
      uint32_t h[NT][2], l0[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          split_tf32(lds_f32(row[n][x] + (d >> 2) * half[n][x] + ((ch ^ ((2 * t + x) & 7)) << 4) + (g & 3) * 4), h[n][x], l0[n][x]);
      float c[4] = {0.f, 0.f, 0.f, 0.f};  // the unit's own sum, the small products first
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_tf32(c, lo[n], h[n][0], h[n][1]);
        mma_tf32(c, hi[n], l0[n][0], l0[n][1]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_tf32(c, hi[n], h[n][0], h[n][1]);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] += c[e];
    }
  }
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
  }
  __device__ __forceinline__ static bool leader() { return (threadIdx.x & 3) == 0; }
  __device__ __forceinline__ static int own_row(int i) { return 8 * i + ((threadIdx.x & 31) >> 2); }
  __device__ __forceinline__ void add_to(int i, float* acc, float old, bool keep, float f) const {
    const int t = threadIdx.x & 3;
    float2 x[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) x[n] = keep ? *reinterpret_cast<const float2*>(acc + 8 * n + 2 * t) : make_float2(0.f, 0.f);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      float2 y = make_float2(o[n][2 * i] * f, o[n][2 * i + 1] * f);
      if (keep) y = make_float2(fmaf(x[n].x, old, y.x), fmaf(x[n].y, old, y.y));
      *reinterpret_cast<float2*>(acc + 8 * n + 2 * t) = y;
    }
  }
};

// ------------------------------------------------------------------------------ the kernel --
// Blocks an SM holds, by registers (an SM's four parts hold 512 a lane each: four warps of 128, three of 168) and shared
// memory.  float32, when the 8 sequences above took 205 us: three blocks of 4 groups and 4 slots 205 us, two of 4 groups and 8
// slots 286, two of 7 groups and 7 slots 254 (a unit's feeding takes a feeder longer than its computing takes the groups).  With 32
// query rows two blocks took 333 us and three 317, but 64 rows, whose drafts leave room for two, 671 and 786; one task of 64 rows
// on four tiles instead of two tasks 923.  As it is: 233 us, 376 with 32 rows, 735 with 64.
template <typename DT, int TILES>
struct DtSmem {
  using C = Core<DT>;
  static constexpr bool kHalves = sizeof(DT) == 2, kPacked = false;
  static constexpr int kUnit = C::UNIT, kTaskCost = 12, kLeast = 4;
  static constexpr int kGroups = TILES == 1 ? 4 : 2, kCons = 32 * TILES * kGroups, kThreads = kCons + 32;
  static constexpr int kRows = C::kRows * TILES;
  static constexpr int kResident = TILES == 1 ? 3 : 2;
  // of the ring; a multiple of the groups, so that a slot is always the same group's
  static constexpr int kSlots = kHalves ? 8 : 4;
  // byte offsets in dynamic shared memory (its base is 1024-byte aligned)
  static constexpr int kAcc = kSlots * kSlotBytes;
  static constexpr int kMax = kAcc + kRows * kAccStride * 4;
  static constexpr int kSum = kMax + (kGroups + 1) * kRows * 4;
  static constexpr int kZero = (kSum + (kGroups + 1) * kRows * 4 + 127) / 128 * 128;
  static constexpr int kFixed = kZero + 128;  // barriers, flag, positions: statically they are padded to the base's 1024 bytes
  static constexpr int kQuery = kFixed + (2 * 8 * kSlots + 16 + 4 * kRows + 127) / 128 * 128;
  static constexpr int kDraft = kQuery + TILES * C::kQueryBytes;
  static size_t bytes(int B, int T) { return kDraft + static_cast<size_t>(T) * kD * 8 + Schedule<kPacked>::bytes(B); }
  static size_t most_bytes() { return bytes(kMaxSeqs, TILES == 1 ? kRows : kMaxDrafts); }
};

template <typename DT, int TILES>
__global__ void __launch_bounds__(DtSmem<DT, TILES>::kThreads, DtSmem<DT, TILES>::kResident)
    dense_tree_kernel(const __grid_constant__ DenseTreeArgs da, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v) {
  using S = DtSmem<DT, TILES>;
  using C = Core<DT>;
  constexpr int UNIT = S::kUnit, ROWS = S::kRows, GROUPS = S::kGroups, CONS = S::kCons;
  constexpr int kSlots = S::kSlots;
  static_assert(kSlots % GROUPS == 0, "a slot belongs to one group");
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + S::kFixed);
  uint64_t* empty_bar = full_bar + kSlots;
  volatile int& s_err = *reinterpret_cast<volatile int*>(empty_bar + kSlots);
  int* s_pos = reinterpret_cast<int*>(smem + S::kFixed + 16 * kSlots + 16);  // positions of a piece's rows
  const TreeArgs& a = da.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (tid == 0) {
    s_err = 0;
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], TILES);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (tid < 32) reinterpret_cast<float*>(smem + S::kZero)[tid] = 0.f;
  const Schedule<S::kPacked> sch(smem + S::kDraft + a.T * kD * 8, a.B);
  build_schedule<S>(a, sch);
  if (tid == 0) clear_splits(da);
  const long long cost = sch.end(a.B);
  const int sharing = sharing_blocks(cost, da.blocks, S::kLeast);
  if (static_cast<int>(blockIdx.x) >= sharing) return;
  const long long u0 = cut(cost, sharing, blockIdx.x), u1 = cut(cost, sharing, blockIdx.x + 1);

  if (warp == CONS / 32) {
    feed<DT, S>(da, sch, u0, u1, &map_k, &map_v, smem, full_bar, empty_bar, &s_err);
    return;
  }

  // ===================================================================== computing warps
  const int tile = warp % TILES, grp = warp / TILES;
  float* s_acc = reinterpret_cast<float*>(smem + S::kAcc);
  float* s_max = reinterpret_cast<float*>(smem + S::kMax);
  float* s_sum = reinterpret_cast<float*>(smem + S::kSum);
  float* s_draft = reinterpret_cast<float*>(smem + S::kDraft);
  const uint32_t ring = smem_addr(smem), zero = smem_addr(smem + S::kZero);
  int count = 0;
  for (long long u = u0; u < u1;) {
    const Task k = task_of<S>(a, sch, u, u1);
    u = k.start + k.units + S::kTaskCost;
    if (k.first == k.last) continue;
    if (tid == 0) note_split<S>(da, k, cost, sharing);
    const bool tail = k.last == k.units, whole = tail && k.first == 0;
    const int r0 = k.rb * ROWS, rows = min(ROWS, a.G * k.n - r0);  // row r0 + i is (query head, node)
    bool ok = true;
    const WarpTree tree = warp_tree(a, k.b, k.n, &ok);
    uint4* qs = reinterpret_cast<uint4*>(smem + S::kQuery + tile * C::kQueryBytes);
    for (int i = grp; i < C::kLoads; i += GROUPS) {
      const int r = C::kRows * tile + C::load_row(i);
      int s = 0;
      const size_t row = r < rows ? row_of(a, k, r0 + r, &s) : 0;
      const int depth = pick32(tree.depth, s);
      const int pos = r < rows ? position_of(a, k, depth, &ok) : 0;
      s_pos[r] = pos;
      C::load_query(a, qs, i, r < rows, row, pos);
    }
    if (tail) stage_drafts<DT, CONS>(a, k, tree, s_draft, &ok);
    cons_sync<CONS>();
    if (tail)
      attend_drafts<CONS>(a, k, tree, s_draft, r0, rows, s_acc, s_max + GROUPS * ROWS, s_sum + GROUPS * ROWS,
                                 [&](int r, int lane4, float(&y)[16]) {
                                   int s;
                                   const size_t row = row_of(a, k, r0 + r, &s);
                                   float2 e[8];
                                   load_part(static_cast<const DT*>(a.q) + row * kD, lane4, y);
                                   rope_row(a.rope_lo, a.rope_hi, s_pos[r], lane4, e);
                                   rotate_part(y, e, false);
#pragma unroll
                                   for (int w = 0; w < 16; ++w) y[w] *= kLog2e / 8.0f;
                                 });
    // ---- the cached rows: a unit in turn for each group
    C core;
    core.clear();
    for (int i = k.first; i < k.last; ++i, ++count) {
      if (count % GROUPS != grp) continue;
      const int slot = count % kSlots;
      if (!warp_wait(&full_bar[slot], (count / kSlots) & 1, da.wait_ns, &s_err)) {
        s_err = 1;
        if (lane == 0) atomicExch(a.status, kStatusTimeout);
        continue;  // (the slot is not released: its rows may still be on their way)
      }
      core.unit(ring + slot * kSlotBytes, qs, zero, k.len - i * UNIT);
      __syncwarp();
      // The slot is released when its values have come, not when their loads were sent: the address waits for the products.  Loads
      // that other blocks' traffic held up in the SM would else be overtaken by the release, and the next copy by them.
      if (lane == 0) mbar_arrive_at(smem_addr(&empty_bar[slot]) + (core.touched() & da.zero));
    }
    // ---- merge the groups (and the drafted keys' part) in a fixed order
    core.finish();
    if (C::leader()) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s_max[grp * ROWS + C::kRows * tile + C::own_row(i)] = core.m[i];
        s_sum[grp * ROWS + C::kRows * tile + C::own_row(i)] = core.l[i];
      }
    }
    cons_sync<CONS>();
    const int parts = GROUPS + (tail ? 1 : 0);
    float f[2], old[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = C::kRows * tile + C::own_row(i);
      float all = -INFINITY;
#pragma unroll
      for (int x = 0; x < GROUPS; ++x) all = fmaxf(all, s_max[x * ROWS + r]);
      const bool drafts = tail && r < rows;
      const float md = drafts ? s_max[GROUPS * ROWS + r] : -INFINITY;
      all = fmaxf(all, md);
      f[i] = weight_of(core.m[i], core.l[i], all);
      old[i] = grp > 0 ? 1.f : drafts ? weight_of(md, s_sum[GROUPS * ROWS + r], all) : 0.f;
    }
    // even groups into one sum, odd ones into another, which takes the query's room (and the drafts'): two turns of four groups
    float* s_odd = reinterpret_cast<float*>(smem + S::kQuery);
    static_assert(TILES * C::kQueryBytes + kD * 8 >= ROWS * kAccStride * 4, "room for the odd groups' sum");
    for (int turn = 0; turn < GROUPS / 2; ++turn) {
      if (grp / 2 == turn) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = C::kRows * tile + C::own_row(i);
          if (r < rows) core.add_to(i, (grp & 1 ? s_odd : s_acc) + r * kAccStride, old[i], turn > 0 || (grp == 0 && tail), f[i]);
        }
      }
      cons_sync<CONS>();
    }
    if (!ok) atomicExch(a.status, kStatusDeviceAssert);
    if (!s_err) write_rows<DT, ROWS, CONS>(da, k, whole, k.start >= u0 ? 1 : 0, r0, rows, s_acc, s_odd, s_max, s_sum, parts);
    cons_sync<CONS>();  // all of it is free again
  }
}

template <typename DT, int TILES>
constexpr int kGrid = 152 * DtSmem<DT, TILES>::kResident;  // 152 SMs

template <typename DT, int TILES>
cudaError_t launch(const DenseTreeArgs& args, cudaStream_t stream) {
  using S = DtSmem<DT, TILES>;
  DenseTreeArgs da = args;
  da.blocks = kGrid<DT, TILES>;
  da.split = reinterpret_cast<Split*>(da.part + static_cast<size_t>(da.blocks) * 2 * S::kRows * kDtPart);
  const TreeArgs& a = da.a;
  const size_t smem = S::bytes(a.B, a.T);
  cudaError_t e = allow_shared(dense_tree_kernel<DT, TILES>, S::most_bytes());
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  e = maps_of(a, static_cast<int>(sizeof(DT)), S::kUnit, &mk, &mv);
  if (e != cudaSuccess) return e;
  dense_tree_kernel<DT, TILES><<<da.blocks, S::kThreads, smem, stream>>>(da, mk, mv);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_join<DT, S>(da, stream);
}

template <typename DT, int TILES>
size_t part_bytes() {
  return static_cast<size_t>(kGrid<DT, TILES>) * (2 * DtSmem<DT, TILES>::kRows * kDtPart * sizeof(float) + 2 * sizeof(Split));
}

}  // namespace

// The most that the kernels of so many query rows or fewer need, so that what serves a call serves every smaller one: a kernel for more
// rows may have half the blocks.
size_t dense_tree_workspace_bytes(int Hq, int H, int T, int dtype) {
  const int rows = Hq / H * T;
  if (dtype == FIB_DTYPE_F32) return rows <= 16 ? part_bytes<float, 1>() : std::max(part_bytes<float, 1>(), part_bytes<float, 2>());
  const size_t few = part_bytes<__nv_bfloat16, 1>();
  return rows <= kMmaRows ? few : std::max(few, dense_tree_tc_bytes(rows));
}

cudaError_t launch_dense_tree(const TreeArgs& a, int dtype, unsigned long long wait_ns, int skip_copy, void* ws, cudaStream_t stream) {
  DenseTreeArgs da;
  da.skip_copy = skip_copy;
  da.a = a;
  da.part = static_cast<float*>(ws);
  da.wait_ns = wait_ns;
  da.split = nullptr;
  da.zero = 0;
  da.blocks = 0;
  const int rows = a.G * a.T;
  if (dtype == FIB_DTYPE_F32) return rows <= 16 ? launch<float, 1>(da, stream) : launch<float, 2>(da, stream);
  return rows <= kMmaRows ? launch<__nv_bfloat16, 1>(da, stream) : launch_dense_tree_tc(da, stream);
}

}  // namespace fibattn
