// Dense decode of a tree of drafted tokens over the paged cache (sm_103a): the dense control's
// form of tree.cu.  Node s of a sequence attends every cached row, its ancestors and itself:
// O_s = sum_j p_sj v_j, p = softmax(q'_s . k'_j / 8).
//
// What bounds it: every cached row is read once for all nodes and query heads of its key head, so up to some
// 64 rows of queries a key the read of the cache from HBM is the floor.
//
// Work: a unit is kUnit consecutive cached rows of one task; a task is a (sequence, key head, block of
// ROWS query rows) and costs its units and kTaskCost more, what a block spends before and after
// its rows.  The costs of all tasks, in that order, are cut into one equal run a block (split of the
// long axis), whatever the lengths are: lengths live on the device, so every block computes the
// cut from them.  A block that holds a whole task writes its outputs; else it leaves a
// partial (max, sum, unnormalised O) in the workspace and join_kernel adds the partials of a
// task in the order of the blocks.
//
// Block: 4 warps that compute and one that feeds them.  The feeder copies K and V rows of a unit by
// TMA (128-byte swizzle) into a slot of a ring, a page at a time.  The computing warps are TILES row
// tiles times 4 / TILES groups; the groups take the units in turn, and each warp keeps an online
// softmax (running maximum and sum, O in registers) over its units; the groups merge at the end of the run.
//   bf16: mma.sync m16n8k16 with the keys (then the dimensions of V) as the 16 rows of a tile and 8
//   query rows as its columns, so that a single query pays for 8 rows and not for 16, and a warp that
//   holds 32 reads each K and V row once for all of them.  K and V enter as they are stored; the rotated
//   query and the softmax weights are split in two bf16 (x = hi + lo, 16 bits of significand), each
//   product twice, so that neither is rounded to 8 bits.
//   float32: mma.sync m16n8k8 on tf32 with both operands split (hi, lo): hi*hi + hi*lo + lo*hi, 21 bits;
//   16 query rows a tile, whose weights are in place for the second product as the first leaves them.
// The drafted keys (at most 64, each seen by its own descendants only) are added by the block that holds a
// task's last unit, on CUDA cores in float32: a quad a query row, over the row's ancestors
// alone, so that another branch's values, NaN included, never meet a product.
#include <cuda.h>

#include "tree.cuh"

namespace fibattn {

namespace {

constexpr int kDtWarps = 4;
constexpr int kDtCons = 32 * kDtWarps;
constexpr int kDtThreads = kDtCons + 32;
constexpr int kSlotBytes = 8192;  // K and V of a unit
constexpr int kHalf = kSlotBytes / 2;
constexpr int kTaskCost = 12;     // a task's own cost in units
constexpr int kAccStride = 68;   // floats of a row of O in shared memory
constexpr int kDtPart = kD + 2;  // floats of a partial's row: O, max, sum

struct DenseTreeArgs {
  TreeArgs a;
  float* part;  // [blocks][2][ROWS][kDtPart]
  unsigned long long wait_ns;
  int blocks;   // blocks of the grid
};

// ------------------------------------------------------------------------------ schedule --
// In shared memory: the cost before each sequence, and the sequences' rows and nodes.
struct Schedule {
  long long* start;  // [B + 1]
  int* len;          // [B]
  int* n;            // [B]; 0 where the sequence has nothing to do
};

__device__ __forceinline__ Schedule schedule_at(unsigned char* smem, int B) {
  Schedule s;
  s.start = reinterpret_cast<long long*>(smem);
  s.len = reinterpret_cast<int*>(s.start + B + 1);
  s.n = s.len + B;
  return s;
}
inline size_t schedule_bytes(int B) { return (sizeof(long long) * (B + 1) + 2 * sizeof(int) * B + 127) / 128 * 128; }

template <typename DT>
constexpr int kUnit = kHalf / (kD * static_cast<int>(sizeof(DT)));  // cached rows of a unit: 32 (bf16), 16 (float32)

template <int UNIT>
__device__ __forceinline__ int units_of(int len) {
  return len <= UNIT ? 1 : (len + UNIT - 1) / UNIT;
}

// Every thread of the block; ends synchronised.
template <int UNIT, int ROWS>
__device__ __forceinline__ void build_schedule(const TreeArgs& a, const Schedule& s) {
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    int n, len;
    if (!sequence_of(a, b, &n, &len)) {
      atomicExch(a.status, kStatusDeviceAssert);
      n = len = 0;
    }
    s.len[b] = len;
    s.n[b] = n;
    s.start[b + 1] = n == 0 ? 0 : static_cast<long long>(units_of<UNIT>(len) + kTaskCost) * a.H * ((a.G * n + ROWS - 1) / ROWS);
  }
  if (threadIdx.x == 0) s.start[0] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    long long base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + static_cast<int>(threadIdx.x);
      long long x = b < a.B ? s.start[b + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (static_cast<int>(threadIdx.x) >= d) x += y;
      }
      if (b < a.B) s.start[b + 1] = base + x;
      base += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
}

// How many of the grid's blocks share the `cost`: fewer where a block would get less than a unit a warp.
__device__ __forceinline__ int sharing_blocks(long long cost, int blocks) {
  const long long want = (cost + kDtWarps - 1) / kDtWarps;
  return want < blocks ? static_cast<int>(want) : blocks;
}
// Block c's run begins at cut(c); block_at(x) is the block whose run holds place x.
__device__ __forceinline__ long long cut(long long cost, int sharing, int c) { return cost * c / sharing; }
__device__ __forceinline__ int block_at(long long cost, int sharing, long long x) {
  return static_cast<int>(((x + 1) * sharing - 1) / cost);  // the largest c with cost * c < (x + 1) * sharing
}

// The task at place u of the cost, and the units of it that lie in [u, end).
struct Task {
  int b, h, rb;
  int len, n;
  int units;         // of the whole task
  long long start;   // its place in the cost
  int first, last;   // units [first, last); none where only a part of the task's own cost is in the run
};
template <int UNIT, int ROWS>
__device__ __forceinline__ Task task_of(const TreeArgs& a, const Schedule& s, long long u, long long end) {
  int lo = 0, hi = a.B;  // start[lo] <= u < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.start[mid] <= u)
      lo = mid;
    else
      hi = mid;
  }
  Task t;
  t.b = lo;
  t.len = s.len[lo];
  t.n = s.n[lo];
  t.units = units_of<UNIT>(t.len);
  const int rbs = (a.G * t.n + ROWS - 1) / ROWS, each = t.units + kTaskCost;
  const long long off = u - s.start[lo];
  const int task = static_cast<int>(off / each);
  t.start = s.start[lo] + static_cast<long long>(task) * each;
  t.h = task / rbs;
  t.rb = task - t.h * rbs;
  const long long last = min(end - t.start, static_cast<long long>(each)) - kTaskCost;
  t.first = max(0, static_cast<int>(u - t.start) - kTaskCost);
  t.last = max(0, static_cast<int>(last));
  return t;
}

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
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// x0, x1 as bf16 pairs hi + lo
__device__ __forceinline__ void split_bf16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf2_rn(x0, x1);
  lo = pack_bf2_rn(x0 - bf_lo(hi), x1 - bf_hi(hi));
}
// x as tf32 hi (the upper 10 bits of the fraction) + the rest (exact in float32; the product takes
// its upper 10 bits).  An infinity or NaN stays in hi; its rest is NaN, as is the product's sum then.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}

// What a partial of maximum m and sum l counts where the common maximum is `all`.  One without a finite
// score counts nothing, unless a NaN is in it, which goes on.
__device__ __forceinline__ float weight_of(float m, float l, float all) {
  return m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : ex2(m - all);
}

__device__ __forceinline__ void cons_sync() { asm volatile("bar.sync 1, %0;\n" ::"n"(kDtCons) : "memory"); }

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

// The 16 dims D_t of a row (common.cuh) as they are stored.
__device__ __forceinline__ void load_raw(const __nv_bfloat16* row, int t, uint4 (&x)[2]) {
  x[0] = __ldg(reinterpret_cast<const uint4*>(row + 8 * t));
  x[1] = __ldg(reinterpret_cast<const uint4*>(row + kFreq + 8 * t));
}
__device__ __forceinline__ void load_raw(const float* row, int t, uint4 (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __ldg(reinterpret_cast<const uint4*>(row + (i >> 1) * kFreq + 8 * t) + (i & 1));
}
__device__ __forceinline__ void raw_to_float(const uint4 (&x)[2], float (&v)[16], const __nv_bfloat16*) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] = bf_lo(w[j]);
      v[8 * i + 2 * j + 1] = bf_hi(w[j]);
    }
  }
}
__device__ __forceinline__ void raw_to_float(const uint4 (&x)[4], float (&v)[16], const float*) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[4 * i] = __uint_as_float(x[i].x);
    v[4 * i + 1] = __uint_as_float(x[i].y);
    v[4 * i + 2] = __uint_as_float(x[i].z);
    v[4 * i + 3] = __uint_as_float(x[i].w);
  }
}

// What a computing warp holds and does, by type.  kRows: query rows of its tile.  load_query: a row of
// the query, rotated and times log2(e)/8, into the fragments of its tile in shared memory, where the groups'
// warps share them (registers are left for O and the scores).  unit: one unit's keys; rows of it from `valid` on
// were not filled for this sequence and count as absent, whatever lies there (`zero`: 128 bytes of 0,
// read in their place).  each(f): f(row, dim, pair of values) over O, dims d and d + step.
template <typename DT, int NR>
struct Core;

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}

// bf16, 8 NR query rows.  Lane (g, t): of the scores keys g and g + 8 of each 16, rows 8n + 2t and + 1;
// of O dims g and g + 8 of each 16, the same rows.
template <int NR>
struct Core<__nv_bfloat16, NR> {
  static constexpr int kRows = 8 * NR, kOwn = 2 * NR, UNIT = kUnit<__nv_bfloat16>;
  static constexpr int kQueryBytes = NR * 4 * 512;  // [8 rows][k-step of 16 dims][lane]: hi, hi, lo, lo
  float o[NR][4][4];                                // [8 rows][16 dims][fragment]
  float m[NR][2], l[NR][2];

  // rows of the query that this lane loads: row 8n + g
  static constexpr int kLoads = NR;
  __device__ __forceinline__ static int load_row(int i) { return 8 * i + ((threadIdx.x & 31) >> 2); }
  __device__ __forceinline__ static void load_query(const TreeArgs& a, uint4* qs, int i, bool in, size_t row, int pos) {
    uint4* at = qs + i * 128 + (threadIdx.x & 31);
    if (!in) {
#pragma unroll
      for (int s = 0; s < 4; ++s) at[32 * s] = make_uint4(0, 0, 0, 0);
      return;
    }
    uint32_t qh[4][2], ql[4][2];
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
        split_bf16(x0 * e0.x - y0 * e0.y, x1 * e1.x - y1 * e1.y, qh[s][f], ql[s][f]);
        split_bf16(x0 * e0.y + y0 * e0.x, x1 * e1.y + y1 * e1.x, qh[s + 2][f], ql[s + 2][f]);
      }
#pragma unroll
    for (int s = 0; s < 4; ++s) at[32 * s] = make_uint4(qh[s][0], qh[s][1], ql[s][0], ql[s][1]);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) o[n][x][0] = o[n][x][1] = o[n][x][2] = o[n][x][3] = 0.f;
    }
  }
  __device__ __forceinline__ static void scores(uint32_t kt, const uint4* qs, float (&s)[2][NR][4]) {
    const int mi = (threadIdx.x & 31) >> 3, rl = threadIdx.x & 7;
    const uint32_t row = kt + ((mi & 1) * 8 + rl) * 128;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int n = 0; n < NR; ++n) s[x][n][0] = s[x][n][1] = s[x][n][2] = s[x][n][3] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t a[2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x) ldsm_x4(a[x], row + x * 2048 + (((2 * k + (mi >> 1)) ^ rl) << 4));
      uint4 q[NR];
#pragma unroll
      for (int n = 0; n < NR; ++n) q[n] = qs[n * 128 + k * 32 + (threadIdx.x & 31)];
      // all upper parts, then all lower ones: two products on one sum stay 2 NR apart
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) mma_bf16(s[x][n], a[x], q[n].x, q[n].y);
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) mma_bf16(s[x][n], a[x], q[n].z, q[n].w);
    }
  }
  // Where a score came out NaN, the upper parts' product alone: an infinite key keeps its sign there, where
  // hi + lo may add two infinities of opposite signs.
  __device__ __forceinline__ static void mend(uint32_t kt, const uint4* qs, float (&s)[2][NR][4]) {
    const int mi = (threadIdx.x & 31) >> 3, rl = threadIdx.x & 7;
    const uint32_t row = kt + ((mi & 1) * 8 + rl) * 128;
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          uint32_t a[4];
          ldsm_x4(a, row + x * 2048 + (((2 * k + (mi >> 1)) ^ rl) << 4));
          const uint4 q = qs[n * 128 + k * 32 + (threadIdx.x & 31)];
          mma_bf16(c, a, q.x, q.y);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (isnan(s[x][n][e])) s[x][n][e] = c[e];
      }
  }
  __device__ __forceinline__ void unit(uint32_t slot, const uint4* qs, uint32_t zero, int valid) {
    const int lane = threadIdx.x & 31, g = lane >> 2, mi = lane >> 3, rl = lane & 7;
    float s[2][NR][4], sum[NR][2];
    for (bool again = false;;) {  // a second time only where an infinite key made a NaN of hi + lo
      scores(slot, qs, s);
      if (again) mend(slot, qs, s);
      if (valid < UNIT) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (16 * x + g + 8 * (e >> 1) >= valid) s[x][n][e] = -INFINITY;
      }
      // the reference moves only when a score passes it by more than 8 (weights <= 256 until then), so
      // that the lanes of a row need not agree on a maximum for each unit
      bool past = false;
      float mx[NR][2];
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[n][e] = fmaxf(fmaxf(s[0][n][e], s[0][n][2 + e]), fmaxf(s[1][n][e], s[1][n][2 + e]));
          past |= mx[n][e] > m[n][e] + 8.f;
        }
      if (__any_sync(0xffffffffu, past)) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = mx[n][e];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            x = fmaxf(x, m[n][e]);
            const float corr = m[n][e] == -INFINITY ? 1.f : ex2(m[n][e] - x);  // (nothing but zeros or a NaN yet)
            m[n][e] = x;
            l[n][e] *= corr;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              o[n][d][e] *= corr;
              o[n][d][2 + e] *= corr;
            }
          }
      }
      bool bad = false;
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float ref = m[n][e] == -INFINITY ? 0.f : m[n][e];  // no key yet: every weight is 0
          sum[n][e] = 0.f;
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              s[x][n][2 * h + e] = ex2(s[x][n][2 * h + e] - ref);
              sum[n][e] += s[x][n][2 * h + e];
            }
          bad |= isnan(sum[n][e]);
        }
      if (again || !__any_sync(0xffffffffu, bad)) break;
      again = true;
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      l[n][0] += sum[n][0];
      l[n][1] += sum[n][1];
    }
    // O += V^T P: the weights turned from (key, row) to (row, key) 8 x 8 at a time
    const uint32_t vt = slot + kHalf;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t ph[NR][2], pl[NR][2];
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t hi, lo;
          split_bf16(s[x][n][2 * h], s[x][n][2 * h + 1], hi, lo);
          ph[n][h] = transpose8x8(hi);
          pl[n][h] = transpose8x8(lo);
        }
      const int key = 16 * x + (mi >> 1) * 8 + rl;
      const uint32_t row = key < valid ? vt + key * 128 : zero;
      uint32_t a[4][4];
#pragma unroll
      for (int d = 0; d < 4; ++d) ldsm_x4_t(a[d], row + (((2 * d + (mi & 1)) ^ rl) << 4));
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int n = 0; n < NR; ++n) mma_bf16(o[n][d], a[d], ph[n][0], ph[n][1]);
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int n = 0; n < NR; ++n) mma_bf16(o[n][d], a[d], pl[n][0], pl[n][1]);
    }
  }
  // the rows' sums over the lanes; the rows of own value i
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
      }
  }
  __device__ __forceinline__ static bool leader() { return (threadIdx.x & 31) < 4; }
  __device__ __forceinline__ static int own_row(int i) { return 8 * (i >> 1) + 2 * (threadIdx.x & 3) + (i & 1); }
  __device__ __forceinline__ float own_max(int i) const { return m[i >> 1][i & 1]; }
  __device__ __forceinline__ float own_sum(int i) const { return l[i >> 1][i & 1]; }
  // O of own value i into row `acc`: f times O, and `old` times what is there where `keep`; the loads of a
  // row first, so that they do not wait for one another's stores
  __device__ __forceinline__ void add_to(int i, float* acc, float old, bool keep, float f) const {
    const int g = (threadIdx.x & 31) >> 2;
    float x[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) x[d] = keep ? acc[8 * d + g] : 0.f;
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      const float y = o[i >> 1][d >> 1][2 * (d & 1) + (i & 1)] * f;
      acc[8 * d + g] = keep ? fmaf(x[d], old, y) : y;
    }
  }
};

// float32, 16 query rows.  Lane (g, t): rows g and g + 8; of the scores keys 2t and 2t + 1 of each 8, of
// O dims 2t and 2t + 1 of each 8.
template <int NR>
struct Core<float, NR> {
  static constexpr int kRows = 16, kOwn = 2, UNIT = kUnit<float>, NT = UNIT / 8;
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
        split_tf32(x * e.x - y * e.y, at[256 * s + 2 * f], at[256 * s + 128 + 2 * f]);
        split_tf32(x * e.y + y * e.x, at[256 * (s + 4) + 2 * f], at[256 * (s + 4) + 128 + 2 * f]);
      }
  }
  __device__ __forceinline__ void clear() {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int n = 0; n < 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  }
  __device__ __forceinline__ static void scores(uint32_t kt, const uint4* qs, float (&s)[NT][4]) {
    const int mi = (threadIdx.x & 31) >> 3, rl = threadIdx.x & 7;
    const uint32_t row = kt + rl * 128;  // dims 0..31, then 32..63 a half tile further
    float c[2][NT][4];                   // the small products apart: three chains a tile instead of one
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = c[0][n][e] = c[1][n][e] = 0.f;
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
          mma_tf32(s[n], h[k], h0, h1);
          mma_tf32(c[0][n], lo[k], h0, h1);
          mma_tf32(c[1][n], h[k], l0, l1);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] += c[0][n][e] + c[1][n][e];
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
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t hi[4], lo[4];
      split_tf32(s[n][0], hi[0], lo[0]);
      split_tf32(s[n][2], hi[1], lo[1]);
      split_tf32(s[n][1], hi[2], lo[2]);
      split_tf32(s[n][3], hi[3], lo[3]);
      const int k0 = 8 * n + 2 * t, k1 = k0 + 1;
      const uint32_t r0 = k0 < valid ? vt + k0 * 128 : zero, r1 = k1 < valid ? vt + k1 * 128 : zero;
      const uint32_t s0 = k0 < valid ? kHalf / 2 : 0, s1 = k1 < valid ? kHalf / 2 : 0;
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        const int ch = 2 * (d & 3) + (g >> 2);
        uint32_t h0, l0, h1, l1;
        split_tf32(lds_f32(r0 + (d >> 2) * s0 + ((ch ^ (k0 & 7)) << 4) + (g & 3) * 4), h0, l0);
        split_tf32(lds_f32(r1 + (d >> 2) * s1 + ((ch ^ (k1 & 7)) << 4) + (g & 3) * 4), h1, l1);
        mma_tf32(o[d], hi, h0, h1);
        mma_tf32(o[d], lo, h0, h1);
        mma_tf32(o[d], hi, l0, l1);
      }
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
  __device__ __forceinline__ float own_max(int i) const { return m[i]; }
  __device__ __forceinline__ float own_sum(int i) const { return l[i]; }
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
template <typename DT, int NR, int TILES>
struct DtSmem {
  using C = Core<DT, NR>;
  static constexpr int kRows = C::kRows * TILES, kGroups = kDtWarps / TILES;
  // Blocks an SM holds, by registers (its four parts hold 512 a lane each: four warps of 128, three of
  // 168) and shared memory.
  static constexpr int kResident = sizeof(DT) == 2 && kRows <= 16 ? 3 : 2;
  // of the ring; a multiple of the groups, so that a slot is always the same group's
  static constexpr int kSlots = TILES == 1 ? 8 : 4;
  static constexpr int kRegs = kResident == 3 ? 128 : 168;
  // byte offsets in dynamic shared memory (its base is 1024-byte aligned)
  static constexpr int kAcc = kSlots * kSlotBytes;
  static constexpr int kMax = kAcc + kRows * kAccStride * 4;
  static constexpr int kSum = kMax + (kGroups + 1) * kRows * 4;
  static constexpr int kZero = (kSum + (kGroups + 1) * kRows * 4 + 127) / 128 * 128;
  static constexpr int kQuery = kZero + 128;
  static constexpr int kDraft = kQuery + TILES * C::kQueryBytes;
  static size_t bytes(int B, int T) { return kDraft + static_cast<size_t>(T) * kD * 4 + schedule_bytes(B); }
};

template <typename DT, int NR, int TILES>
__global__ void __launch_bounds__(kDtThreads) __maxnreg__((DtSmem<DT, NR, TILES>::kRegs))
    dense_tree_kernel(const __grid_constant__ DenseTreeArgs da, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v) {
  using S = DtSmem<DT, NR, TILES>;
  using C = Core<DT, NR>;
  constexpr int UNIT = kUnit<DT>, ROWS = S::kRows, GROUPS = S::kGroups;
  constexpr int kSlots = S::kSlots, kRaw = sizeof(DT);  // (16 values of a quad's lane in 16-byte words)
  static_assert(kSlots % GROUPS == 0, "a slot belongs to one group");
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(8) uint64_t full_bar[kSlots], empty_bar[kSlots];
  __shared__ volatile int s_err;
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
  const Schedule sch = schedule_at(smem + S::kDraft + a.T * kD * 4, a.B);
  build_schedule<UNIT, ROWS>(a, sch);
  const long long cost = sch.start[a.B];
  const int sharing = sharing_blocks(cost, da.blocks);
  if (static_cast<int>(blockIdx.x) >= sharing) return;
  const long long u0 = cut(cost, sharing, blockIdx.x), u1 = cut(cost, sharing, blockIdx.x + 1);

  // ===================================================================== feeder
  if (warp == kDtWarps) {
    const int box = min(UNIT, 1 << a.page_shift);  // rows a copy
    int count = 0, seq = -1, first = 0, page = 0;  // lane x holds the page of entry first + x
    bool stop = false;
    for (long long u = u0; u < u1 && !stop;) {
      const Task k = task_of<UNIT, ROWS>(a, sch, u, u1);
      for (int i = k.first; i < k.last && !stop; ++i, ++count) {
        const int slot = count % kSlots;
        const int rows = min(UNIT, k.len - i * UNIT), boxes = (rows + box - 1) / box;  // none of an empty cache
        const int entry = (i * UNIT) >> a.page_shift;
        if (boxes > 0 && (seq != k.b || entry < first || entry + boxes > first + 32)) {
          seq = k.b;
          first = entry;
          page = entry + lane < a.max_pages ? __ldg(a.table + static_cast<size_t>(k.b) * a.max_pages + entry + lane) : 0;
        }
        int ok = 1;
        if (lane == 0) ok = !s_err && mbar_wait_backoff(&empty_bar[slot], ((count / kSlots) & 1) ^ 1, da.wait_ns);
        if (!__shfl_sync(0xffffffffu, ok, 0)) {
          s_err = 1;
          stop = true;
          break;
        }
        const uint32_t dst = smem_addr(smem + slot * kSlotBytes);
        if (lane == 0) mbar_arrive_tx(&full_bar[slot], boxes * box * 2 * kD * static_cast<int>(sizeof(DT)));
        for (int x = 0; x < boxes; ++x) {
          int id = __shfl_sync(0xffffffffu, page, entry + x - first);
          if (lane == 0) {
            if (id < 0 || id >= a.n_pages) {
              atomicExch(a.status, kStatusDeviceAssert);
              id = 0;
            }
            const int y = ((id * a.H + k.h) << a.page_shift) + ((i * UNIT) & ((1 << a.page_shift) - 1));
            const uint32_t at = dst + x * box * 128;
            tma_2d(at, &map_k, 0, y, &full_bar[slot]);
            tma_2d(at + kHalf, &map_v, 0, y, &full_bar[slot]);
            if constexpr (sizeof(DT) == 4) {
              tma_2d(at + kHalf / 2, &map_k, 32, y, &full_bar[slot]);
              tma_2d(at + kHalf + kHalf / 2, &map_v, 32, y, &full_bar[slot]);
            }
          }
        }
      }
      u = k.start + k.units + kTaskCost;
    }
    // nothing may be in flight when the block ends
    if (lane == 0) {
      for (int c = count - kSlots < 0 ? 0 : count - kSlots; c < count; ++c)
        mbar_wait(&full_bar[c % kSlots], (c / kSlots) & 1, da.wait_ns);
      if (s_err) atomicExch(a.status, kStatusTimeout);
    }
    return;
  }

  // ===================================================================== computing warps
  const int t = lane & 3, tile = warp % TILES, grp = warp / TILES;
  float* s_acc = reinterpret_cast<float*>(smem + S::kAcc);
  float* s_max = reinterpret_cast<float*>(smem + S::kMax);
  float* s_sum = reinterpret_cast<float*>(smem + S::kSum);
  float* s_draft = reinterpret_cast<float*>(smem + S::kDraft);
  const uint32_t ring = smem_addr(smem), zero = smem_addr(smem + S::kZero);
  int count = 0;
  for (long long u = u0; u < u1;) {
    const Task k = task_of<UNIT, ROWS>(a, sch, u, u1);
    u = k.start + k.units + kTaskCost;
    if (k.first == k.last) continue;
    const bool tail = k.last == k.units, whole = tail && k.first == 0;
    const int r0 = k.rb * ROWS, rows = min(ROWS, a.G * k.n - r0);  // row r0 + i is (query head, node)
    bool ok = true;
    const WarpTree tree = warp_tree(a.parent == nullptr ? nullptr : a.parent + static_cast<size_t>(k.b) * a.T, k.n, &ok);
    auto position = [&](int depth) {
      if (k.len + depth >= a.N) {
        ok = false;
        return a.N - 1;
      }
      return k.len + depth;
    };
    auto row_of = [&](int r, int& s) {  // the row of q and o
      const int head = r / k.n;
      s = r - head * k.n;
      return (static_cast<size_t>(k.b) * a.Hq + k.h * a.G + head) * a.T + s;
    };
    uint4* qs = reinterpret_cast<uint4*>(smem + S::kQuery + tile * C::kQueryBytes);
    for (int i = grp; i < C::kLoads; i += GROUPS) {
      const int r = C::kRows * tile + C::load_row(i);
      int s = 0;
      const size_t row = r < rows ? row_of(r0 + r, s) : 0;
      const int depth = pick32(tree.depth, s);
      C::load_query(a, qs, i, r < rows, row, r < rows ? position(depth) : 0);
    }
    const size_t fresh = (static_cast<size_t>(k.b) * a.H + k.h) * a.T * kD;
    const DT* vn = static_cast<const DT*>(a.vn) + fresh;
    if (tail) {
      // drafted keys, rotated, then a quad a row over its ancestors
      const DT* kn = static_cast<const DT*>(a.kn) + fresh;
      for (int x = 0; x < (k.n + kDtCons / 4 - 1) / (kDtCons / 4); ++x) {
        const int s = x * (kDtCons / 4) + (tid >> 2);
        const int depth = pick32(tree.depth, s & 63);
        if (s < k.n) {
          float y[16];
          float2 e[8];
          load_part(kn + static_cast<size_t>(s) * kD, t, y);
          // the values too, into L1: the rows' loops below would wait for each in turn
          const char* vr = reinterpret_cast<const char*>(vn + static_cast<size_t>(s) * kD) + t * (kD * sizeof(DT) / 4);
          asm volatile("{ .reg .b32 x; ld.global.nc.b32 x, [%0]; }\n" ::"l"(vr));
          rope_row(a.rope_lo, a.rope_hi, position(depth), t, e);
          rotate_part(y, e, false);
          store_part(s_draft + s * kD, t, y);
        }
      }
    }
    cons_sync();
    if (tail) {
      for (int x = 0; x < (rows + kDtCons / 4 - 1) / (kDtCons / 4); ++x) {
        const int r = x * (kDtCons / 4) + (tid >> 2);
        const bool in = r < rows;
        int s = 0;
        const size_t row = in ? row_of(r0 + r, s) : 0;
        const int depth = pick32(tree.depth, s);
        uint64_t set = pick64(tree.above, s);
        if (!in) set = 0;
        float y[16], o[16], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < 16; ++w) y[w] = o[w] = 0.f;
        if (in) {
          float2 e[8];
          load_part(static_cast<const DT*>(a.q) + row * kD, t, y);
          rope_row(a.rope_lo, a.rope_hi, position(depth), t, e);
          rotate_part(y, e, false);
#pragma unroll
          for (int w = 0; w < 16; ++w) y[w] *= kLog2e / 8.0f;
        }
        // the values of the next ancestor are on their way while one is added
        uint4 next[kRaw];
        int key = set != 0 ? __ffsll(static_cast<long long>(set)) - 1 : 0;
        if (set != 0) load_raw(vn + static_cast<size_t>(key) * kD, t, next);
        while (__any_sync(0xffffffffu, set != 0)) {
          const bool on = set != 0;
          float sc = 0.f, v[16];
          raw_to_float(next, v, vn);
          if (on) {
            float kx[16];
            const float4* kr = reinterpret_cast<const float4*>(s_draft + key * kD);
            *reinterpret_cast<float4*>(kx) = kr[2 * t];
            *reinterpret_cast<float4*>(kx + 4) = kr[2 * t + 1];
            *reinterpret_cast<float4*>(kx + 8) = kr[8 + 2 * t];
            *reinterpret_cast<float4*>(kx + 12) = kr[8 + 2 * t + 1];
#pragma unroll
            for (int w = 0; w < 16; ++w) sc = fmaf(y[w], kx[w], sc);
          }
          set &= set - 1;
          if (set != 0) {
            key = __ffsll(static_cast<long long>(set)) - 1;
            load_raw(vn + static_cast<size_t>(key) * kD, t, next);
          }
          sc = quad_sum(sc);
          if (on && sc != -INFINITY) {  // weight 0 (a NaN goes on)
            const float mn = fmaxf(m, sc);
            const float corr = ex2(m - mn), p = ex2(sc - mn);
            l = l * corr + p;
#pragma unroll
            for (int w = 0; w < 16; ++w) o[w] = fmaf(p, v[w], o[w] * corr);
            m = mn;
          }
        }
        if (in) {
          store_part(s_acc + r * kAccStride, t, o);
          if (t == 0) {
            s_max[GROUPS * ROWS + r] = m;
            s_sum[GROUPS * ROWS + r] = l;
          }
        }
      }
    }
    // ---- the cached rows: a unit in turn for each group
    C core;
    core.clear();
    for (int i = k.first; i < k.last; ++i, ++count) {
      if (count % GROUPS != grp) continue;
      const int slot = count % kSlots;
      if (!s_err && !mbar_wait(&full_bar[slot], (count / kSlots) & 1, da.wait_ns)) {
        s_err = 1;
        atomicExch(a.status, kStatusTimeout);
      }
      if (!s_err) core.unit(ring + slot * kSlotBytes, qs, zero, k.len - i * UNIT);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty_bar[slot]);
    }
    // ---- merge the groups (and the drafted keys' part) in a fixed order
    core.finish();
    if (C::leader()) {
#pragma unroll
      for (int i = 0; i < C::kOwn; ++i) {
        s_max[grp * ROWS + C::kRows * tile + C::own_row(i)] = core.own_max(i);
        s_sum[grp * ROWS + C::kRows * tile + C::own_row(i)] = core.own_sum(i);
      }
    }
    cons_sync();
    const int parts = GROUPS + (tail ? 1 : 0);
    float f[C::kOwn], old[C::kOwn];
#pragma unroll
    for (int i = 0; i < C::kOwn; ++i) {
      const int r = C::kRows * tile + C::own_row(i);
      float all = -INFINITY;
#pragma unroll
      for (int x = 0; x < GROUPS; ++x) all = fmaxf(all, s_max[x * ROWS + r]);
      const bool drafts = tail && r < rows;
      const float md = drafts ? s_max[GROUPS * ROWS + r] : -INFINITY;
      all = fmaxf(all, md);
      f[i] = weight_of(core.own_max(i), core.own_sum(i), all);
      old[i] = grp > 0 ? 1.f : drafts ? weight_of(md, s_sum[GROUPS * ROWS + r], all) : 0.f;
    }
    for (int turn = 0; turn < GROUPS; ++turn) {
      if (grp == turn) {
#pragma unroll
        for (int i = 0; i < C::kOwn; ++i) {
          const int r = C::kRows * tile + C::own_row(i);
          if (r < rows) core.add_to(i, s_acc + r * kAccStride, old[i], turn > 0 || tail, f[i]);
        }
      }
      cons_sync();
    }
    if (!ok) atomicExch(a.status, kStatusDeviceAssert);
    if (!s_err) {
      // row max and sum, by the threads that write the row: 16 a row
      float* part = da.part + (static_cast<size_t>(blockIdx.x) * 2 + (k.start >= u0 ? 1 : 0)) * ROWS * kDtPart;
      for (int i = tid; i < rows * 16; i += kDtCons) {
        const int r = i >> 4, d = (i & 15) * 4;
        float mr = -INFINITY, sum = 0.f;
        for (int x = 0; x < parts; ++x) mr = fmaxf(mr, s_max[x * ROWS + r]);
        for (int x = 0; x < parts; ++x)
          sum += s_sum[x * ROWS + r] * weight_of(s_max[x * ROWS + r], s_sum[x * ROWS + r], mr);
        const float4 x = *reinterpret_cast<const float4*>(s_acc + r * kAccStride + d);
        if (whole) {
          int s;
          const size_t row = row_of(r0 + r, s);
          const float inv = 1.f / sum;
          if constexpr (sizeof(DT) == 4) {
            *reinterpret_cast<float4*>(static_cast<float*>(a.o) + row * kD + d) =
                make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
          } else {
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + row * kD + d) =
                make_uint2(pack_bf2(x.x * inv, x.y * inv), pack_bf2(x.z * inv, x.w * inv));
          }
          if (d == 0 && a.lse != nullptr) a.lse[row] = (mr + log2f(sum)) * kLn2;
        } else {
          *reinterpret_cast<float2*>(part + r * kDtPart + d) = make_float2(x.x, x.y);
          *reinterpret_cast<float2*>(part + r * kDtPart + d + 2) = make_float2(x.z, x.w);
          if (d == 0) *reinterpret_cast<float2*>(part + r * kDtPart + kD) = make_float2(mr, sum);
        }
      }
    }
    cons_sync();  // s_acc, s_max and s_sum are free again
  }
}

// Adds the partials of the tasks whose units more than one block holds.  Block (c, y) serves 8 rows of the task
// whose first cut is the one in front of block c.  A row has two teams of 16 threads, which take every
// second partial; the weights come first, so that the loads of O do not wait for one another.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 8;

template <typename DT, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ DenseTreeArgs da) {
  constexpr int UNIT = kUnit<DT>;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ float4 s_o[kJoinRows][16];
  const TreeArgs& a = da.a;
  const Schedule sch = schedule_at(smem, a.B);
  build_schedule<UNIT, ROWS>(a, sch);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const long long cost = sch.start[a.B];
  const int sharing = sharing_blocks(cost, da.blocks);
  const int c = blockIdx.x;
  if (c == 0 || c >= sharing) return;
  const long long u = cut(cost, sharing, c);
  const Task k = task_of<UNIT, ROWS>(a, sch, u, cost);
  // the cut lies behind the task's first unit, and is the first that does
  const long long t0 = k.start + kTaskCost, t1 = t0 + k.units;
  if (u <= t0 || cut(cost, sharing, c - 1) > t0) return;
  const int r0 = k.rb * ROWS, rows = min(ROWS, a.G * k.n - r0);
  const int team = threadIdx.x >> 4, d = (threadIdx.x & 15) * 4, share = team & 1, at = team >> 1;
  const int r = kJoinRows * blockIdx.y + at;
  if (kJoinRows * static_cast<int>(blockIdx.y) >= rows) return;
  const int parts = block_at(cost, sharing, t1 - 1) - (c - 1) + 1;  // blocks that hold some of it
  // partial i lies in block c - 1 + i: in its first place, or its second where the block began before the task
  const int first_slot = k.start >= cut(cost, sharing, c - 1) ? 1 : 0;
  auto partial = [&](int i) {
    const int slot = i == 0 ? first_slot : 0;
    return da.part + ((static_cast<size_t>(c - 1 + i) * 2 + slot) * ROWS + r) * kDtPart;
  };
  float all = -INFINITY, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r < rows) {
    for (int i = threadIdx.x & 15; i < parts; i += 16) all = fmaxf(all, partial(i)[kD]);
  }
#pragma unroll
  for (int x = 1; x < 16; x <<= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, x));
  if (r < rows) {
    for (int i = threadIdx.x & 15; i < parts; i += 16) {
      const float2 ml = *reinterpret_cast<const float2*>(partial(i) + kD);
      sum += ml.y * weight_of(ml.x, ml.y, all);
    }
  }
#pragma unroll
  for (int x = 1; x < 16; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  if (r < rows) {
#pragma unroll 4
    for (int i = share; i < parts; i += 2) {
      const float* p = partial(i);
      const float2 x = *reinterpret_cast<const float2*>(p + d), y = *reinterpret_cast<const float2*>(p + d + 2);
      const float2 ml = *reinterpret_cast<const float2*>(p + kD);
      const float f = weight_of(ml.x, ml.y, all);
      o.x += x.x * f;
      o.y += x.y * f;
      o.z += y.x * f;
      o.w += y.y * f;
    }
  }
  if (share) s_o[at][d / 4] = o;
  __syncthreads();
  if (share || r >= rows) return;
  const float4 x = s_o[at][d / 4];
  const float inv = 1.f / sum;
  o = make_float4((o.x + x.x) * inv, (o.y + x.y) * inv, (o.z + x.z) * inv, (o.w + x.w) * inv);
  const int head = (r0 + r) / k.n, s = (r0 + r) - head * k.n;
  const size_t row = (static_cast<size_t>(k.b) * a.Hq + k.h * a.G + head) * a.T + s;
  if constexpr (sizeof(DT) == 4)
    *reinterpret_cast<float4*>(static_cast<float*>(a.o) + row * kD + d) = o;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + row * kD + d) =
        make_uint2(pack_bf2(o.x, o.y), pack_bf2(o.z, o.w));
  if (d == 0 && a.lse != nullptr) a.lse[row] = (all + log2f(sum)) * kLn2;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A layer's pool as a matrix of rows of 64 values; a copy takes `box` rows of 128 bytes.
cudaError_t map_of(CUtensorMap* m, const void* pool, long long rows, int es, int box) {
  static const EncodeTiled encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<EncodeTiled>(fn);
  }();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {kD, static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kD) * es};
  const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(box)};
  const cuuint32_t steps[2] = {1, 1};
  const CUresult r = encode(m, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                            const_cast<void*>(pool), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Calls f.template operator()<NR, TILES>() with the shape for `rows` query rows of a key head: as few
// rows as hold them all, 64 at most.
template <typename DT, typename F>
auto with_shape(int rows, F&& f) {
  if constexpr (sizeof(DT) == 4) {
    if (rows <= 16) return f.template operator()<2, 1>();
    if (rows <= 32) return f.template operator()<2, 2>();
    return f.template operator()<2, 4>();
  } else {
    if (rows <= 8) return f.template operator()<1, 1>();
    if (rows <= 16) return f.template operator()<2, 1>();
    if (rows <= 24) return f.template operator()<3, 1>();
    if (rows <= 32) return f.template operator()<4, 1>();
    if (rows <= 48) return f.template operator()<3, 2>();
    return f.template operator()<4, 2>();
  }
}

template <typename DT, int NR, int TILES>
constexpr int kGrid = 152 * DtSmem<DT, NR, TILES>::kResident;  // 152 SMs

template <typename DT, int NR, int TILES>
cudaError_t launch(const DenseTreeArgs& args, cudaStream_t stream) {
  using S = DtSmem<DT, NR, TILES>;
  DenseTreeArgs da = args;
  da.blocks = kGrid<DT, NR, TILES>;
  const TreeArgs& a = da.a;
  const int es = static_cast<int>(sizeof(DT));
  const int box = (1 << a.page_shift) < kUnit<DT> ? 1 << a.page_shift : kUnit<DT>;
  const long long rows = (static_cast<long long>(a.n_pages) * a.H) << a.page_shift;
  CUtensorMap mk, mv;
  cudaError_t e = map_of(&mk, a.kc, rows, es, box);
  if (e == cudaSuccess) e = map_of(&mv, a.vc, rows, es, box);
  if (e != cudaSuccess) return e;
  const size_t smem = S::bytes(a.B, a.T);
  e = cudaFuncSetAttribute(dense_tree_kernel<DT, NR, TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  dense_tree_kernel<DT, NR, TILES><<<da.blocks, kDtThreads, smem, stream>>>(da, mk, mv);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int most = a.G * a.T < S::kRows ? a.G * a.T : S::kRows;
  cfg.gridDim = dim3(static_cast<unsigned>(da.blocks), (most + kJoinRows - 1) / kJoinRows);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = schedule_bytes(a.B);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<DT, S::kRows>, da);
}

template <typename DT>
size_t part_bytes(int rows) {
  return with_shape<DT>(rows, []<int NR, int TILES>() {
    return static_cast<size_t>(kGrid<DT, NR, TILES>) * 2 * DtSmem<DT, NR, TILES>::kRows * kDtPart * sizeof(float);
  });
}

template <typename DT>
cudaError_t launch_rows(const DenseTreeArgs& da, cudaStream_t stream) {
  return with_shape<DT>(da.a.G * da.a.T, [&]<int NR, int TILES>() { return launch<DT, NR, TILES>(da, stream); });
}

}  // namespace

size_t dense_tree_workspace_bytes(int B, int Hq, int H, int T, int dtype) {
  const int rows = Hq / H * T;
  return dtype == FIB_DTYPE_F32 ? part_bytes<float>(rows) : part_bytes<__nv_bfloat16>(rows);
}

cudaError_t launch_dense_tree(const TreeArgs& a, int dtype, unsigned long long wait_ns, void* ws, cudaStream_t stream) {
  DenseTreeArgs da;
  da.a = a;
  da.part = static_cast<float*>(ws);
  da.wait_ns = wait_ns;
  da.blocks = 0;
  return dtype == FIB_DTYPE_F32 ? launch_rows<float>(da, stream) : launch_rows<__nv_bfloat16>(da, stream);
}

}  // namespace fibattn
