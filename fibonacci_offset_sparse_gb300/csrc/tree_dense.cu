// Dense decode of a tree of drafted tokens over the paged cache (sm_103a): the dense control's
// form of tree.cu.  Node s of a sequence attends every cached row, its ancestors and itself:
// O_s = sum_j p_sj v_j, p = softmax(q'_s . k'_j / 8).
//
// What bounds it: every cached row is read once for all nodes and query heads of its key head, so up to some
// 64 rows of queries a key the read of the cache from HBM is the floor.
//
// Work: a unit is kUnit consecutive cached rows of one task; a task is a (sequence, key head, block of
// ROWS query rows).  The units of all tasks, in that order, are cut into one equal run a block
// (split of the long axis), whatever the lengths are: lengths live on the device, so every block
// computes the cut from them.  A block that holds a whole task writes its outputs; else it leaves a
// partial (max, sum, unnormalised O) in the workspace and join_kernel adds the partials of a
// task in the order of the blocks.
//
// Block: 4 warps that compute and one that feeds them.  The feeder copies K and V rows of a unit by
// TMA (128-byte swizzle) into a ring of 16 KB slots, a page at a time.  The computing warps are MT
// row tiles of 16 query rows times 4 / MT groups of keys; each keeps an online softmax (running
// maximum and sum, O in registers) over its keys, and the groups merge at the end of the run.
//   bf16: mma.sync m16n8k16.  K and V enter as they are stored; the rotated query and the softmax weights
//   are split in two bf16 (x = hi + lo, 16 bits of significand), each product twice, so that neither is
//   rounded to 8 bits.
//   float32: mma.sync m16n8k8 on tf32 with both operands split (hi, lo): hi*hi + hi*lo + lo*hi, 21 bits.
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
constexpr int kDtSlots = 4;
constexpr int kDtSlotBytes = 16384;  // K then V of a unit
constexpr int kDtHalf = kDtSlotBytes / 2;
constexpr int kDtPart = kD + 2;      // floats of a partial's row: O, max, sum

template <typename DT>
constexpr int kUnit = kDtHalf / (kD * static_cast<int>(sizeof(DT)));  // 64 rows (bf16), 32 (float32)

struct DenseTreeArgs {
  TreeArgs a;
  float* part;  // [blocks][2][ROWS][kDtPart]
  unsigned long long wait_ns;
  int blocks;   // blocks of the grid
};

// ------------------------------------------------------------------------------ schedule --
// In shared memory: units before each sequence, and the sequences' rows and nodes.
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
    s.start[b + 1] = n == 0 ? 0 : static_cast<long long>(units_of<UNIT>(len)) * a.H * ((a.G * n + ROWS - 1) / ROWS);
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

// How many of the grid's blocks share `units`: at least two units each while there are fewer
// than two a block (a block's fixed cost is that of several units).
__device__ __forceinline__ int sharing_blocks(long long units, int blocks) {
  const long long want = (units + 1) / 2;
  return want < blocks ? static_cast<int>(want) : blocks;
}
__device__ __forceinline__ long long cut(long long units, int sharing, int c) { return units * c / sharing; }

// The task that unit u belongs to.
struct Task {
  int b, h, rb;
  int len, n;
  int units, first;  // units of the task; u's place among them
};
template <int UNIT, int ROWS>
__device__ __forceinline__ Task task_of(const TreeArgs& a, const Schedule& s, long long u) {
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
  const int rbs = (a.G * t.n + ROWS - 1) / ROWS;
  const long long off = u - s.start[lo];
  const int task = static_cast<int>(off / t.units);
  t.first = static_cast<int>(off - static_cast<long long>(task) * t.units);
  t.h = task / rbs;
  t.rb = task - t.h * rbs;
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

__device__ __forceinline__ void cons_sync() { asm volatile("bar.sync 1, %0;\n" ::"n"(kDtCons) : "memory"); }

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

// The rotated query of row r of a task, times log2(e)/8, as A fragments (hi, lo) of a warp's row
// tile: lane (g, t) holds rows g and g + 8.
template <typename DT>
struct QFrag;
template <>
struct QFrag<__nv_bfloat16> {
  uint32_t hi[4][4], lo[4][4];  // [k-step of 16 dims][fragment]
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int u = 0; u < 4; ++u) hi[s][u] = lo[s][u] = 0;
  }
  __device__ __forceinline__ void load(const TreeArgs& a, size_t row, int pos, int half) {
    const int t = threadIdx.x & 3;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) + row * kD);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int m = 16 * s + 8 * f + 2 * t;
        const uint32_t x = __ldg(q + m / 2), y = __ldg(q + m / 2 + kFreq / 2);
        const float2 e0 = rope_factor(a.rope_lo, a.rope_hi, pos, m), e1 = rope_factor(a.rope_lo, a.rope_hi, pos, m + 1);
        const float sc = kLog2e / 8.0f;
        const float x0 = bf_lo(x) * sc, x1 = bf_hi(x) * sc, y0 = bf_lo(y) * sc, y1 = bf_hi(y) * sc;
        split_bf16(x0 * e0.x - y0 * e0.y, x1 * e1.x - y1 * e1.y, hi[s][2 * f + half], lo[s][2 * f + half]);
        split_bf16(x0 * e0.y + y0 * e0.x, x1 * e1.y + y1 * e1.x, hi[s + 2][2 * f + half], lo[s + 2][2 * f + half]);
      }
  }
};
template <>
struct QFrag<float> {
  uint32_t hi[8][4], lo[8][4];  // [k-step of 8 dims][fragment]
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int s = 0; s < 8; ++s)
#pragma unroll
      for (int u = 0; u < 4; ++u) hi[s][u] = lo[s][u] = 0;
  }
  __device__ __forceinline__ void load(const TreeArgs& a, size_t row, int pos, int half) {
    const int t = threadIdx.x & 3;
    const float* q = static_cast<const float*>(a.q) + row * kD;
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int m = 8 * s + 4 * f + t;
        const float2 e = rope_factor(a.rope_lo, a.rope_hi, pos, m);
        const float x = __ldg(q + m) * (kLog2e / 8.0f), y = __ldg(q + m + kFreq) * (kLog2e / 8.0f);
        split_tf32(x * e.x - y * e.y, hi[s][2 * f + half], lo[s][2 * f + half]);
        split_tf32(x * e.y + y * e.x, hi[s + 4][2 * f + half], lo[s + 4][2 * f + half]);
      }
  }
};

// Scores of 8 keys (rows key0 .. key0 + 7 of the K tile) against the row tile: lane (g, t) gets keys
// key0 + 2t, + 1 of rows g (c[0], c[1]) and g + 8 (c[2], c[3]).  HI: the upper parts' product alone (an
// infinity keeps its sign there, where hi + lo may add two of opposite signs).
template <bool HI>
__device__ __forceinline__ void scores8(const QFrag<__nv_bfloat16>& q, uint32_t kt, int key0, float (&c)[4]) {
  const int mi = (threadIdx.x & 31) >> 3, rl = threadIdx.x & 7;
  const uint32_t row = kt + (key0 + rl) * 128;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint32_t b[4];
    ldsm_x4(b, row + (((4 * p + mi) ^ rl) << 4));
    mma_bf16(c, q.hi[2 * p], b[0], b[1]);
    if constexpr (!HI) mma_bf16(c, q.lo[2 * p], b[0], b[1]);
    mma_bf16(c, q.hi[2 * p + 1], b[2], b[3]);
    if constexpr (!HI) mma_bf16(c, q.lo[2 * p + 1], b[2], b[3]);
  }
}
template <bool HI>
__device__ __forceinline__ void scores8(const QFrag<float>& q, uint32_t kt, int key0, float (&c)[4]) {
  const int mi = (threadIdx.x & 31) >> 3, rl = threadIdx.x & 7;
  const uint32_t row = kt + (key0 + rl) * 128;  // dims 0..31, then 32..63 a half tile further
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    uint32_t b[4];
    ldsm_x4(b, row + (p >> 1) * (kDtHalf / 2) + (((4 * (p & 1) + mi) ^ rl) << 4));
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t h0, l0, h1, l1;
      split_tf32(__uint_as_float(b[2 * s]), h0, l0);
      split_tf32(__uint_as_float(b[2 * s + 1]), h1, l1);
      mma_tf32(c, q.hi[2 * p + s], h0, h1);
      if constexpr (!HI) {
        mma_tf32(c, q.lo[2 * p + s], h0, h1);
        mma_tf32(c, q.hi[2 * p + s], l0, l1);
      }
    }
  }
}

// O += P V over the keys of NT score tiles (keys key0 + 8 nt + 2t, + 1 of lane (g, t)).  Rows from
// `valid` on are read from `zero`, 128 bytes of 0: what lies there was not copied for this sequence.
template <int NT>
__device__ __forceinline__ void add_values(const __nv_bfloat16*, const float (&p)[NT][4], uint32_t vt, uint32_t zero, int key0,
                                           int valid, float (&o)[8][4]) {
  const int mi = (threadIdx.x & 31) >> 3, rl = threadIdx.x & 7;
#pragma unroll
  for (int j = 0; j < NT / 2; ++j) {
    uint32_t hi[4], lo[4];
    split_bf16(p[2 * j][0], p[2 * j][1], hi[0], lo[0]);
    split_bf16(p[2 * j][2], p[2 * j][3], hi[1], lo[1]);
    split_bf16(p[2 * j + 1][0], p[2 * j + 1][1], hi[2], lo[2]);
    split_bf16(p[2 * j + 1][2], p[2 * j + 1][3], hi[3], lo[3]);
    const int key = key0 + 16 * j + (mi & 1) * 8 + rl;
    const uint32_t row = key < valid ? vt + key * 128 : zero;
#pragma unroll
    for (int nd = 0; nd < 8; nd += 2) {
      uint32_t b[4];
      ldsm_x4_t(b, row + (((nd + (mi >> 1)) ^ rl) << 4));
      mma_bf16(o[nd], hi, b[0], b[1]);
      mma_bf16(o[nd], lo, b[0], b[1]);
      mma_bf16(o[nd + 1], hi, b[2], b[3]);
      mma_bf16(o[nd + 1], lo, b[2], b[3]);
    }
  }
}
template <int NT>
__device__ __forceinline__ void add_values(const float*, const float (&p)[NT][4], uint32_t vt, uint32_t zero, int key0, int valid,
                                           float (&o)[8][4]) {
  // k index t of the product is key 2t, t + 4 is key 2t + 1: what a lane holds of the scores
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint32_t hi[4], lo[4];
    split_tf32(p[nt][0], hi[0], lo[0]);
    split_tf32(p[nt][2], hi[1], lo[1]);
    split_tf32(p[nt][1], hi[2], lo[2]);
    split_tf32(p[nt][3], hi[3], lo[3]);
    const int k0 = key0 + 8 * nt + 2 * t, k1 = k0 + 1;
    const uint32_t r0 = k0 < valid ? vt + k0 * 128 : zero, r1 = k1 < valid ? vt + k1 * 128 : zero;
    const uint32_t s0 = k0 < valid ? kDtHalf / 2 : 0, s1 = k1 < valid ? kDtHalf / 2 : 0;
#pragma unroll
    for (int nd = 0; nd < 8; ++nd) {
      const int ch = 2 * (nd & 3) + (g >> 2);
      uint32_t h0, l0, h1, l1;
      split_tf32(lds_f32(r0 + (nd >> 2) * s0 + ((ch ^ (k0 & 7)) << 4) + (g & 3) * 4), h0, l0);
      split_tf32(lds_f32(r1 + (nd >> 2) * s1 + ((ch ^ (k1 & 7)) << 4) + (g & 3) * 4), h1, l1);
      mma_tf32(o[nd], hi, h0, h1);
      mma_tf32(o[nd], lo, h0, h1);
      mma_tf32(o[nd], hi, l0, l1);
    }
  }
}

// ------------------------------------------------------------------------------ the kernel --
template <typename DT, int MT>
struct DtSmem {
  static constexpr int kRows = 16 * MT, kGroups = kDtWarps / MT;
  // byte offsets in dynamic shared memory (its base is 1024-byte aligned)
  static constexpr int kAcc = kDtSlots * kDtSlotBytes;
  static constexpr int kMax = kAcc + kRows * kD * 4;
  static constexpr int kSum = kMax + (kGroups + 1) * kRows * 4;
  static constexpr int kZero = kSum + (kGroups + 1) * kRows * 4;
  static constexpr int kDraft = kZero + 128;
  static size_t bytes(int B, int T) { return kDraft + static_cast<size_t>(T) * kD * 4 + schedule_bytes(B); }
};

template <typename DT, int MT>
__global__ void __launch_bounds__(kDtThreads, sizeof(DT) == 2 ? 3 : 2)
    dense_tree_kernel(const __grid_constant__ DenseTreeArgs da, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v) {
  using S = DtSmem<DT, MT>;
  constexpr int UNIT = kUnit<DT>, ROWS = S::kRows, GROUPS = S::kGroups;
  constexpr int KW = UNIT / GROUPS, NT = KW / 8;  // keys of a unit a warp takes
  static_assert(sizeof(DT) == 4 || NT % 2 == 0, "a bf16 product takes 16 keys");
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(8) uint64_t full_bar[kDtSlots], empty_bar[kDtSlots];
  __shared__ volatile int s_err;
  const TreeArgs& a = da.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (tid == 0) {
    s_err = 0;
    for (int s = 0; s < kDtSlots; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], kDtWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (tid < 32) reinterpret_cast<float*>(smem + S::kZero)[tid] = 0.f;
  const Schedule sch = schedule_at(smem + S::kDraft + a.T * kD * 4, a.B);
  build_schedule<UNIT, ROWS>(a, sch);
  const long long units = sch.start[a.B];
  const int sharing = sharing_blocks(units, da.blocks);
  if (static_cast<int>(blockIdx.x) >= sharing) return;
  const long long u0 = cut(units, sharing, blockIdx.x), u1 = cut(units, sharing, blockIdx.x + 1);

  // ===================================================================== feeder
  if (warp == kDtWarps) {
    const int box = min(UNIT, 1 << a.page_shift);  // rows a copy
    int count = 0, seq = -1, first = 0, page = 0;  // lane x holds the page of entry first + x
    bool stop = false;
    for (long long u = u0; u < u1 && !stop;) {
      const Task k = task_of<UNIT, ROWS>(a, sch, u);
      const int end = static_cast<int>(min(static_cast<long long>(k.units), k.first + (u1 - u)));
      for (int i = k.first; i < end && !stop; ++i, ++count) {
        const int slot = count % kDtSlots;
        const int rows = min(UNIT, k.len - i * UNIT), boxes = (rows + box - 1) / box;  // none of an empty cache
        const int entry = (i * UNIT) >> a.page_shift;
        if (boxes > 0 && (seq != k.b || entry < first || entry + boxes > first + 32)) {
          seq = k.b;
          first = entry;
          page = entry + lane < a.max_pages ? __ldg(a.table + static_cast<size_t>(k.b) * a.max_pages + entry + lane) : 0;
        }
        int ok = 1;
        if (lane == 0) ok = !s_err && mbar_wait_backoff(&empty_bar[slot], ((count / kDtSlots) & 1) ^ 1, da.wait_ns);
        if (!__shfl_sync(0xffffffffu, ok, 0)) {
          s_err = 1;
          stop = true;
          break;
        }
        const uint32_t dst = smem_addr(smem + slot * kDtSlotBytes);
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
            tma_2d(at + kDtHalf, &map_v, 0, y, &full_bar[slot]);
            if constexpr (sizeof(DT) == 4) {
              tma_2d(at + kDtHalf / 2, &map_k, 32, y, &full_bar[slot]);
              tma_2d(at + kDtHalf + kDtHalf / 2, &map_v, 32, y, &full_bar[slot]);
            }
          }
        }
      }
      u += end - k.first;
    }
    // nothing may be in flight when the block ends
    if (lane == 0) {
      for (int c = count - kDtSlots < 0 ? 0 : count - kDtSlots; c < count; ++c)
        mbar_wait(&full_bar[c % kDtSlots], (c / kDtSlots) & 1, da.wait_ns);
      if (s_err) atomicExch(a.status, kStatusTimeout);
    }
    return;
  }

  // ===================================================================== computing warps
  const int g = lane >> 2, t = lane & 3, tile = warp % MT, grp = warp / MT;
  float* s_acc = reinterpret_cast<float*>(smem + S::kAcc);
  float* s_max = reinterpret_cast<float*>(smem + S::kMax);
  float* s_sum = reinterpret_cast<float*>(smem + S::kSum);
  float* s_draft = reinterpret_cast<float*>(smem + S::kDraft);
  const uint32_t ring = smem_addr(smem), zero = smem_addr(smem + S::kZero);
  int count = 0;
  for (long long u = u0; u < u1;) {
    const Task k = task_of<UNIT, ROWS>(a, sch, u);
    const int end = static_cast<int>(min(static_cast<long long>(k.units), k.first + (u1 - u)));
    const bool tail = end == k.units, whole = tail && k.first == 0;
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
    QFrag<DT> q;
    q.zero();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = 16 * tile + g + 8 * half;
      int s = 0;
      size_t row = 0;
      if (r < rows) row = row_of(r0 + r, s);
      const int depth = pick32(tree.depth, s);
      if (r < rows) q.load(a, row, position(depth), half);
    }
    if (tail) {
      // drafted keys, rotated, then a quad a row over its ancestors
      const size_t fresh = (static_cast<size_t>(k.b) * a.H + k.h) * a.T * kD;
      const DT* kn = static_cast<const DT*>(a.kn) + fresh;
      const DT* vn = static_cast<const DT*>(a.vn) + fresh;
      for (int x = 0; x < (k.n + kDtCons / 4 - 1) / (kDtCons / 4); ++x) {
        const int s = x * (kDtCons / 4) + (tid >> 2);
        const int depth = pick32(tree.depth, s & 63);
        if (s < k.n) {
          float y[16];
          float2 e[8];
          load_part(kn + static_cast<size_t>(s) * kD, t, y);
          rope_row(a.rope_lo, a.rope_hi, position(depth), t, e);
          rotate_part(y, e, false);
          store_part(s_draft + s * kD, t, y);
        }
      }
      cons_sync();
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
        while (__any_sync(0xffffffffu, set != 0)) {
          const bool on = set != 0;
          const int key = on ? __ffsll(static_cast<long long>(set)) - 1 : 0;
          set &= set - 1;
          float sc = 0.f, v[16];
          if (on) {
            float kx[16];
            load_part(vn + static_cast<size_t>(key) * kD, t, v);
            const float4* kr = reinterpret_cast<const float4*>(s_draft + key * kD);
            *reinterpret_cast<float4*>(kx) = kr[2 * t];
            *reinterpret_cast<float4*>(kx + 4) = kr[2 * t + 1];
            *reinterpret_cast<float4*>(kx + 8) = kr[8 + 2 * t];
            *reinterpret_cast<float4*>(kx + 12) = kr[8 + 2 * t + 1];
#pragma unroll
            for (int w = 0; w < 16; ++w) sc = fmaf(y[w], kx[w], sc);
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
          store_part(s_acc + r * kD, t, o);
          if (t == 0) {
            s_max[GROUPS * ROWS + r] = m;
            s_sum[GROUPS * ROWS + r] = l;
          }
        }
      }
    }
    // ---- the cached rows
    float o[8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int nd = 0; nd < 8; ++nd) o[nd][0] = o[nd][1] = o[nd][2] = o[nd][3] = 0.f;
    for (int i = k.first; i < end; ++i, ++count) {
      const int slot = count % kDtSlots;
      if (!s_err && !mbar_wait(&full_bar[slot], (count / kDtSlots) & 1, da.wait_ns)) {
        s_err = 1;
        atomicExch(a.status, kStatusTimeout);
      }
      if (s_err) break;
      const uint32_t kt = ring + slot * kDtSlotBytes, vt = kt + kDtHalf;
      const int valid = min(UNIT, k.len - i * UNIT);
      const int key0 = grp * KW;
      float s[NT][4], sum[2];
      for (bool again = false;;) {  // a second time only where an infinite key made a NaN of hi + lo
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
          scores8<false>(q, kt, key0 + 8 * nt, s[nt]);
        }
        if (again) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            scores8<true>(q, kt, key0 + 8 * nt, c);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (isnan(s[nt][e])) s[nt][e] = c[e];
          }
        }
        if (valid < UNIT) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key0 + 8 * nt + 2 * t + (e & 1) >= valid) s[nt][e] = -INFINITY;
        }
        // online softmax; the reference moves only when a score passes it by more than 8 (p <= 256
        // until then)
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], s[nt][e]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        }
        if (__any_sync(0xffffffffu, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mn = fmaxf(m[h], mx[h]);
            const float corr = m[h] == -INFINITY ? 1.f : ex2(m[h] - mn);  // (nothing but zeros or a NaN yet)
            m[h] = mn;
            l[h] *= corr;
#pragma unroll
            for (int nd = 0; nd < 8; ++nd) {
              o[nd][2 * h] *= corr;
              o[nd][2 * h + 1] *= corr;
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float ref = m[h] == -INFINITY ? 0.f : m[h];  // no key yet: every weight is 0
          sum[h] = 0.f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              s[nt][2 * h + e] = ex2(s[nt][2 * h + e] - ref);
              sum[h] += s[nt][2 * h + e];
            }
        }
        if (again || !__any_sync(0xffffffffu, isnan(sum[0]) || isnan(sum[1]))) break;
        again = true;
      }
      l[0] += sum[0];
      l[1] += sum[1];
      add_values<NT>(static_cast<const DT*>(nullptr), s, vt, zero, key0, valid, o);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty_bar[slot]);
    }
    // ---- merge the groups (and the drafted keys' part) in a fixed order
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (t == 0) {
        s_max[grp * ROWS + 16 * tile + g + 8 * h] = m[h];
        s_sum[grp * ROWS + 16 * tile + g + 8 * h] = l[h];
      }
    }
    cons_sync();
    const int parts = GROUPS + (tail ? 1 : 0);
    float all[2], f[2], fd[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 16 * tile + g + 8 * h;
      float x = -INFINITY;
      if (r < rows)
        for (int i = 0; i < parts; ++i) x = fmaxf(x, s_max[i * ROWS + r]);
      all[h] = x;
      f[h] = m[h] == -INFINITY ? (l[h] == 0.f ? 0.f : 1.f) : ex2(m[h] - x);  // (no finite key, but a NaN: keep it)
      const float md = tail && r < rows ? s_max[GROUPS * ROWS + r] : -INFINITY;
      fd[h] = md == -INFINITY ? 0.f : ex2(md - x);
    }
    for (int turn = 0; turn < GROUPS; ++turn) {
      if (grp == turn) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * tile + g + 8 * h;
          if (r >= rows) continue;
#pragma unroll
          for (int nd = 0; nd < 8; ++nd) {
            float2* at = reinterpret_cast<float2*>(s_acc + r * kD + 8 * nd + 2 * t);
            float2 x = make_float2(0.f, 0.f);
            if (turn > 0 || tail) x = *at;
            if (turn == 0 && tail) {
              x.x *= fd[h];
              x.y *= fd[h];
            }
            x.x += o[nd][2 * h] * f[h];
            x.y += o[nd][2 * h + 1] * f[h];
            *at = x;
          }
        }
      }
      cons_sync();
    }
    if (!ok) atomicExch(a.status, kStatusDeviceAssert);
    if (!s_err) {
      // row max and sum, by the threads that write the row: 16 a row
      float* part = da.part + (static_cast<size_t>(blockIdx.x) * 2 + (u > u0 ? 1 : 0)) * ROWS * kDtPart;
      for (int i = tid; i < rows * 16; i += kDtCons) {
        const int r = i >> 4, d = (i & 15) * 4;
        float mr = -INFINITY, sum = 0.f;
        for (int x = 0; x < parts; ++x) mr = fmaxf(mr, s_max[x * ROWS + r]);
        for (int x = 0; x < parts; ++x) {
          const float mx = s_max[x * ROWS + r];
          sum += s_sum[x * ROWS + r] * (mx == -INFINITY ? (s_sum[x * ROWS + r] == 0.f ? 0.f : 1.f) : ex2(mx - mr));
        }
        const float4 x = *reinterpret_cast<const float4*>(s_acc + r * kD + d);
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
    u += end - k.first;
  }
}

// Adds the partials of the tasks that more than one block holds.  Block c serves the task whose
// first cut is the one before block c; 16 threads a row, groups of them share the partials and merge in order.
constexpr int kJoinThreads = 256;

template <typename DT, int MT>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ DenseTreeArgs da) {
  constexpr int UNIT = kUnit<DT>, ROWS = 16 * MT;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ float s_o[kJoinThreads / 16][kD], s_m[kJoinThreads / 16], s_l[kJoinThreads / 16];
  const TreeArgs& a = da.a;
  const Schedule sch = schedule_at(smem, a.B);
  build_schedule<UNIT, ROWS>(a, sch);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const long long units = sch.start[a.B];
  const int sharing = sharing_blocks(units, da.blocks);
  const int c = blockIdx.x;
  if (c == 0 || c >= sharing) return;
  const long long u = cut(units, sharing, c);
  const Task k = task_of<UNIT, ROWS>(a, sch, u);
  const long long t0 = u - k.first, t1 = t0 + k.units;
  if (k.first == 0 || cut(units, sharing, c - 1) > t0) return;  // no cut inside a task, or not its first
  int last = c;  // the last block that holds some of it
  while (last + 1 < sharing && cut(units, sharing, last + 1) < t1) ++last;
  const int parts = last - (c - 1) + 1;
  const int r0 = k.rb * ROWS, rows = min(ROWS, a.G * k.n - r0);
  int rp = 1;  // rows at a time, a power of two
  while (rp < rows && rp < kJoinThreads / 16) rp *= 2;
  const int team = threadIdx.x >> 4, d = (threadIdx.x & 15) * 4, teams = kJoinThreads / 16 / rp;
  const int mine = team / rp;  // which share of the partials
  for (int base = 0; base < rows; base += rp) {
    const int r = base + team % rp;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows) {
      for (int i = mine; i < parts; i += teams) {
        const int blk = c - 1 + i;
        const int slot = cut(units, sharing, blk) >= t0 ? 0 : 1;
        const float* p = da.part + ((static_cast<size_t>(blk) * 2 + slot) * ROWS + r) * kDtPart;
        const float2 x = *reinterpret_cast<const float2*>(p + d), y = *reinterpret_cast<const float2*>(p + d + 2);
        const float2 ml = *reinterpret_cast<const float2*>(p + kD);
        const float mn = fmaxf(m, ml.x);
        const float f0 = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : ex2(m - mn);
        const float f1 = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2(ml.x - mn);
        l = l * f0 + ml.y * f1;
        o.x = o.x * f0 + x.x * f1;
        o.y = o.y * f0 + x.y * f1;
        o.z = o.z * f0 + y.x * f1;
        o.w = o.w * f0 + y.y * f1;
        m = mn;
      }
      *reinterpret_cast<float4*>(&s_o[team][d]) = o;
      if (d == 0) {
        s_m[team] = m;
        s_l[team] = l;
      }
    }
    __syncthreads();
    if (mine == 0 && r < rows) {
      float all = -INFINITY, sum = 0.f;
      for (int i = 0; i < teams; ++i) all = fmaxf(all, s_m[team + i * rp]);
      o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = 0; i < teams; ++i) {
        const float mi = s_m[team + i * rp], li = s_l[team + i * rp];
        const float f = mi == -INFINITY ? (li == 0.f ? 0.f : 1.f) : ex2(mi - all);
        const float4 x = *reinterpret_cast<const float4*>(&s_o[team + i * rp][d]);
        sum += li * f;
        o.x += x.x * f;
        o.y += x.y * f;
        o.z += x.z * f;
        o.w += x.w * f;
      }
      const float inv = 1.f / sum;
      const int head = (r0 + r) / k.n, s = (r0 + r) - head * k.n;
      const size_t row = (static_cast<size_t>(k.b) * a.Hq + k.h * a.G + head) * a.T + s;
      if constexpr (sizeof(DT) == 4)
        *reinterpret_cast<float4*>(static_cast<float*>(a.o) + row * kD + d) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + row * kD + d) =
            make_uint2(pack_bf2(o.x * inv, o.y * inv), pack_bf2(o.z * inv, o.w * inv));
      if (d == 0 && a.lse != nullptr) a.lse[row] = (all + log2f(sum)) * kLn2;
    }
    __syncthreads();
  }
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

// Row tiles a block: as few as hold every query row of a key head, four at most.
int row_tiles(int rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }
// Blocks of the grid: those that share an SM (by registers and shared memory) times 152.
int grid_blocks(int dtype, int tiles) { return 152 * (dtype == FIB_DTYPE_F32 || tiles == 4 ? 2 : 3); }

template <typename DT, int MT>
cudaError_t launch(const DenseTreeArgs& da, cudaStream_t stream) {
  const TreeArgs& a = da.a;
  const int es = static_cast<int>(sizeof(DT));
  const int box = (1 << a.page_shift) < kUnit<DT> ? 1 << a.page_shift : kUnit<DT>;
  const long long rows = (static_cast<long long>(a.n_pages) * a.H) << a.page_shift;
  CUtensorMap mk, mv;
  cudaError_t e = map_of(&mk, a.kc, rows, es, box);
  if (e == cudaSuccess) e = map_of(&mv, a.vc, rows, es, box);
  if (e != cudaSuccess) return e;
  const size_t smem = DtSmem<DT, MT>::bytes(a.B, a.T);
  e = cudaFuncSetAttribute(dense_tree_kernel<DT, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  dense_tree_kernel<DT, MT><<<da.blocks, kDtThreads, smem, stream>>>(da, mk, mv);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(da.blocks));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = schedule_bytes(a.B);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<DT, MT>, da);
}

template <typename DT>
cudaError_t launch_rows(const DenseTreeArgs& da, int tiles, cudaStream_t stream) {
  if (tiles == 1) return launch<DT, 1>(da, stream);
  if (tiles == 2) return launch<DT, 2>(da, stream);
  return launch<DT, 4>(da, stream);
}

}  // namespace

size_t dense_tree_workspace_bytes(int B, int Hq, int H, int T, int dtype) {
  const int tiles = row_tiles(Hq / H * T);
  return static_cast<size_t>(grid_blocks(dtype, tiles)) * 2 * 16 * tiles * kDtPart * sizeof(float);
}

cudaError_t launch_dense_tree(const TreeArgs& a, int dtype, unsigned long long wait_ns, void* ws, cudaStream_t stream) {
  DenseTreeArgs da;
  const int tiles = row_tiles(a.G * a.T);
  da.a = a;
  da.part = static_cast<float*>(ws);
  da.wait_ns = wait_ns;
  da.blocks = grid_blocks(dtype, tiles);
  return dtype == FIB_DTYPE_F32 ? launch_rows<float>(da, tiles, stream) : launch_rows<__nv_bfloat16>(da, tiles, stream);
}

}  // namespace fibattn
