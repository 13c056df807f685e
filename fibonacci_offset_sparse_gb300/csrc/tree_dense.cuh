// What the two kernels of the dense tree decode share (tree_dense.cu, tree_dense_tc.cu): the cut of the work,
// the feeding warp, the drafted keys' part, the rows' output and the join of partials.
//
// A kernel's shape P: kUnit cached rows a unit, kRows query rows a block, kTaskCost a task's own cost in
// units, kLeast units a block at least, kSlots of the ring.
#pragma once
#include <cuda.h>

#include "tree.cuh"

namespace fibattn {

constexpr int kAccStride = 68;   // floats of a row of O in shared memory
constexpr int kDtPart = kD + 2;  // floats of a partial's row: O, max, sum

// A task whose units several blocks hold, as each of them leaves it for the join: [0] the one that its run begins
// with, [1] the one that it is the first block of.
struct Split {
  int parts;  // 0: none
  int first;  // block; the others follow it
  int slot;   // of the first block's partial; the others' lie in slot 0
  int b, h, rb, n;
  int unused;
};

struct DenseTreeArgs {
  TreeArgs a;
  float* part;   // [blocks][2][ROWS][kDtPart]
  Split* split;  // [blocks][2]
  unsigned long long wait_ns;
  int blocks;   // blocks of the grid
  int skip_copy;  // test hook: the first unit's K of every task is never copied
  uint32_t zero;  // 0, which the compiler does not know
};

// ------------------------------------------------------------------------------ schedule --
// In shared memory: the cost before each sequence, and the sequences' rows and nodes (which where n is 0 are never looked up).
template <bool PACKED>
struct Schedule {
  long long* at;  // [B + 1]
  int* rows;      // [B]
  int* nodes;     // [B]

  __device__ __forceinline__ Schedule(unsigned char* smem, int B)
      : at(reinterpret_cast<long long*>(smem)), rows(reinterpret_cast<int*>(at + B + 1)), nodes(rows + B) {}
  static size_t bytes(int B) { return (sizeof(long long) * (B + 1) + 2 * sizeof(int) * B + 127) / 128 * 128; }
  __device__ __forceinline__ long long start(int b) const { return at[b]; }
  __device__ __forceinline__ int len(int b) const { return rows[b]; }
  __device__ __forceinline__ int n(int b) const { return nodes[b]; }
  __device__ __forceinline__ void set(int b, long long start, int len, int n) const {
    at[b] = start;
    rows[b] = len;
    nodes[b] = n;
  }
  __device__ __forceinline__ void move(int b, long long start) const { at[b] = start; }
  __device__ __forceinline__ void end(int B, long long cost) const { at[B] = cost; }
  __device__ __forceinline__ long long end(int B) const { return *static_cast<volatile long long*>(at + B); }
};
// The same in half the room, for batches so long that it decides how many blocks share an SM; a little slower to look up.  Of
// a word the upper 38 bits are the cost (at most 2^16 units and kTaskCost for 1024 query heads of 64 nodes in tasks of 32 rows, or
// 1024 heads of one, for 1024 sequences), 20 the rows (below 2^20, as positions are), 6 the nodes less 1.
template <>
struct Schedule<true> {
  unsigned long long* word;  // [B + 1]

  __device__ __forceinline__ Schedule(unsigned char* smem, int) : word(reinterpret_cast<unsigned long long*>(smem)) {}
  static size_t bytes(int B) { return sizeof(unsigned long long) * (B + 1); }
  __device__ __forceinline__ long long start(int b) const { return static_cast<long long>(word[b] >> 26); }
  __device__ __forceinline__ int len(int b) const { return static_cast<int>(word[b] >> 6) & 0xfffff; }
  __device__ __forceinline__ int n(int b) const { return (static_cast<int>(word[b]) & 63) + 1; }
  __device__ __forceinline__ void set(int b, long long start, int len, int n) const {
    word[b] = static_cast<unsigned long long>(start) << 26 | static_cast<unsigned long long>(len & 0xfffff) << 6 | ((n - 1) & 63);
  }
  __device__ __forceinline__ void move(int b, long long start) const {
    word[b] = static_cast<unsigned long long>(start) << 26 | (word[b] & 0x3ffffff);
  }
  __device__ __forceinline__ void end(int B, long long cost) const { word[B] = static_cast<unsigned long long>(cost) << 26; }
  __device__ __forceinline__ long long end(int B) const {
    return static_cast<long long>(*static_cast<volatile unsigned long long*>(word + B) >> 26);
  }
};
static_assert(kMaxDrafts == 64 && kMaxSeqs == 1024 && FIB_MAX_HEADS == 1024, "bits of a word");

template <int UNIT>
__device__ __forceinline__ int units_of(int len) {
  return len <= UNIT ? 1 : (len + UNIT - 1) / UNIT;
}

// Every thread of the block; ends synchronised.
template <typename P>
__device__ __forceinline__ void build_schedule(const TreeArgs& a, const Schedule<P::kPacked>& s) {
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    int n, len;
    if (!sequence_of(a, b, &n, &len)) {
      atomicExch(a.status, kStatusDeviceAssert);
      n = len = 0;
    }
    // the sequence's own cost first
    s.set(b, n == 0 ? 0 : static_cast<long long>(units_of<P::kUnit>(len) + P::kTaskCost) * a.H * ((a.G * n + P::kRows - 1) / P::kRows), len, n);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    long long base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + static_cast<int>(threadIdx.x);
      const long long own = b < a.B ? s.start(b) : 0;
      long long x = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (static_cast<int>(threadIdx.x) >= d) x += y;
      }
      if (b < a.B) s.move(b, base + x - own);
      base += __shfl_sync(0xffffffffu, x, 31);
    }
    if (threadIdx.x == 0) s.end(a.B, base);
  }
  __syncthreads();
}

// How many of the grid's blocks share the `cost`: fewer where a block would get less than `least` units.
__device__ __forceinline__ int sharing_blocks(long long cost, int blocks, int least) {
  const long long want = (cost + least - 1) / least;
  return want < blocks ? static_cast<int>(want) : blocks;
}
// Block c's run begins at cut(c); block_at(x) is the block whose run holds place x.
__device__ __forceinline__ long long cut(long long cost, int sharing, int c) {
  if (cost < 1 << 22) return static_cast<uint32_t>(cost) * static_cast<uint32_t>(c) / static_cast<uint32_t>(sharing);  // (c < 512)
  return cost * c / sharing;
}
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
template <typename P>
__device__ __forceinline__ Task task_of(const TreeArgs& a, const Schedule<P::kPacked>& s, long long u, long long end) {
  int lo = 0, hi = a.B;  // start(lo) <= u < start(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.start(mid) <= u)
      lo = mid;
    else
      hi = mid;
  }
  Task t;
  t.b = lo;
  t.len = s.len(lo);
  t.n = s.n(lo);
  t.units = units_of<P::kUnit>(t.len);
  const int rbs = (a.G * t.n + P::kRows - 1) / P::kRows, each = t.units + P::kTaskCost;
  const long long off = u - s.start(lo);
  const int task = off < 1LL << 31 ? static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(each)) : static_cast<int>(off / each);
  t.start = s.start(lo) + static_cast<long long>(task) * each;
  t.h = task / rbs;
  t.rb = task - t.h * rbs;
  const long long last = min(end - t.start, static_cast<long long>(each)) - P::kTaskCost;
  t.first = max(0, static_cast<int>(u - t.start) - P::kTaskCost);
  t.last = max(0, static_cast<int>(last));
  return t;
}

// ------------------------------------------------------------------------------ small pieces --
// x0, x1 as bf16 pairs hi + lo
__device__ __forceinline__ void split_bf16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf2_rn(x0, x1);
  lo = pack_bf2_rn(x0 - bf_lo(hi), x1 - bf_hi(hi));
}
// ... as hi + mid + lo: all 24 bits
__device__ __forceinline__ void split_bf16(float x0, float x1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_bf2_rn(x0, x1);
  x0 -= bf_lo(hi);
  x1 -= bf_hi(hi);
  split_bf16(x0, x1, mid, lo);
}
// What a partial of maximum m and sum l counts where the common maximum is `all`.  One without a finite
// score counts nothing, unless a NaN is in it, which goes on.
__device__ __forceinline__ float weight_of(float m, float l, float all) {
  return m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : ex2(m - all);
}

// The CONS computing threads of the block.
template <int CONS>
__device__ __forceinline__ void cons_sync() {
  asm volatile("bar.sync 1, %0;\n" ::"n"(CONS) : "memory");
}

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// ------------------------------------------------------------------------------ feeder --
// For what is in flight when a block gives up: its wait is not the caller's, which may be too short for a copy.
constexpr unsigned long long kDrainNs = 2000000000ull;

// A whole warp's wait, with one answer for all its lanes: false where one of them gave up (limit_ns) or the block already
// had (s_err).  What follows, warp-wide instructions among it, is every lane's or none's.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned long long limit_ns, volatile int* s_err) {
  const bool there = !*s_err && mbar_wait(bar, parity, limit_ns);
  return __all_sync(0xffffffffu, there);
}

__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}

// The feeding warp: K and V rows of the units of [u0, u1) into the ring's slots, a page at a time.  A slot
// is K, then V, kHalf bytes each; float32 rows lie as two halves of 32 dims, a quarter slot apart.  A slot is filled again only
// when every warp that reads it has seen its rows land and is done with them: one that gives up does not release it, and the
// feeder then gives up too, so that no copy is ever under way into a slot of which another has not landed.
template <typename DT, typename P>
__device__ __forceinline__ void feed(const DenseTreeArgs& da, const Schedule<P::kPacked>& sch, long long u0, long long u1, const CUtensorMap* map_k,
                                     const CUtensorMap* map_v, unsigned char* ring, uint64_t* full_bar, uint64_t* empty_bar,
                                     volatile int* s_err) {
  static_assert(sizeof(DT) == 2 || P::kUnit <= 16, "a unit's float32 rows are one copy: they lie in one page");
  constexpr int UNIT = P::kUnit, kSlots = P::kSlots, kHalf = UNIT * kD * static_cast<int>(sizeof(DT));
  const TreeArgs& a = da.a;
  const int lane = threadIdx.x & 31;
  const int box = min(UNIT, 1 << a.page_shift);  // rows a copy
  int count = 0, seq = -1, first = 0, page = 0;  // lane x holds the page of entry first + x
  bool stop = false;
  uint32_t left_out = 0;  // slots that the test hook never fills
  for (long long u = u0; u < u1 && !stop;) {
    const Task k = task_of<P>(a, sch, u, u1);
    for (int i = k.first; i < k.last; ++i, ++count) {
      const int slot = count % kSlots;
      const int rows = min(UNIT, k.len - i * UNIT), boxes = (rows + box - 1) / box;  // none of an empty cache
      const int entry = (i * UNIT) >> a.page_shift;
      if (boxes > 0 && (seq != k.b || entry < first || entry + boxes > first + 32)) {
        seq = k.b;
        first = entry;
        page = entry + lane < a.max_pages ? __ldg(a.table + static_cast<size_t>(k.b) * a.max_pages + entry + lane) : 0;
      }
      // lane x copies box x: its row in the pools
      int y = 0;
      const int id = __shfl_sync(0xffffffffu, page, (entry - first + lane) & 31);
      if (lane < boxes) {
        const bool ok = id >= 0 && id < a.n_pages;
        if (!ok) atomicExch(a.status, kStatusDeviceAssert);
        y = (((ok ? id : 0) * a.H + k.h) << a.page_shift) + ((i * UNIT) & ((1 << a.page_shift) - 1));
      }
      if (!warp_wait(&empty_bar[slot], ((count / kSlots) & 1) ^ 1, da.wait_ns, s_err)) {
        *s_err = 1;
        stop = true;
        break;
      }
      if (da.skip_copy && i == 0) {
        left_out |= 1u << slot;
        continue;
      }
      if (lane == 0) mbar_arrive_tx(&full_bar[slot], boxes * box * 2 * kD * static_cast<int>(sizeof(DT)));
      __syncwarp();
      if (lane < boxes) {
        const uint32_t at = smem_addr(ring + slot * 2 * kHalf) + lane * box * 128;
        if constexpr (sizeof(DT) == 4) {
          tma_3d(at, map_k, 0, y, 0, &full_bar[slot]);
          tma_3d(at + kHalf, map_v, 0, y, 0, &full_bar[slot]);
        } else {
          tma_2d(at, map_k, 0, y, &full_bar[slot]);
          tma_2d(at + kHalf, map_v, 0, y, &full_bar[slot]);
        }
      }
    }
    u = k.start + k.units + P::kTaskCost;
  }
  // nothing may be in flight when the block ends
  if (lane == 0) {
    for (int c = count - kSlots < 0 ? 0 : count - kSlots; c < count; ++c)
      if (!(left_out >> (c % kSlots) & 1)) mbar_wait(&full_bar[c % kSlots], (c / kSlots) & 1, kDrainNs);
    if (*s_err) atomicExch(a.status, kStatusTimeout);
  }
}

// ------------------------------------------------------------------------------ a run's pieces --
// Row r of a task (query head, node): its row of q and o, and the node.
__device__ __forceinline__ size_t row_of(const TreeArgs& a, const Task& k, int r, int* s) {
  const int head = r / k.n;
  *s = r - head * k.n;
  return (static_cast<size_t>(k.b) * a.Hq + k.h * a.G + head) * a.T + *s;
}
// Position of a node; one that N does not hold is reported and clamped, so that the tables are read in bounds.
__device__ __forceinline__ int position_of(const TreeArgs& a, const Task& k, int depth, bool* ok) {
  if (k.len + depth < a.N) return k.len + depth;
  *ok = false;
  return a.N - 1;
}

// The task's drafted keys, rotated, and their values into `draft` ([n][64] each, float); by the CONS computing
// threads.
template <typename DT, int CONS>
__device__ __forceinline__ void stage_drafts(const TreeArgs& a, const Task& k, const WarpTree& tree, float* draft, bool* ok) {
  const int tid = threadIdx.x, t = tid & 3;
  const size_t fresh = (static_cast<size_t>(k.b) * a.H + k.h) * a.T * kD;
  const DT* kn = static_cast<const DT*>(a.kn) + fresh;
  const DT* vn = static_cast<const DT*>(a.vn) + fresh;
  for (int x = 0; x < (k.n + CONS / 4 - 1) / (CONS / 4); ++x) {
    const int s = x * (CONS / 4) + (tid >> 2);
    const int depth = pick32(tree.depth, s & 63);
    if (s < k.n) {
      float y[16], v[16];
      float2 e[8];
      load_part(kn + static_cast<size_t>(s) * kD, t, y);
      load_part(vn + static_cast<size_t>(s) * kD, t, v);
      rope_row(a.rope_lo, a.rope_hi, position_of(a, k, depth, ok), t, e);
      rotate_part(y, e, false);
      store_part(draft + s * kD, t, y);
      store_part(draft + (k.n + s) * kD, t, v);
    }
  }
}

__device__ __forceinline__ void read_part(const float* row, int t, float (&x)[16]) {
  const float4* r = reinterpret_cast<const float4*>(row);
  *reinterpret_cast<float4*>(x) = r[2 * t];
  *reinterpret_cast<float4*>(x + 4) = r[2 * t + 1];
  *reinterpret_cast<float4*>(x + 8) = r[8 + 2 * t];
  *reinterpret_cast<float4*>(x + 12) = r[8 + 2 * t + 1];
}

// The part of the drafted keys in each row: O (not divided) into acc, maximum and sum into mx and sm.  A quad a
// row, over the row's ancestors alone.  query(r, t, y): the rotated query of row r times log2(e)/8, dims D_t.
template <int CONS, typename Q>
__device__ __forceinline__ void attend_drafts(const TreeArgs& a, const Task& k, const WarpTree& tree, const float* draft, int r0, int rows,
                                              float* acc, float* mx, float* sm, Q&& query) {
  const int tid = threadIdx.x, t = tid & 3;
  for (int x = 0; x < (rows + CONS / 4 - 1) / (CONS / 4); ++x) {
    const int r = x * (CONS / 4) + (tid >> 2);
    const bool in = r < rows;
    const int s = in ? (r0 + r) % k.n : 0;
    uint64_t set = pick64(tree.above, s);
    if (!in) set = 0;
    float y[16], o[16], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) y[w] = o[w] = 0.f;
    if (in) query(r, t, y);
    while (__any_sync(0xffffffffu, set != 0)) {
      const bool on = set != 0;
      float sc = 0.f, v[16];
      if (on) {
        const int key = __ffsll(static_cast<long long>(set)) - 1;
        set &= set - 1;
        float kx[16];
        read_part(draft + key * kD, t, kx);
        read_part(draft + (k.n + key) * kD, t, v);
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
      store_part(acc + r * kAccStride, t, o);
      if (t == 0) {
        mx[r] = m;
        sm[r] = l;
      }
    }
  }
}

// The rows of a piece, O in acc (and the rest of it in `more`, where that is given) for the common maximum of `parts` (maximum, sum) pairs a row: divided, to o
// and lse, where the piece is a whole task; as a partial else.
template <typename DT, int ROWS, int CONS>
__device__ __forceinline__ void write_rows(const DenseTreeArgs& da, const Task& k, bool whole, int slot, int r0, int rows,
                                           const float* acc, const float* more, const float* mx, const float* sm, int parts) {
  const TreeArgs& a = da.a;
  float* part = da.part + (static_cast<size_t>(blockIdx.x) * 2 + slot) * ROWS * kDtPart;
  for (int i = threadIdx.x; i < rows * 16; i += CONS) {  // 16 threads a row
    const int r = i >> 4, d = (i & 15) * 4;
    float mr = -INFINITY, sum = 0.f;
    for (int x = 0; x < parts; ++x) mr = fmaxf(mr, mx[x * ROWS + r]);
    for (int x = 0; x < parts; ++x) sum += sm[x * ROWS + r] * weight_of(mx[x * ROWS + r], sm[x * ROWS + r], mr);
    float4 x = *reinterpret_cast<const float4*>(acc + r * kAccStride + d);
    if (more != nullptr) {
      const float4 y = *reinterpret_cast<const float4*>(more + r * kAccStride + d);
      x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
    }
    if (whole) {
      int s;
      const size_t row = row_of(a, k, r0 + r, &s);
      const float inv = 1.f / sum;
      if constexpr (sizeof(DT) == 4) {
        *reinterpret_cast<float4*>(static_cast<float*>(a.o) + row * kD + d) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
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

// ------------------------------------------------------------------------------ join --
// Notes task k where other blocks hold units of it too (one thread, for each piece).
template <typename P>
__device__ __forceinline__ void note_split(const DenseTreeArgs& da, const Task& k, long long cost, int sharing) {
  if (k.first == 0 && k.last == k.units) return;
  const long long begin = k.start + P::kTaskCost;
  const int first = block_at(cost, sharing, begin), last = block_at(cost, sharing, begin + k.units - 1);
  da.split[2 * blockIdx.x + (k.first == 0 ? 1 : 0)] =
      Split{last - first + 1, first, k.start >= cut(cost, sharing, first) ? 1 : 0, k.b, k.h, k.rb, k.n, 0};
}
__device__ __forceinline__ void clear_splits(const DenseTreeArgs& da) { da.split[2 * blockIdx.x].parts = da.split[2 * blockIdx.x + 1].parts = 0; }

// Adds the partials of the tasks whose units several blocks hold.  As many blocks as hold a task share its rows here, so
// that the work is spread however few the tasks are.  16 threads read a row of a partial.  Up to 16 partials: such a team
// a row, the weights in its lanes.  More: a row at a time, its weights in shared memory, 16 teams that take
// every 16th partial and meet in order.  One sequence and head, 60000 rows: a call of
// one query 15 us, 8 queries 18; 39 and 48 where a block in order joined four rows of a task.
constexpr int kJoinThreads = 256;
constexpr int kJoinTeams = kJoinThreads / 16;
constexpr int kMostBlocks = 512;  // of a grid

__device__ __forceinline__ void add_row(float4& o, const float* p, float f) {
  const float2 x = *reinterpret_cast<const float2*>(p), y = *reinterpret_cast<const float2*>(p + 2);
  o.x += x.x * f;
  o.y += x.y * f;
  o.z += y.x * f;
  o.w += y.y * f;
}

template <typename DT, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ DenseTreeArgs da) {
  __shared__ float s_w[kMostBlocks], s_red[2][kJoinThreads / 32];
  __shared__ float4 s_o[kJoinTeams][16];
  const TreeArgs& a = da.a;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int tid = threadIdx.x, team = tid >> 4, lane = tid & 15, d = 4 * lane;
  const Split sp = da.split[2 * blockIdx.x + blockIdx.y];
  if (sp.parts == 0) return;
  const int q0 = sp.rb * ROWS, rows = min(ROWS, a.G * sp.n - q0), each = (rows + sp.parts - 1) / sp.parts;
  const int begin = (static_cast<int>(blockIdx.x) - sp.first) * each, end = min(rows, begin + each);
  const float* one = da.part + (static_cast<size_t>(sp.first) * 2 + sp.slot) * ROWS * kDtPart;
  const float* more = da.part + static_cast<size_t>(sp.first) * 2 * ROWS * kDtPart;
  auto partial = [&](int i, int r) { return (i == 0 ? one : more + static_cast<size_t>(i) * (2 * ROWS * kDtPart)) + r * kDtPart; };
  auto write = [&](int r, float4 o, float all, float sum) {
    const float inv = 1.f / sum;
    o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    const int head = (q0 + r) / sp.n, s = (q0 + r) - head * sp.n;
    const size_t row = (static_cast<size_t>(sp.b) * a.Hq + sp.h * a.G + head) * a.T + s;
    if constexpr (sizeof(DT) == 4)
      *reinterpret_cast<float4*>(static_cast<float*>(a.o) + row * kD + d) = o;
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + row * kD + d) = make_uint2(pack_bf2(o.x, o.y), pack_bf2(o.z, o.w));
    if (d == 0 && a.lse != nullptr) a.lse[row] = (all + log2f(sum)) * kLn2;
  };
  if (sp.parts <= 16) {
    for (int r0 = begin; r0 < end; r0 += kJoinTeams) {  // (the same trips in every warp: its two teams meet in the shuffles)
      const int r = r0 + team;
      const bool in = r < end;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (in && lane < sp.parts) ml = *reinterpret_cast<const float2*>(partial(lane, r) + kD);
      float all = ml.x;
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, x));
      const float w = weight_of(ml.x, ml.y, all);
      float sum = ml.y * w;
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int i = 0; i < sp.parts; ++i) {
        const float f = __shfl_sync(0xffffffffu, w, i, 16);
        if (in) add_row(o, partial(i, r) + d, f);
      }
      if (in) write(r, o, all, sum);
    }
    return;
  }
  for (int r = begin; r < end; ++r) {
    float2 ml[kMostBlocks / kJoinThreads];
    float all = -INFINITY, sum = 0.f;
#pragma unroll
    for (int u = 0; u < kMostBlocks / kJoinThreads; ++u) {
      const int i = tid + u * kJoinThreads;
      ml[u] = i < sp.parts ? *reinterpret_cast<const float2*>(partial(i, r) + kD) : make_float2(-INFINITY, 0.f);
      all = fmaxf(all, ml[u].x);
    }
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, x));
    if ((tid & 31) == 0) s_red[0][tid >> 5] = all;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kJoinThreads / 32; ++x) all = fmaxf(all, s_red[0][x]);
#pragma unroll
    for (int u = 0; u < kMostBlocks / kJoinThreads; ++u) {
      const float w = weight_of(ml[u].x, ml[u].y, all);
      s_w[tid + u * kJoinThreads] = w;
      sum += ml[u].y * w;
    }
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    if ((tid & 31) == 0) s_red[1][tid >> 5] = sum;
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = team; i < sp.parts; i += kJoinTeams) add_row(o, partial(i, r) + d, s_w[i]);
    s_o[team][lane] = o;
    __syncthreads();
    if (team == 0) {
      sum = s_red[1][0];
#pragma unroll
      for (int x = 1; x < kJoinThreads / 32; ++x) sum += s_red[1][x];
#pragma unroll
      for (int x = 1; x < kJoinTeams; ++x) {
        const float4 y = s_o[x][lane];
        o = make_float4(o.x + y.x, o.y + y.y, o.z + y.z, o.w + y.w);
      }
      write(r, o, all, sum);
    }
    __syncthreads();  // the shared memory is the next row's
  }
}

template <typename DT, typename P>
cudaError_t launch_join(const DenseTreeArgs& da, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(da.blocks), 2);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<DT, P::kRows>, da);
}

// The most dynamic shared memory that a kernel's launches ask for.  The same for every call: the limit is the kernel's, not a
// launch's, and host threads set it and launch at the same time.
template <typename Kernel>
cudaError_t allow_shared(Kernel kernel, size_t most) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
}

// ------------------------------------------------------------------------------ copies --
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A layer's pool as rows of 64 values (float32: as two halves of 32); a copy takes `box` rows, 128 bytes at a time.
inline cudaError_t map_of(CUtensorMap* m, const void* pool, long long rows, int es, int box) {
  static const EncodeTiled encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<EncodeTiled>(fn);
  }();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t n = static_cast<cuuint64_t>(rows), row_bytes = static_cast<cuuint64_t>(kD) * es;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(128 / es), n, row_bytes / 128}, strides[2] = {row_bytes, 128};
  const cuuint32_t boxes[3] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(box), static_cast<cuuint32_t>(row_bytes / 128)};
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUresult r = encode(m, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, es == 2 ? 2 : 3,
                            const_cast<void*>(pool), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Both pools' maps for units of `unit` rows.  After a call of the runtime that needs the device's context: encode is the driver's, and
// a host thread has no context of its own accord until then.
inline cudaError_t maps_of(const TreeArgs& a, int es, int unit, CUtensorMap* mk, CUtensorMap* mv) {
  const int box = (1 << a.page_shift) < unit ? 1 << a.page_shift : unit;
  const long long rows = (static_cast<long long>(a.n_pages) * a.H) << a.page_shift;
  const cudaError_t e = map_of(mk, a.kc, rows, es, box);
  return e == cudaSuccess ? map_of(mv, a.vc, rows, es, box) : e;
}


// tree_dense_tc.cu: bf16, more than 8 query rows a key head
size_t dense_tree_tc_bytes(int rows);
cudaError_t launch_dense_tree_tc(const DenseTreeArgs& da, cudaStream_t stream);

}  // namespace fibattn
