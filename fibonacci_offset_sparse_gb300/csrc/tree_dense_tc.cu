// Dense decode of a tree of drafted tokens, bf16 with more than 8 query rows a key head (sm_103a): the
// work, its cut and its join as in tree_dense.cu, the products on the 5th-generation tensor cores.
//
// What bounds it: the read of the cache, as there.  With mma.sync the products alone took as long as the
// read from some 24 query rows on; here the tensor pipes are busy for a fifth of the time.  16 sequences of 4096, 8192 .. 65536
// rows, 8 heads (1.14 GB): 16 query rows 177 us (6.4 TB/s, 95% of a measured copy), 24 and 32 rows 182; 48 rows 225 and 64 rows
// 263, where one block an SM is bound by the steps of its softmax warps.  Every 64 rows read the cache once: 128 take 506, 256 997.
//
// Per unit of 128 cached rows, with the keys as the 128 rows of the accumulator:
//   S^T [128 keys x ROWS] = K Q'^T    K from the ring as TMA left it (K-major, 128-byte swizzle), the rotated
//                                     query split in three bf16 (24 bits), all added up
//   P = 2^(S - m)                     a thread a key: its row of S^T from tensor memory to registers, its
//                                     weights, again hi + lo, to shared memory (16 bytes for 8 query rows)
//   O^T [64 dims x ROWS] += V^T P^T   V from the ring (its transpose by the descriptor), P as written; O stays
//                                     in tensor memory for 16 units, then the softmax warps add it to the run's sum there
// The maximum m of a row is common to a unit's keys and moves only when a score passes it by more than
// 8 (weights <= 256 until then): one vote of four warps a unit; the exact maximum, and O rescaled, are the
// exception's work.
//
// Block: softmax warps (warp w reads lanes 32 (w % 4) .. of tensor memory; four warps share 16 query
// rows), the feeder, and a warp whose one thread issues the products as their operands arrive: S of the next
// unit runs while a unit's weights are formed.
#include <algorithm>
#include <cfloat>

#include "tree_dense.cuh"

namespace fibattn {

namespace {

// Units whose products the tensor pipes add to one another.  They round toward zero at each product (16 a unit), 3.6e-8 of the sum in
// the mean and all to one side: over 131072 rows 5.6e-4 of O were lost where a run was one chain, a tenth of a step of bf16,
// and 1e-5 are at 16 units.
constexpr int kChain = 16;
constexpr float kNoKey = FLT_MAX;  // a row's reference, negated, before it has met a finite score: below every score

// Barriers and what the warps tell one another.
struct TcFixed {
  uint64_t full[10], empty[10];  // slots of the ring
  uint64_t scores[2];            // S of a unit is in its buffer (units alternate)
  uint64_t weights;              // P of a unit is in shared memory
  uint64_t added;                // ... and in O
  uint64_t query;                // Q' of a piece is in shared memory
  uint64_t drained;
  long long run[2], place;       // the block's run; where in it the softmax warps are
  uint32_t tmem;
  int err;
};

template <int ROWS, bool PACKED>
struct TcShape {
  // Task cost: 256 tasks of 64 rows over 4096 cached ones take 99 us at 12, 96 at 8 and 100 at 16; the 16 sequences above with 24
  // query rows 181, 180 and 183.  Units a block: one sequence and head of 30000 rows takes 15.8 us at 3, 17.4 at 1 and 17.0 at 6; 8
  // heads of 4096 17.1, 16.2 and 18.0.
  static constexpr int kUnit = 128, kRows = ROWS, kTaskCost = 12, kLeast = 3;
  static constexpr int kSlotBytes = kUnit * kD * 2;  // K or V of a unit
  static constexpr int kGroupRows = 16, kGroups = ROWS / kGroupRows;  // query rows of four softmax warps
  static constexpr int kCons = 128 * kGroups, kThreads = kCons + 64;
  // Two blocks an SM where the rest beside their rings is small: when the 16 sequences took 172 us with 16 query rows, one block
  // of 9 slots took 179; with 32 rows 178 and 185; 32 sequences of up to 2048, 16 rows, 27 and 35.  What is on its way from memory
  // is what the ring holds, so it takes what shared memory is left: K's slot is free once the scores are formed.
  static constexpr int kResident = ROWS <= 32 ? 2 : 1;
  static constexpr int kSlots = ROWS <= 32 ? 5 : 9;
  static constexpr int kColumns = ROWS == 16 ? 64 : ROWS == 32 ? 128 : 256;  // of tensor memory: S twice, O, the sum of earlier O
  static_assert(4 * ROWS <= kColumns, "columns");
  // byte offsets in dynamic shared memory (its base is 1024-byte aligned)
  static constexpr int kQuery = kSlots * kSlotBytes;    // hi [ROWS][64], mid, lo: K-major, 128-byte swizzle
  static constexpr int kWeights = kQuery + ROWS * 384;  // hi [ROWS/8][16][8 keys][8 rows], lo; see below for its other uses
  static constexpr int kRef = kWeights + ROWS * 512;    // [ROWS] the rows' references, negated
  static constexpr int kMax = kRef + ROWS * 4;          // [2][ROWS]: of the cached keys, of the drafted ones
  static constexpr int kSum = kMax + 2 * ROWS * 4;
  static constexpr int kWarpMax = kSum + 2 * ROWS * 4;  // [4][ROWS]; at the end the two parts' weights [2][ROWS]
  // Where two blocks share an SM the barriers are dynamic memory too: static memory is padded to the dynamic base's 1024 bytes.
  static constexpr int kFixed = kWarpMax + 4 * ROWS * 4;
  static constexpr int kSchedule = kFixed + (kResident == 2 ? sizeof(TcFixed) : 0);
  static constexpr bool kPacked = PACKED;
  static size_t bytes(int B) { return kSchedule + Schedule<PACKED>::bytes(B); }
};

// ------------------------------------------------------------------- tensor memory and products --
__device__ __forceinline__ void tmem_alloc(uint32_t* out, int columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_addr(out)), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
}
__device__ __forceinline__ void tmem_free(uint32_t at, int columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(at), "r"(columns));
}
// Shared-memory matrix descriptor: start, leading and stride byte offsets; swizzle 2 = 128 bytes, 0 = none.
__device__ __forceinline__ uint64_t matrix_at(uint32_t start, uint32_t lead, uint32_t stride, uint32_t swizzle) {
  return static_cast<uint64_t>((start & 0x3ffffu) >> 4) | static_cast<uint64_t>(lead >> 4) << 16 |
         static_cast<uint64_t>(stride >> 4) << 32 | 1ull << 46 | static_cast<uint64_t>(swizzle) << 61;
}
// bf16 x bf16 -> float32, M x N; a_mn, b_mn: the operand's rows lie along memory (not its k index).
constexpr uint32_t product_of(int M, int N, bool a_mn, bool b_mn) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | static_cast<uint32_t>(N >> 3) << 17 |
         static_cast<uint32_t>(M >> 4) << 24;
}
__device__ __forceinline__ void mma_tc(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b),
      "r"(desc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
// Arrives at the barrier when every product issued so far is done.
__device__ __forceinline__ void commit_tc(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(smem_addr(bar)) : "memory");
}
// One lane of the warp, which the compiler can tell is one: the products' operands then need no loop over lanes.
__device__ __forceinline__ bool one_lane() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_smem() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

// N columns (8 or 16) of a warp's 32 lanes.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t at, float (&x)[N]) {
  static_assert(N == 8 || N == 16, "shapes used here");
  uint32_t r[N];
  if constexpr (N == 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
  else
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at)
                 : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = __uint_as_float(r[i]);
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t at, const float (&x)[N]) {
  uint32_t r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = __float_as_uint(x[i]);
  if constexpr (N == 16)
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};\n" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
        : "memory");
  else
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};\n" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(at)
                 : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p)); }

// Whether any of a group's 128 softmax threads says so; they are synchronised by it.
__device__ __forceinline__ bool any_of_group(int group, bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(2 + group)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int group) { asm volatile("barrier.cta.sync %0, 128;\n" ::"r"(2 + group) : "memory"); }
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(y) : "f"(x));
  return y;
}

// x0 += y0, x1 += y1
__device__ __forceinline__ void add2(float& x0, float& x1, float y0, float y1) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(x0), "+f"(x1)
      : "f"(y0), "f"(y1));
}
// The largest of three; NaN where one is.
__device__ __forceinline__ float max_nan(float x, float y, float z) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// The units' K and V tiles in turn: the tile 2 count (K) or 2 count + 1 (V), its slot and its round's parity.
template <int SLOTS>
struct Tile {
  int slot;
  uint32_t parity;
  __device__ __forceinline__ explicit Tile(int n) : slot(n % SLOTS), parity((n / SLOTS) & 1) {}
};

// Their feeder: K, then V of each unit of [u0, u1), a page at a time.
template <typename P>
__device__ __forceinline__ void feed_tiles(const DenseTreeArgs& da, const Schedule<P::kPacked>& sch, long long u0, long long u1, const CUtensorMap* map_k,
                                           const CUtensorMap* map_v, unsigned char* ring, uint64_t* full_bar, uint64_t* empty_bar,
                                           volatile int* s_err) {
  const TreeArgs& a = da.a;
  const int lane = threadIdx.x & 31;
  const int box = min(P::kUnit, 1 << a.page_shift);  // rows a copy
  int n = 0, seq = -1, first = 0, page = 0;          // lane x holds the page of entry first + x
  bool stop = false;
  uint32_t left_out = 0;  // slots that the test hook never fills
  for (long long u = u0; u < u1 && !stop;) {
    const Task k = task_of<P>(a, sch, u, u1);
    for (int i = k.first; i < k.last && !stop; ++i) {
      const int rows = min(P::kUnit, k.len - i * P::kUnit), boxes = (rows + box - 1) / box;  // none of an empty cache
      const int entry = (i * P::kUnit) >> a.page_shift;
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
        y = (((ok ? id : 0) * a.H + k.h) << a.page_shift) + ((i * P::kUnit) & ((1 << a.page_shift) - 1));
      }
#pragma unroll
      for (int v = 0; v < 2; ++v, ++n) {
        const Tile<P::kSlots> tile(n);
        if (!warp_wait(&empty_bar[tile.slot], tile.parity ^ 1, da.wait_ns, s_err)) {
          *s_err = 1;
          stop = true;
          break;
        }
        if (da.skip_copy && i == 0 && v == 0) {
          left_out |= 1u << tile.slot;
          continue;
        }
        if (lane == 0) mbar_arrive_tx(&full_bar[tile.slot], boxes * box * kD * 2);
        __syncwarp();
        if (lane < boxes)
          tma_2d(smem_addr(ring + tile.slot * P::kSlotBytes) + lane * box * 128, v ? map_v : map_k, 0, y, &full_bar[tile.slot]);
      }
    }
    u = k.start + k.units + P::kTaskCost;
  }
  // nothing may be in flight when the block ends
  for (int c = n - P::kSlots < 0 ? 0 : n - P::kSlots; c < n; ++c) {
    const Tile<P::kSlots> tile(c);
    if (!(left_out >> tile.slot & 1)) mbar_wait(&full_bar[tile.slot], tile.parity, kDrainNs);
  }
  __syncwarp();
  if (*s_err && lane == 0) atomicExch(a.status, kStatusTimeout);
}

template <typename P>
__device__ __forceinline__ TcFixed* fixed_at(unsigned char* smem) {
  if constexpr (P::kResident == 2) {
    return reinterpret_cast<TcFixed*>(smem + P::kFixed);
  } else {
    __shared__ __align__(8) TcFixed fixed;
    return &fixed;
  }
}

template <int ROWS, bool PACKED>
__global__ void __launch_bounds__(TcShape<ROWS, PACKED>::kThreads, TcShape<ROWS, PACKED>::kResident)
    dense_tree_tc_kernel(const __grid_constant__ DenseTreeArgs da, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v) {
  using P = TcShape<ROWS, PACKED>;
  constexpr int CONS = P::kCons, GR = P::kGroupRows, kFeeder = CONS / 32, kIssuer = kFeeder + 1;
  extern __shared__ __align__(1024) unsigned char smem[];
  TcFixed& bars = *fixed_at<P>(smem);
  volatile int& s_err = bars.err;
  volatile long long(&s_run)[2] = bars.run;
  volatile long long& s_place = bars.place;
  const TreeArgs& a = da.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (tid == 0) {
    s_err = 0;
    for (int s = 0; s < P::kSlots; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    mbar_init(&bars.scores[0], 1);
    mbar_init(&bars.scores[1], 1);
    mbar_init(&bars.weights, 4 * P::kGroups);
    mbar_init(&bars.added, 1);
    mbar_init(&bars.query, 4 * P::kGroups);
    mbar_init(&bars.drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  // The queries and drafted rows, read once a task behind a full queue of copies: into L2 before it fills.
  {
    const long long q_lines = static_cast<long long>(a.B) * a.Hq * a.T, n_lines = static_cast<long long>(a.B) * a.H * a.T;
    const long long at = static_cast<long long>(blockIdx.x) * P::kThreads + tid, step = static_cast<long long>(gridDim.x) * P::kThreads;
    for (long long x = at; x < q_lines; x += step) prefetch_l2(static_cast<const __nv_bfloat16*>(a.q) + x * kD);
    for (long long x = at; x < n_lines; x += step) {
      prefetch_l2(static_cast<const __nv_bfloat16*>(a.kn) + x * kD);
      prefetch_l2(static_cast<const __nv_bfloat16*>(a.vn) + x * kD);
    }
  }
  const Schedule<PACKED> sch(smem + P::kSchedule, a.B);
  build_schedule<P>(a, sch);
  if (tid == 0) clear_splits(da);
  const long long cost = sch.end(a.B);
  const int sharing = sharing_blocks(cost, da.blocks, P::kLeast);
  if (static_cast<int>(blockIdx.x) >= sharing) return;
  const long long u0 = cut(cost, sharing, blockIdx.x), u1 = cut(cost, sharing, blockIdx.x + 1);
  if (tid == 0) {
    s_run[0] = u0;
    s_run[1] = u1;
  }
  if (warp == kIssuer) tmem_alloc(&bars.tmem, P::kColumns);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = bars.tmem, tmem_o = tmem + 2 * ROWS, tmem_sum = tmem + 3 * ROWS;
  const uint32_t base = smem_addr(smem);

  if (warp == kFeeder) {
    // =================================================================== feeder
    feed_tiles<P>(da, sch, u0, u1, &map_k, &map_v, smem, bars.full, bars.empty, &s_err);
  } else if (warp == kIssuer) {
    // =================================================================== products
    if (one_lane()) {
      constexpr uint32_t kScores = product_of(128, ROWS, false, false), kValues = product_of(64, ROWS, true, true);
      // two cursors over the units of the run: the next S, the next O += V P
      struct Cursor {
        long long u;
        int i, begin, last, count;
        bool first;  // of its piece
      } s{u0, 0, 0, 0, 0, false}, o{u0, 0, 0, 0, 0, false};
      auto next = [&](Cursor& c) {  // moves to a unit; false at the run's end
        while (c.i == c.last) {
          if (c.u >= u1) return false;
          const Task k = task_of<P>(a, sch, c.u, u1);
          c.u = k.start + k.units + P::kTaskCost;
          c.i = c.begin = k.first;
          c.last = k.last;
          c.first = true;
        }
        return true;
      };
      int pieces = 0;
      bool more_s = next(s), more_o = next(o);
      unsigned long long since = global_ns();
      while (more_o && !s_err) {
        bool did = false;
        // S of a unit: its keys and its piece's query are there, and its buffer's last user is past it
        const Tile<P::kSlots> kt(2 * s.count), vt(2 * o.count + 1);
        if (more_s && s.count - o.count < 2 && mbar_try(&bars.full[kt.slot], kt.parity) && (!s.first || mbar_try(&bars.query, pieces & 1))) {
          if (s.first) ++pieces;
          fence_after();
          const uint32_t from = base + kt.slot * P::kSlotBytes, d = tmem + (s.count & 1) * ROWS;
#pragma unroll
          for (int part = 2; part >= 0; --part)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              mma_tc(d, matrix_at(from + 32 * x, 16, 1024, 2), matrix_at(base + P::kQuery + part * ROWS * 128 + 32 * x, 16, 1024, 2), kScores,
                     part < 2 || x > 0);
          commit_tc(&bars.empty[kt.slot]);
          commit_tc(&bars.scores[s.count & 1]);
          ++s.count;
          ++s.i;
          s.first = false;
          more_s = next(s);
          did = true;
        }
        if (o.count < s.count && mbar_try(&bars.weights, o.count & 1) && mbar_try(&bars.full[vt.slot], vt.parity)) {
          fence_after();
          const uint32_t from = base + vt.slot * P::kSlotBytes;
          const bool add = (o.i - o.begin) % kChain != 0;
#pragma unroll
          for (int part = 1; part >= 0; --part)
#pragma unroll
            for (int x = 0; x < 8; ++x)
              mma_tc(tmem_o, matrix_at(from + 2048 * x, 16, 1024, 2), matrix_at(base + P::kWeights + part * ROWS * 256 + 256 * x, 128, 2048, 0),
                     kValues, add || part == 0 || x > 0);
          commit_tc(&bars.empty[vt.slot]);
          commit_tc(&bars.added);
          ++o.count;
          ++o.i;
          o.first = false;
          more_o = next(o);
          did = true;
        }
        if (did) {
          since = global_ns();
        } else if (global_ns() - since > da.wait_ns) {
          s_err = 1;
          atomicExch(a.status, kStatusTimeout);
        }
      }
      commit_tc(&bars.drained);  // nothing may be in flight when the block ends
      mbar_wait(&bars.drained, 0, kDrainNs);
    }
    __syncwarp();
  } else {
    // =================================================================== softmax
    float* s_ref = reinterpret_cast<float*>(smem + P::kRef);
    float* s_max = reinterpret_cast<float*>(smem + P::kMax);
    float* s_sum = reinterpret_cast<float*>(smem + P::kSum);
    float* s_warp = reinterpret_cast<float*>(smem + P::kWarpMax);
    float* s_draft = reinterpret_cast<float*>(smem + P::kWeights);  // before a piece's weights
    float* s_part = reinterpret_cast<float*>(smem + P::kWeights);   // after them: [ROWS][128] sums, then O
    const int group = warp >> 2, g0 = group * GR, key = tid & 127, wq = warp & 3;  // the thread's query rows and key
    const uint32_t lanes = static_cast<uint32_t>(wq) << 21;                        // its warp's lanes of tensor memory
    int count = 0;
    // After a wait that gave up, nothing is waited for any more; what follows works on whatever lies there, in bounds, and is
    // not written.  A warp waits as a whole (its tensor memory instructions are warp-wide), but for a lone thread's wait.
    auto wait_alone = [&](uint64_t* bar, uint32_t parity) {
      if (s_err || mbar_wait(bar, parity, da.wait_ns)) return;
      s_err = 1;
      atomicExch(a.status, kStatusTimeout);
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      wait_alone(bar, parity);
      __syncwarp();
    };
    // Of a piece, formed anew from shared memory where they are needed: held over the units' loop they would cost it
    // spills, and what shared memory leaves of L1 does not hold those (64 query rows over the 16 sequences: 297 us with them, 264
    // without, at the time).
    auto task_here = [&] { return task_of<P>(a, sch, s_place, s_run[1]); };
    auto drafts_here = [&] {  // the drafted keys' O
      uint32_t block;
      asm volatile("mov.u32 %0, %%ctaid.x;\n" : "=r"(block));
      return da.part + static_cast<size_t>(da.blocks) * 2 * ROWS * kDtPart + static_cast<size_t>(block) * ROWS * kAccStride;
    };
    for (long long u = s_run[0]; u < s_run[1];) {
      const Task k = task_of<P>(a, sch, u, s_run[1]);
      if (k.first == k.last) {
        u = k.start + k.units + P::kTaskCost;
        continue;
      }
      if (tid == 0) s_place = u;
      if (tid == 0) {
        const long long all = sch.end(a.B);
        note_split<P>(da, k, all, sharing_blocks(all, da.blocks, P::kLeast));
      }
      const int k_first = k.first, k_last = k.last, k_len = k.len;
      const int mine = min(GR, max(0, a.G * k.n - k.rb * ROWS - g0));  // rows of this group
      {
      const bool tail = k.last == k.units;
      const int r0 = k.rb * ROWS, rows = min(ROWS, a.G * k.n - r0);
      bool ok = true;
      const WarpTree tree = warp_tree(a, k.b, k.n, &ok);
      // the rotated query: a quad a row, 16 bytes of each part for 8 dims
      for (int r = tid >> 2; r < ROWS; r += CONS / 4) {
        const int t = lane & 3;
        int s = 0;
        const size_t row = r < rows ? row_of(a, k, r0 + r, &s) : 0;
        const int depth = pick32(tree.depth, s);
        uint32_t hi[8], mid[8], lo[8];
        if (r < rows) {
          float x[16];
          float2 e[8];
          load_part(static_cast<const __nv_bfloat16*>(a.q) + row * kD, t, x);
          rope_row(a.rope_lo, a.rope_hi, position_of(a, k, depth, &ok), t, e);
          rotate_part(x, e, false);
#pragma unroll
          for (int w = 0; w < 8; ++w) split_bf16(x[2 * w] * (kLog2e / 8.0f), x[2 * w + 1] * (kLog2e / 8.0f), hi[w], mid[w], lo[w]);
        } else {
#pragma unroll
          for (int w = 0; w < 8; ++w) hi[w] = mid[w] = lo[w] = 0;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          unsigned char* at = smem + P::kQuery + r * 128 + (((t + 4 * h) ^ (r & 7)) << 4);
          *reinterpret_cast<uint4*>(at) = make_uint4(hi[4 * h], hi[4 * h + 1], hi[4 * h + 2], hi[4 * h + 3]);
          *reinterpret_cast<uint4*>(at + ROWS * 128) = make_uint4(mid[4 * h], mid[4 * h + 1], mid[4 * h + 2], mid[4 * h + 3]);
          *reinterpret_cast<uint4*>(at + ROWS * 256) = make_uint4(lo[4 * h], lo[4 * h + 1], lo[4 * h + 2], lo[4 * h + 3]);
        }
      }
      if (tid < ROWS) s_ref[tid] = tid < rows ? kNoKey : 0.f;  // (a row that is none has scores of 0)
      fence_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.query);
      if (tail) stage_drafts<__nv_bfloat16, CONS>(a, k, tree, s_draft, &ok);
      cons_sync<CONS>();
      if (tail) {
        attend_drafts<CONS>(a, k, tree, s_draft, r0, rows, drafts_here(), s_max + ROWS, s_sum + ROWS, [&](int r, int t, float(&y)[16]) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const unsigned char* at = smem + P::kQuery + r * 128 + (((t + 4 * h) ^ (r & 7)) << 4);
#pragma unroll
            for (int w = 0; w < 8; ++w) y[8 * h + w] = 0.f;
#pragma unroll
            for (int part = 2; part >= 0; --part) {
              const uint4 q = *reinterpret_cast<const uint4*>(at + part * ROWS * 128);
              const uint32_t x[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                y[8 * h + 2 * w] += bf_lo(x[w]);
                y[8 * h + 2 * w + 1] += bf_hi(x[w]);
              }
            }
          }
        });
        cons_sync<CONS>();  // the drafted keys' room is the weights' room
      }
      if (!ok) atomicExch(a.status, kStatusDeviceAssert);
      }

      float l[GR];
#pragma unroll
      for (int r = 0; r < GR; ++r) l[r] = 0.f;
      for (int i = k_first; i < k_last; ++i, ++count) {
        const bool all = k_len - i * P::kUnit >= P::kUnit, in = key < k_len - i * P::kUnit;
        wait(&bars.scores[count & 1], (count >> 1) & 1);
        fence_after();
        float x[GR];  // the scores, then over their references
        auto load = [&] {
          tmem_load(tmem + (count & 1) * ROWS + g0 + lanes, x);
          if (!all) {
#pragma unroll
            for (int r = 0; r < GR; ++r) x[r] = in ? x[r] : -INFINITY;
          }
        };
        auto refer = [&] {
#pragma unroll
          for (int c = 0; c < GR / 4; ++c) {
            const float4 ref = *reinterpret_cast<const float4*>(s_ref + g0 + 4 * c);
            add2(x[4 * c], x[4 * c + 1], ref.x, ref.y);
            add2(x[4 * c + 2], x[4 * c + 3], ref.z, ref.w);
          }
        };
        load();
        refer();
        float most = x[0];
#pragma unroll
        for (int r = 1; r + 1 < GR; r += 2) most = max_nan(most, x[r], x[r + 1]);
        if (any_of_group(group, !(max_nan(most, x[GR - 1], x[GR - 1]) <= 8.f))) {  // (a NaN too)
          // A NaN may come of an infinite key, where the parts' sum adds infinities of opposite signs: the upper
          // parts' product alone keeps the sign.
          load();  // (its buffer is not written before this unit's weights are there)
          bool bad = false;
#pragma unroll
          for (int r = 0; r < GR; ++r) bad |= r < mine && isnan(x[r]);
          if (bad) {
            const Task now = task_here();
            const long long at = cache_row(a, now.b, now.h, i * P::kUnit + key);  // (the tile's slot may hold another by now)
#pragma unroll 1
            for (int r = 0; r < mine && at >= 0; ++r) {
              float y = 0.f;
#pragma unroll 1
              for (int d = 0; d < kD; ++d) {
                const __nv_bfloat16 kx = static_cast<const __nv_bfloat16*>(a.kc)[at + d];
                const __nv_bfloat16 qx =
                    *reinterpret_cast<const __nv_bfloat16*>(smem + P::kQuery + (g0 + r) * 128 + (((d >> 3) ^ (r & 7)) << 4) + (d & 7) * 2);
                y = fmaf(__bfloat162float(kx), __bfloat162float(qx), y);
              }
#pragma unroll
              for (int j = 0; j < GR; ++j)
                if (j == r && isnan(x[j])) x[j] = y;
            }
          }
          __syncwarp();
#pragma unroll
          for (int r = 0; r < GR; ++r) {
            const float y = warp_max(x[r]);
            if (lane == 0) s_warp[wq * ROWS + g0 + r] = y;
          }
          if (count > 0) wait(&bars.added, (count - 1) & 1);  // O is at rest
          fence_after();
          group_sync(group);
          // O, then the sum of earlier O.  By the same instructions 24 query rows take 178 us, with a copy for each 189; 64
          // rows, whose registers are shorter, 267 and 259.
#pragma unroll
          for (int c = 0; c < GR / 8; ++c) {
#pragma unroll(ROWS == 64 ? 2 : 1)
            for (int part = 0; part < 2; ++part) {
              if (part == 1 && i <= k_first + kChain) break;
              const uint32_t from = tmem_o + part * ROWS + g0 + 8 * c + lanes;
              float y[8];
              tmem_load(from, y);  // (unused at a piece's first unit)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float* w = s_warp + g0 + 8 * c + e;
                const float m = -s_ref[g0 + 8 * c + e];
                const float corr = ex2(m - fmaxf(m, fmaxf(fmaxf(w[0], w[ROWS]), fmaxf(w[2 * ROWS], w[3 * ROWS]))));
                if (part == 0) l[8 * c + e] *= corr;
                y[e] *= corr;
              }
              if (part == 1 || i > k_first) tmem_store(from, y);
            }
          }
          group_sync(group);
          if (key < GR) {
            const float* w = s_warp + g0 + key;
            s_ref[g0 + key] = -fmaxf(-s_ref[g0 + key], fmaxf(fmaxf(w[0], w[ROWS]), fmaxf(w[2 * ROWS], w[3 * ROWS])));
          }
          group_sync(group);
          refer();
        }
        // the weights of the thread's key, 8 rows to 16 bytes
        uint32_t hi[GR / 2], lo[GR / 2];
#pragma unroll
        for (int c = 0; c < GR / 2; ++c) {
          float p0 = ex2(x[2 * c]), p1 = ex2(x[2 * c + 1]);
          add2(l[2 * c], l[2 * c + 1], p0, p1);
          hi[c] = pack_bf2_rn(p0, p1);
          add2(p0, p1, -bf_lo(hi[c]), -bf_hi(hi[c]));
          lo[c] = pack_bf2_rn(p0, p1);
        }
        if (count > 0) wait(&bars.added, (count - 1) & 1);  // P of the unit before is in O
        if (i > k_first && (i - k_first) % kChain == 0) {   // O to the sum; the next product starts anew
          fence_after();
#pragma unroll
          for (int c = 0; c < GR / 8; ++c) {
            float y[8], z[8];
            tmem_load(tmem_o + g0 + 8 * c + lanes, y);
            if (i > k_first + kChain) {
              tmem_load(tmem_sum + g0 + 8 * c + lanes, z);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] += z[e];
            }
            tmem_store(tmem_sum + g0 + 8 * c + lanes, y);
          }
        }
        unsigned char* at = smem + P::kWeights + (g0 >> 3) * 2048 + (key >> 3) * 128 + (key & 7) * 16;
#pragma unroll
        for (int c = 0; c < GR / 8; ++c) {
          *reinterpret_cast<uint4*>(at + c * 2048) = make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
          *reinterpret_cast<uint4*>(at + ROWS * 256 + c * 2048) = make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
        }
        if (group == 0 && !in) {  // a row that was not filled for this sequence: its weight is 0, and so must be what it holds
          const Tile<P::kSlots> vt(2 * count + 1);
          wait_alone(&bars.full[vt.slot], vt.parity);  // after the copy, which would undo it
          uint4* v = reinterpret_cast<uint4*>(smem + vt.slot * P::kSlotBytes + key * 128);
#pragma unroll
          for (int x = 0; x < 8; ++x) v[x] = make_uint4(0, 0, 0, 0);
        }
        fence_smem();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.weights);
      }
      // ---- the run's O, sums and references; with the drafted keys' part, in a fixed order
      const Task done = task_here();
      const bool tail = done.last == done.units;
      const int r0 = done.rb * ROWS, rows = min(ROWS, a.G * done.n - r0);
      wait(&bars.added, (count - 1) & 1);
      fence_after();
      float o[GR];
      tmem_load(tmem_o + g0 + lanes, o);
      if (k_last > k_first + kChain) {
        float z[GR];
        tmem_load(tmem_sum + g0 + lanes, z);
#pragma unroll
        for (int r = 0; r < GR; ++r) o[r] += z[r];
      }
      cons_sync<CONS>();
#pragma unroll
      for (int r = 0; r < GR; ++r) s_part[(g0 + r) * 128 + key] = l[r];
      cons_sync<CONS>();
      {
        // warp w sums rows w, w + CONS / 32, ...; then lane j has its j-th row's maximum, sum and parts' weights
        constexpr int WARPS = CONS / 32, MOST = (ROWS + WARPS - 1) / WARPS;
        float sum[MOST];
#pragma unroll
        for (int j = 0; j < MOST; ++j) {
          const int r = warp + WARPS * j;
          const float4 x = r < rows ? *reinterpret_cast<const float4*>(s_part + r * 128 + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
          sum[j] = (x.x + x.y) + (x.z + x.w);
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
#pragma unroll
          for (int j = 0; j < MOST; ++j) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], d);
        float mine_sum = 0.f;
#pragma unroll
        for (int j = 0; j < MOST; ++j)
          if (lane == j) mine_sum = sum[j];
        const int r = warp + WARPS * lane;
        if (lane < MOST && r < rows) {
          const float m = s_ref[r] == kNoKey ? -INFINITY : -s_ref[r];
          const float md = tail ? s_max[ROWS + r] : -INFINITY, ld = tail ? s_sum[ROWS + r] : 0.f, all = fmaxf(m, md);
          const float w = weight_of(m, mine_sum, all), wd = weight_of(md, ld, all);
          s_warp[r] = w;
          s_warp[ROWS + r] = wd;
          s_max[r] = all;
          s_sum[r] = mine_sum * w + ld * wd;
        }
      }
      cons_sync<CONS>();
      if (lane < 16) {  // 16 rows of O^T lie in a warp's first 16 lanes
        const int at = g0 * kAccStride + 16 * wq + lane;
        const float* drafts = drafts_here();
        float d[GR];  // (every load before a store, which it might seem to depend on)
#pragma unroll
        for (int r = 0; r < GR; ++r) d[r] = tail && r < mine ? drafts[at + r * kAccStride] : 0.f;
#pragma unroll
        for (int c = 0; c < GR / 4; ++c) {
          const float4 w4 = *reinterpret_cast<const float4*>(s_warp + g0 + 4 * c), d4 = *reinterpret_cast<const float4*>(s_warp + ROWS + g0 + 4 * c);
          const float w[4] = {w4.x, w4.y, w4.z, w4.w}, wd[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[4 * c + e] *= w[e];
            if (tail) o[4 * c + e] = fmaf(d[4 * c + e], wd[e], o[4 * c + e]);
          }
        }
#pragma unroll
        for (int r = 0; r < GR; ++r)
          if (r < mine) s_part[at + r * kAccStride] = o[r];
      }
      fence_before();
      cons_sync<CONS>();
      if (!s_err) write_rows<__nv_bfloat16, ROWS, CONS>(da, done, tail && done.first == 0, done.start >= s_run[0] ? 1 : 0, r0, rows, s_part, nullptr, s_max, s_sum, 1);
      u = done.start + done.units + P::kTaskCost;
      cons_sync<CONS>();  // everything of the piece is free again
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kIssuer) tmem_free(tmem, P::kColumns);
}

template <int ROWS, bool PACKED = false>
cudaError_t launch(const DenseTreeArgs& args, cudaStream_t stream) {
  using P = TcShape<ROWS, PACKED>;
  DenseTreeArgs da = args;
  da.blocks = 152 * P::kResident;  // 152 SMs
  da.split = reinterpret_cast<Split*>(da.part + static_cast<size_t>(da.blocks) * ROWS * (2 * kDtPart + kAccStride));
  const size_t smem = P::bytes(da.a.B);
  cudaError_t e = allow_shared(dense_tree_tc_kernel<ROWS, PACKED>, P::bytes(kMaxSeqs));
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  e = maps_of(da.a, 2, P::kUnit, &mk, &mv);
  if (e != cudaSuccess) return e;
  dense_tree_tc_kernel<ROWS, PACKED><<<da.blocks, P::kThreads, smem, stream>>>(da, mk, mv);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_join<__nv_bfloat16, P>(da, stream);
}

template <int ROWS>
size_t part_bytes() {
  // two partials a block, and the drafted keys' part of a piece
  return static_cast<size_t>(152) * TcShape<ROWS, false>::kResident * (ROWS * (2 * kDtPart + kAccStride) * sizeof(float) + 2 * sizeof(Split));
}

}  // namespace

// (the most of any number of rows up to this)
size_t dense_tree_tc_bytes(int rows) {
  size_t most = part_bytes<16>();
  if (rows > 16) most = std::max(most, part_bytes<32>());
  if (rows > 32) most = std::max(most, part_bytes<48>());
  if (rows > 48) most = std::max(most, part_bytes<64>());
  return most;
}

cudaError_t launch_dense_tree_tc(const DenseTreeArgs& da, cudaStream_t stream) {
  const int rows = da.a.G * da.a.T;
  if (rows <= 16) return launch<16>(da, stream);
  // 32 rows: a packed schedule where the other would leave room for one block an SM.  200 sequences of 1024 rows take 136 us
  // without and 141 with it, 256 244 and 172, 400 378 and 263.
  if (rows <= 32) return 2 * (TcShape<32, false>::bytes(da.a.B) + 1024) > 228 * 1024 ? launch<32, true>(da, stream) : launch<32>(da, stream);
  if (rows <= 48) return launch<48>(da, stream);
  return launch<64>(da, stream);
}

}  // namespace fibattn
