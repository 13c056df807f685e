// The attention weight of cached rows for bf16 with more than 8 query rows a key head (sm_103a): the products on the 5th-generation
// tensor cores, the rest as in weigh.cu.
//
// A tile is 128 rows of K, as TMA leaves them (K-major, 128-byte swizzle), times up to 128 query rows of the split query, all three parts
// added up into one accumulator of tensor memory: S [128 rows x queries] (32 queries at most: side by side in one of three times as many columns, of
// which the threads add up three).  There a thread has a row, so its sum is a loop over its columns:
//   one load from tensor memory, one exp2, one add; no shuffle.  (That -lse is added by one more product, ones times its parts: with an add
//   and a read of lse a column the warps that sum were what bounded it.)
// A task is up to four tiles (of few: two, or one) of a sequence, layer and head, which stay in shared memory while its queries pass by (those that see the
// tile), or, where there are 64 at most, eight tiles that pass by the queries.  Blocks take tasks as they come, so that those of
// prompts, which cost from 4 products to hundreds, fill all SMs.  A row's sum is one thread's, in the order of the queries, whichever block it is.
//
// What bounds it: few query rows the read of K, many the products (13 a tile and chunk of queries).  32 tokens over 4 sequences of up to 8192
// rows, 16 layers, 8 heads (242 MB): 47 us with the queries' launch; once under way a block's tasks follow one another in 2.95 us, which is HBM's rate,
// the rest is the start, the queries' 6 and the last tasks.  (13 products of 32 columns a tile, 30 us of tensor pipe, took 49.)  Prompts of
// 2048 and 1523, 4 layers (104 million scores, in whole tiles 112): 50 us, 14 of them the queries' launch; the products alone are 23 where all SMs have the same, 25 on
// the one that has the longest task.
//
// Block: 16 warps that sum (four a tile), and one warp each for the tasks, the queries, the copies of each of the four tiles and the
// products of each.  A warp's step (a wait, a few addresses, a copy) takes 500 to 1000 cycles, as much as a tile may take: with one
// warp for tasks, queries and copies a window of 32 tokens took 85 us, whatever else was changed, with warps of their own for
// the copies 73, with four for the products 67.
#include <climits>

#include "tcgen05.cuh"
#include "tree_dense.cuh"
#include "weigh.cuh"

namespace fibattn {

namespace {

constexpr int kTile = 128, kTiles = 4, kGroupRows = kTile * kTiles;  // rows of a round
constexpr int kTileBytes = kTile * kD * 2;
constexpr int kOnesBytes = kTile * 16 * 2;  // 128 rows of 1 1 1 0 ..., whose product with the references' parts is each of them
constexpr int kSumWarps = 4 * kTiles, kIssuer = kSumWarps, kFeedK = kIssuer + kTiles, kTasks = kFeedK + kTiles, kFeedQ = kTasks + 1;
constexpr int kThreads = 32 * (kFeedQ + 1);

// COLS query rows a product.  32, where a key head has no more: the three parts are columns of one product (96, which takes hardly longer than 32 do)
// and a score is the sum of three; one buffer of tensor memory a tile.  64, where it has no more: the parts add up in 64 columns, two buffers.
// Both have two slots of shared memory a tile, and tasks of two rounds; else 128, one buffer, and two slots for the first two tiles.  A product takes
// 48.5, 54 and 64.6 cycles with 32, 64 and 128 columns, and what a warp does a chunk of queries beside its columns costs as much as 40 of them:
// prompts of 2048 took 66 us with 64.  The window above takes 47 us with 32 columns; with 64 tokens, or twice the query heads, 64 columns: 54 (floor 36).
template <int COLS>
struct Shape {
  static constexpr bool kSpread = COLS == kSpreadRows;  // parts are columns: of 8 queries 24, part by part
  static constexpr int kRounds = COLS < 128 ? 2 : 1;
  static constexpr int kBufferCols = kSpread ? 128 : COLS, kBuffers = 512 / (kTiles * kBufferCols);  // of tensor memory, a tile
  static constexpr int kSlots = COLS < 128 ? 2 * kTiles : kTiles + 2, kQuerySlots = 2;
  static constexpr int kRefBytes = (kSpread ? 3 : 1) * kRefGroupBytes;  // of 8 queries
  static constexpr int kQueryRefs = COLS / 8 * kGroupBytes, kQuerySlot = kQueryRefs + COLS / 8 * kRefBytes;  // a slot: queries, references
  static constexpr int kQueries = kSlots * kTileBytes, kOnes = kQueries + kQuerySlots * kQuerySlot, kSchedule = kOnes + kOnesBytes;
  static_assert(kQuerySlot % 1024 == 0, "layout");
  // Tile t's slots: this one and, where there is one, the next.
  __device__ __forceinline__ static int slot(int t) { return COLS < 128 || t < 2 ? 2 * t : t + 2; }
  __device__ __forceinline__ static int slots(int t) { return COLS < 128 || t < 2 ? 2 : 1; }
};

struct TcTask {
  int b, l, h;
  int before, used;  // query row m sees rows up to before + m / G; query rows
  int first;
  int r0, end, rounds;  // rows r0 .. end - 1; rounds 0: there is none any more
};

// A barrier of one warp's or of one tile's warps, which wait for each of its rounds, one after the other: its parity cannot tell one that is a
// round ahead from one that is not.
struct TcBars {
  uint64_t k_full[2 * kTiles], k_empty[2 * kTiles];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2 * kTiles], s_empty[2 * kTiles];
  uint64_t t_full[2], t_empty[2];
  uint64_t drained;
  TcTask task[2];
  uint32_t tmem;
  int err;
  int parts;  // of a round's four tiles 4, 2 or 1 are a task (1, 2, 4)
  int issued[kTiles];  // chunks of queries that are past the products of the tile
};

// Rows of a task of a sequence with `used` query rows; parts: of a round's four tiles.
template <int COLS>
__device__ __forceinline__ int task_rows(int used, int parts) {
  return used <= COLS ? Shape<COLS>::kRounds * kGroupRows / parts : kGroupRows / parts;
}
// The chunk of queries from which on some of them see row r, of a task.
template <int COLS>
__device__ __forceinline__ int first_chunk(const WeighArgs& a, const TcTask& k, int r) {
  return max(0, r - k.before) * a.G / COLS;
}
template <int COLS>
__device__ __forceinline__ int chunks(const TcTask& k) {
  return (k.used + COLS - 1) / COLS;
}
// Columns of chunk c's product.
template <int COLS>
__device__ __forceinline__ int columns(const TcTask& k, int c) {
  return min(COLS, (k.used - c * COLS + 15) / 16 * 16);
}

// The sequences, in shared memory: the tasks before each, and what it is.
struct TcSchedule {
  long long* start;  // [B + 1]
  WeighSeq* seq;     // [B]
  __device__ __forceinline__ TcSchedule(unsigned char* at, int B) : start(reinterpret_cast<long long*>(at)), seq(reinterpret_cast<WeighSeq*>(start + B + 1)) {}
  static size_t bytes(int B) { return sizeof(long long) * (B + 1) + sizeof(WeighSeq) * B; }
};

// Task `id` of the call, if there is one (rounds > 0): sequences in order, of each the first rows of all layers and heads before the next.
template <int COLS>
__device__ __forceinline__ TcTask task_at(const WeighArgs& a, const TcSchedule& sch, unsigned long long id, int parts) {
  TcTask k = {};
  const long long* start = sch.start;
  if (id >= static_cast<unsigned long long>(start[a.B])) return k;
  const long long u = static_cast<long long>(id);
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= u)
      lo = mid;
    else
      hi = mid;
  }
  const WeighSeq s = sch.seq[lo];
  const int per = a.c.L * a.c.H;
  const long long off = u - start[lo];
  const int j = off < 1LL << 31 ? static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(per)) : static_cast<int>(off / per);
  const int lh = static_cast<int>(off - static_cast<long long>(j) * per);
  k.b = lo;
  k.l = lh / a.c.H;
  k.h = lh - k.l * a.c.H;
  k.before = s.len - s.n;
  k.used = s.n * a.G;
  k.first = s.first;
  const int rows = task_rows<COLS>(k.used, parts);
  k.r0 = j * rows;
  k.end = min(s.len, k.r0 + rows);
  k.rounds = (k.end - k.r0 + kGroupRows - 1) / kGroupRows;
  return k;
}

__device__ __forceinline__ void ld16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
}
// Every load so far has come; r passes through, so that no use of it is moved ahead.
__device__ __forceinline__ void wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]),
                 "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// ... r too had come by then.
__device__ __forceinline__ void pass16(uint32_t (&r)[16]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]),
                 "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

// Offset of cache row r in K, in elements; -1 where its page lies outside the pool.
__device__ __forceinline__ long long row_at(const WeighArgs& a, const TcTask& k, int r) {
  const CacheDev& c = a.c;
  const int page = __ldg(c.table + static_cast<size_t>(k.b) * c.max_pages + (r >> c.shift));
  if (page < 0 || page >= c.n_pages) return -1;
  return ((((static_cast<long long>(k.l) * c.n_pages + page) * c.H + k.h) << c.shift) + (r & (c.P - 1))) * kD;
}

// What queries [m0, m1) give to row r where some sum of its products is a NaN.  It may come of an infinite key, whose products with the
// parts are infinities of opposite signs: then the signs of the upper part decide.
__device__ __noinline__ float add_infinite(const WeighArgs& a, const TcTask& k, int r, int m0, int m1) {
  const long long at = row_at(a, k, r);
  if (at < 0) return 0.f;
  const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(a.c.k) + at;
  uint64_t set = 0, negative = 0;
  for (int d = 0; d < kD; ++d) {
    const float x = __bfloat162float(row[d]);
    if (isnan(x)) return x;
    if (isinf(x)) set |= 1ull << d;
    if (x < 0.f) negative |= 1ull << d;
  }
  if (set == 0) return __int_as_float(0x7fffffff);
  const size_t task = (static_cast<size_t>(k.l) * a.B + k.b) * a.c.H + k.h;
  const unsigned char* parts = a.parts + task * (a.mpad / 8) * kGroupBytes;
  float sum = 0.f;
  for (int m = m0; m < m1 && !isnan(sum); ++m) {
    const unsigned char* q = parts + static_cast<size_t>(m >> 3) * kGroupBytes + (m & 7) * 128;
    float s = 0.f;
    for (uint64_t left = set; left != 0; left &= left - 1) {
      const int d = __ffsll(static_cast<long long>(left)) - 1;
      const float x = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(q + (((d >> 3) ^ (m & 7)) << 4) + (d & 7) * 2));
      s += x * (negative >> d & 1 ? -INFINITY : INFINITY);
    }
    sum += ex2(s + a.refs[task * a.mpad + m]);
  }
  return sum;
}

template <int COLS>
__global__ void __launch_bounds__(kThreads, 1) weigh_tc_kernel(const __grid_constant__ WeighArgs a, const __grid_constant__ CUtensorMap map_k) {
  using P = Shape<COLS>;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(16) TcBars bars;
  volatile int& s_err = bars.err;
  const TcSchedule sch(smem + P::kSchedule, a.B);
  long long* start = sch.start;
  const CacheDev& c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    s_err = 0;
    for (int t = 0; t < kTiles; ++t) bars.issued[t] = 0;
    for (int s = 0; s < P::kSlots; ++s) {
      mbar_init(&bars.k_full[s], 1);
      mbar_init(&bars.k_empty[s], 1);
    }
    for (int s = 0; s < P::kQuerySlots; ++s) {
      mbar_init(&bars.q_full[s], 1);
      mbar_init(&bars.q_empty[s], kTiles);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.t_full[s], 1);
      mbar_init(&bars.t_empty[s], 1 + 2 * kTiles + kSumWarps);
    }
    for (int s = 0; s < kTiles * P::kBuffers; ++s) {
      mbar_init(&bars.s_full[s], 1);
      mbar_init(&bars.s_empty[s], 4);
    }
    mbar_init(&bars.drained, kTiles);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  for (int i = tid; i < kOnesBytes / 16; i += kThreads)  // [16][2][8] words of a row's 8 values
    *reinterpret_cast<uint4*>(smem + P::kOnes + 16 * i) = i & 8 ? make_uint4(0, 0, 0, 0) : make_uint4(0x3f803f80u, 0x3f80u, 0, 0);
  fence_smem();
  for (int b = tid; b < a.B; b += kThreads) {
    bool ok;
    sch.seq[b] = weigh_seq(a, b, &ok);
  }
  __syncthreads();
  if (warp == 0) {
    auto count = [&](int parts) {  // the tasks before each sequence's; all of them
      long long base = 0;
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        long long own = 0;
        if (b < a.B && sch.seq[b].n > 0) {
          const int rows = task_rows<COLS>(sch.seq[b].n * a.G, parts);
          own = static_cast<long long>((sch.seq[b].len + rows - 1) / rows) * c.L * c.H;
        }
        long long x = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, x, d);
          if (lane >= d) x += y;
        }
        if (b < a.B) start[b] = base + x - own;
        base += __shfl_sync(0xffffffffu, x, 31);
      }
      if (lane == 0) start[a.B] = base;
      return base;
    };
    // Where few tasks leave blocks without one, they are of two tiles or of one: 32 of 1000 rows and 8000 query rows 102 us, of four tiles 141; 8 of
    // 1672 rows and as many query rows 25, 34.
    const long long total = count(1);
    int parts = 1;
    if constexpr (COLS == 128)
      while (parts < kTiles && total * parts * 2 <= gridDim.x) parts *= 2;
    if (parts > 1) count(parts);
    if (lane == 0) bars.parts = parts;
  }
  if (warp == kIssuer) tmem_alloc(&bars.tmem, 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars.tmem, 0), base = smem_addr(smem);
  // The rows of a block's first task need nothing of the queries' launch: their copies do not wait for it.
  if (warp != kTasks && (warp < kFeedK || warp >= kFeedK + kTiles)) wait_for_first();

  auto wait_for = [&](uint64_t* bar, uint32_t parity, unsigned long long limit_ns) {
    if (warp_wait(bar, parity, limit_ns, &s_err)) return true;
    s_err = 1;
    if (lane == 0) atomicExch(a.status, kStatusTimeout);
    return false;
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_for(bar, parity, a.wait_ns); };
  // Task number tc of the block, and that this warp has read it (a warp that is done with it only later says so itself).
  auto read = [&](int tc, TcTask* k) {
    if (!wait_for(&bars.t_full[tc & 1], (tc >> 1) & 1, a.task_ns)) return false;
    *k = bars.task[tc & 1];
    return k->rounds > 0;
  };
  auto release = [&](int tc) {  // (no fence, which would wait for what the warp has under way: the next task is written as this one is read)
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.t_empty[tc & 1]);
  };

  if (warp == kTasks) {
    // =================================================================== tasks
    for (int tc = 0; wait(&bars.t_empty[tc & 1], ((tc >> 1) & 1) ^ 1); ++tc) {
      unsigned long long id = tc == 0 ? blockIdx.x : lane == 0 ? gridDim.x + atomicAdd(a.next, 1ull) : 0;
      const TcTask k = task_at<COLS>(a, sch, __shfl_sync(0xffffffffu, id, 0), bars.parts);
      if (lane == 0) {
        bars.task[tc & 1] = k;
        mbar_arrive(&bars.t_full[tc & 1]);
      }
      __syncwarp();
      if (k.rounds == 0) break;
      if (tc == 0) wait_for_first();  // (before the limits below begin: they are of this launch's work; and before `next` is read)
      // A long task is taken alone, till the last of its queries is under way: one that waits for its block waits for nothing else.
      if (k.used > COLS && !wait_for(&bars.t_empty[tc & 1], (tc >> 1) & 1, a.task_ns)) break;
    }
  } else if (warp == kFeedQ) {
    // =================================================================== copies of queries
    int n = 0;
    bool go = true;
    TcTask k;
    for (int tc = 0; go && read(tc, &k); ++tc) {
      const size_t m = ((static_cast<size_t>(k.l) * a.B + k.b) * c.H + k.h) * a.mpad;
      const int c1 = chunks<COLS>(k);
      for (int ch = first_chunk<COLS>(a, k, k.r0); ch < c1; ++ch, ++n) {
        const int slot = n % P::kQuerySlots, cols = columns<COLS>(k, ch);
        go = wait(&bars.q_empty[slot], ((n / P::kQuerySlots) & 1) ^ 1);
        if (!go) break;
        if (lane == 0) {
          unsigned char* to = smem + P::kQueries + slot * P::kQuerySlot;
          const size_t at = (m + static_cast<size_t>(ch) * COLS) / 8;
          mbar_arrive_tx(&bars.q_full[slot], cols / 8 * (kGroupBytes + P::kRefBytes));
          bulk_g2s(to, a.parts + at * kGroupBytes, cols / 8 * kGroupBytes, &bars.q_full[slot]);
          bulk_g2s(to + P::kQueryRefs, a.ref_parts + at * P::kRefBytes, cols / 8 * P::kRefBytes, &bars.q_full[slot]);
        }
        __syncwarp();
      }
      release(tc);
    }
    // nothing may be in flight when the block ends
    if (lane == 0)
      for (int x = max(0, n - P::kQuerySlots); x < n; ++x) mbar_wait(&bars.q_full[x % P::kQuerySlots], (x / P::kQuerySlots) & 1, kDrainNs);
    __syncwarp();
  } else if (warp >= kFeedK && warp < kFeedK + kTiles) {
    // =================================================================== copies of rows: tile t of each round
    const int t = warp - kFeedK, box = min(kTile, c.P), slots = P::slots(t);  // rows a copy
    int n = 0;
    bool go = true, left_out[2] = {false, false};        // slots that the test hook does not fill
    TcTask k;
    for (int tc = 0; go && read(tc, &k); ++tc) {
      release(tc);
      for (int x = 0; x < k.rounds; ++x) {
        const int r0 = k.r0 + x * kGroupRows + t * kTile;
        if (r0 >= k.end) break;
        const int boxes = (min(kTile, k.end - r0) + box - 1) / box, s = n & (slots - 1), slot = P::slot(t) + s;
        // lane i copies box i
        const int r = r0 + lane * box;
        int id = lane < boxes ? __ldg(c.table + static_cast<size_t>(k.b) * c.max_pages + (r >> c.shift)) : 0;
        if (id < 0 || id >= c.n_pages) {
          atomicExch(a.status, kStatusDeviceAssert);
          id = 0;
        }
        go = wait(&bars.k_empty[slot], ((n / slots) & 1) ^ 1);
        if (!go) break;
        ++n;
        left_out[s] = a.skip_copy && x == 0 && t == 0;
        if (left_out[s]) continue;
        if (lane == 0) mbar_arrive_tx(&bars.k_full[slot], boxes * box * kD * 2);
        __syncwarp();
        if (lane < boxes)
          tma_3d(base + slot * kTileBytes + lane * box * 128, &map_k, 0, ((id * c.H + k.h) << c.shift) + (r & (c.P - 1)), k.l, &bars.k_full[slot]);
        __syncwarp();
      }
      if (tc == 0) wait_for_first();
    }
    if (lane == 0)
      for (int x = max(0, n - slots); x < n; ++x)
        if (!left_out[x & (slots - 1)]) mbar_wait(&bars.k_full[P::slot(t) + (x & (slots - 1))], (x / slots) & 1, kDrainNs);
    __syncwarp();
  } else if (warp >= kIssuer && warp < kIssuer + kTiles) {
    // =================================================================== products of tile t of each round
    // The warp goes as one and its values are the same in all lanes (shuffled, so that the compiler can tell); one lane issues.
    auto same = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    // Descriptors count 16 bytes: 32 bytes on a k step, a part's 1024 on a part (as columns: eight more rows of the operand).
    constexpr uint32_t kLead = 16 / 16 << 16, kRowsHigh = 1024 / 16 | 1u << 14 | 2u << 29;
    constexpr uint32_t kQueryHigh = (P::kSpread ? kPartBytes : kGroupBytes) / 16 | 1u << 14 | 2u << 29;
    // Ones and references without swizzle: 8 rows of 16 bytes, their other half of k 128 bytes on, 8 more rows 256.
    constexpr uint32_t kPlainLead = 128 / 16 << 16, kPlainHigh = kRefGroupBytes / 16 | 1u << 14;
    auto at = [](uint32_t high, uint32_t low) { return static_cast<uint64_t>(high) << 32 | low; };
    const int t = same(warp - kIssuer);
    const int slots = P::slots(t), slot0 = P::slot(t), buf0 = t * P::kBuffers;
    const uint32_t rows0 = (base + slot0 * kTileBytes) >> 4 | kLead, query0 = (base + P::kQueries) >> 4 | kLead, refs0 = (base + P::kQueries + P::kQueryRefs) >> 4 | kPlainLead,
                   ones = (base + P::kOnes) >> 4 | kPlainLead, out0 = tmem + buf0 * P::kBufferCols;
    // With one buffer a tile the tiles go in order, so that a tile's scores are there while the next one's are made: side by side those of all
    // four were there together, then all sums were formed, and prompts of 2048 took 59 us.
    constexpr bool kInTurn = COLS == 128;
    volatile int* issued = bars.issued;
    auto turn = [&](int step) {  // the tile before this one is past chunk `step` of the block
      const unsigned long long since = global_ns();
      while (issued[t - 1] <= step && !s_err) {
        if (global_ns() - since > a.wait_ns) {
          s_err = 1;
          if (lane == 0) atomicExch(a.status, kStatusTimeout);
        }
      }
      return __all_sync(0xffffffffu, !s_err);
    };
    int qs = 0, q_round = 0, filled = 0, done = 0, step = 0;  // tiles copied, products made, chunks
    bool go = true;
    TcTask k;
    for (int tc = 0; go && read(tc, &k); ++tc) {
      const int c0 = same(first_chunk<COLS>(a, k, k.r0)), c1 = same(chunks<COLS>(k)), last = same(columns<COLS>(k, chunks<COLS>(k) - 1));
      int from[P::kRounds];  // the first chunk that sees rows of the tile
#pragma unroll
      for (int x = 0; x < P::kRounds; ++x) {
        const int r = k.r0 + x * kGroupRows + t * kTile;
        from[x] = same(x < k.rounds && r < k.end ? first_chunk<COLS>(a, k, r) : INT_MAX);
      }
      release(tc);
      for (int ch = c0; ch < c1 && go; ++ch) {
        go = wait(&bars.q_full[qs], q_round & 1);
        if (!go) break;
        const uint32_t query = query0 + qs * (P::kQuerySlot / 16), refs = refs0 + qs * (P::kQuerySlot / 16);
        const uint32_t desc = product_of(kTile, (P::kSpread ? 3 : 1) * (ch == c1 - 1 ? last : COLS), false, false);
#pragma unroll
        for (int x = 0; x < P::kRounds; ++x) {
          if (from[x] > ch) break;
          // the tile is there from the first chunk that sees it to the last
          const int slot = filled & (slots - 1), buf = done & (P::kBuffers - 1);
          if (ch == max(from[x], c0)) go = wait(&bars.k_full[slot0 + slot], (filled / slots) & 1);
          if (go) go = wait(&bars.s_empty[buf0 + buf], ((done / P::kBuffers) & 1) ^ 1);
          if (kInTurn && go && t > 0) go = turn(step);
          if (!go) break;
          fence_after();
          const uint32_t rows = rows0 + slot * (kTileBytes / 16), d = out0 + buf * P::kBufferCols;
          if (one_lane()) {
#pragma unroll
            for (int part = P::kSpread ? 0 : 2; part >= 0; --part)
#pragma unroll
              for (int y = 0; y < 4; ++y)
                mma_tc(d, at(kRowsHigh, rows + 2 * y), at(kQueryHigh, query + part * (kPartBytes / 16) + 2 * y), desc, (!P::kSpread && part < 2) || y > 0);
            mma_tc(d, at(kPlainHigh, ones), at(kPlainHigh, refs), desc, true);  // (the last: a sum is cut where it is added to)
            commit_tc(&bars.s_full[buf0 + buf]);
            if (ch == c1 - 1) commit_tc(&bars.k_empty[slot0 + slot]);
          }
          ++done;
          if (ch == c1 - 1) ++filled;
        }
        ++step;
        if (kInTurn && lane == 0) issued[t] = step;
        if (go && one_lane()) commit_tc(&bars.q_empty[qs]);
        if (++qs == P::kQuerySlots) {
          qs = 0;
          ++q_round;
        }
      }
    }
    if (one_lane()) {  // nothing may be in flight when the block ends
      commit_tc(&bars.drained);
      mbar_wait(&bars.drained, 0, kDrainNs);
    }
    __syncwarp();
  } else {
    // =================================================================== sums
    const int mine = warp >> 2, wq = warp & 3;  // the warp's tile of a round, and its 32 rows of that
    const uint32_t lanes = static_cast<uint32_t>(wq) << 21;
    int done = 0;
    bool go = true;
    TcTask k;
    for (int tc = 0; go && read(tc, &k); ++tc) {
      release(tc);
      float* out = a.weights + ((static_cast<size_t>(k.l) * c.S + k.b) * c.H + k.h) * a.rows;
      const int32_t* table = c.table + static_cast<size_t>(k.b) * c.max_pages;
      float sum[P::kRounds], old[P::kRounds];
      int page[P::kRounds];  // (looked at in the end)
      const int first0 = k.r0 + mine * kTile, row0 = first0 + wq * 32 + lane;  // the tile's and the thread's row in the first round
#pragma unroll
      for (int x = 0; x < P::kRounds; ++x) {
        const int r = row0 + x * kGroupRows;
        sum[x] = 0.f;
        old[x] = x < k.rounds && r < k.first && r < k.end ? out[r] : 0.f;
        page[x] = x < k.rounds && r < k.end ? __ldg(table + (r >> c.shift)) : -1;
      }
      const int c1 = chunks<COLS>(k);
      for (int ch = first_chunk<COLS>(a, k, k.r0); ch < c1 && go; ++ch) {
        const int cols = columns<COLS>(k, ch), m0 = ch * COLS;
#pragma unroll
        for (int x = 0; x < P::kRounds; ++x) {
          const int first = first0 + x * kGroupRows, r = row0 + x * kGroupRows;
          if (x >= k.rounds || first >= k.end || max(0, first - k.before) * a.G >= m0 + COLS) break;  // none of these queries sees the tile
          const int buf = mine * P::kBuffers + (done & (P::kBuffers - 1));
          // (the chunks that see the tile may be the last of the task's)
          go = wait_for(&bars.s_full[buf], (done / P::kBuffers) & 1, a.task_ns);
          if (!go) break;
          ++done;
          fence_after();
          // whether every column is a query row that sees all rows of the tile
          const bool all = m0 + cols <= k.used && max(0, first + kTile - 1 - k.before) * a.G <= m0;
          const int lo = max(0, r - k.before) * a.G - m0, hi = k.used - m0;  // the columns that see row r
          float s[4] = {0.f, 0.f, 0.f, 0.f};
          auto use = [&]<bool ALL>(const uint32_t (&z)[16], int col) {
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              float y[4] = {__uint_as_float(z[e]), __uint_as_float(z[e + 1]), __uint_as_float(z[e + 2]), __uint_as_float(z[e + 3])};
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                y[f] = ex2(y[f]);
                if (!ALL) y[f] = col + e + f >= lo && col + e + f < hi ? y[f] : 0.f;
              }
              s[0] += y[0];
              s[1] += y[1];
              s[2] += y[2];
              s[3] += y[3];
            }
          };
          const uint32_t from = tmem + buf * P::kBufferCols + lanes;
          auto add = [&]<bool ALL>() {
            if constexpr (P::kSpread) {
#pragma unroll
              for (int col = 0; col < COLS; col += 16) {  // 16 queries: twice the columns of 8 queries' upper, middle and lower parts
                if (col >= cols) break;
                uint32_t x[16], y[16], z[16];
                ld16(from + 3 * col, x);
                ld16(from + 3 * col + 16, y);
                ld16(from + 3 * col + 32, z);
                wait16(x);
                pass16(y);
                pass16(z);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  x[e] = __float_as_uint(__uint_as_float(x[e]) + (__uint_as_float(x[8 + e]) + __uint_as_float(y[e])));
                  x[8 + e] = __float_as_uint(__uint_as_float(y[8 + e]) + (__uint_as_float(z[e]) + __uint_as_float(z[8 + e])));
                }
                use.template operator()<ALL>(x, col);
              }
              return;
            }
#pragma unroll
            for (int col = 0; col < COLS; col += 32) {
              if (col >= cols) break;
              uint32_t y[16], z[16];
              const bool second = col + 16 < cols;
              ld16(from + col, y);
              if (second) ld16(from + col + 16, z);
              wait16(y);
              use.template operator()<ALL>(y, col);
              if (!second) break;
              pass16(z);
              use.template operator()<ALL>(z, col + 16);
            }
          };
          if (all)
            add.template operator()<true>();
          else
            add.template operator()<false>();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.s_empty[buf]);
          float part = (s[0] + s[1]) + (s[2] + s[3]);
          if (isnan(part) && r < k.end) part = add_infinite(a, k, r, max(m0, m0 + lo), min(m0 + cols, k.used));
          sum[x] += part;
        }
      }
      if (!go) break;
#pragma unroll
      for (int x = 0; x < P::kRounds; ++x) {
        const int r = row0 + x * kGroupRows;
        if (page[x] >= 0 && page[x] < c.n_pages) out[r] = old[x] + sum[x];
      }
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kIssuer) tmem_free(tmem, 512);
}

// K of all layers as rows of 64 values, [layers][pages * heads * rows]; a copy takes `box` rows.
cudaError_t map_layers(CUtensorMap* m, const CacheDev& c, int box) {
  const cuuint64_t rows = (static_cast<cuuint64_t>(c.n_pages) * c.H) << c.shift;
  const cuuint64_t dims[3] = {kD, rows, static_cast<cuuint64_t>(c.L)}, strides[2] = {kD * 2, rows * kD * 2};
  const cuuint32_t boxes[3] = {kD, static_cast<cuuint32_t>(box), 1}, steps[3] = {1, 1, 1};
  const EncodeTiled encode = encode_tiled();
  if (encode == nullptr) return cudaErrorNotSupported;
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, c.k, dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

}  // namespace

template <int COLS>
static cudaError_t launch(const WeighArgs& a, cudaStream_t stream) {
  using P = Shape<COLS>;
  cudaError_t e = allow_shared(weigh_tc_kernel<COLS>, P::kSchedule + TcSchedule::bytes(kMaxSeqs));
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  e = map_layers(&map, a.c, a.c.P < kTile ? a.c.P : kTile);
  if (e != cudaSuccess) return e;
  return launch_second(weigh_tc_kernel<COLS>, dim3(152), kThreads, P::kSchedule + TcSchedule::bytes(a.B), stream, a, map);  // one block an SM
}

cudaError_t launch_weigh_tc(const WeighArgs& a, cudaStream_t stream) {
  if (a.G * a.T <= kSpreadRows) return launch<kSpreadRows>(a, stream);
  return a.G * a.T <= 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

}  // namespace fibattn
