// The attention weight of cached rows for bf16 with more than 8 query rows a key head (sm_103a): the products on the 5th-generation
// tensor cores, the rest as in weigh.cu.
//
// A tile is 128 rows of K, as TMA leaves them (K-major, 128-byte swizzle), times up to 128 query rows of the split query, all three parts
// added up into one accumulator of tensor memory: S [128 rows x queries].  There a thread has a row, so its sum is a loop over its columns:
//   one load from tensor memory, one add (a pair at a time), one exp2, one add; no shuffle.
// A task is up to four tiles of a sequence, layer and head, which stay in shared memory while its queries pass by 64 at a time
// (of those that see the tile); blocks take tasks as they come, so that those of prompts, which cost from 4 products to hundreds, fill all
// SMs.  A row's sum is one thread's, in the order of the queries, whichever block it is.
//
// What bounds it: few query rows the read of K, many the products (three parts) and exp2.
//
// Block: 16 warps that sum (four a tile of the task), the feeder, and a warp whose one lane issues the products.
#include "tcgen05.cuh"
#include "tree_dense.cuh"
#include "weigh.cuh"

namespace fibattn {

namespace {

constexpr int kTile = 128, kTiles = 4, kGroupRows = kTile * kTiles;  // rows of a task
constexpr int kCols = 64;                                             // query rows of a product
constexpr int kTileBytes = kTile * kD * 2, kSlots = 6;
// Slots of queries: one is free again when its products are done and its references read, so it is for some 2.5 us, of which
// the products of 128 columns took 1.6: with two slots of 128 columns prompts of 2048 took 61 us, a window of 32 tokens 85.
constexpr int kQuerySlots = 4;
constexpr int kQueryBytes = kCols / 8 * kGroupBytes, kQuerySlot = kQueryBytes + 1024;  // and their references; a multiple of 1024
// Buffers of tensor memory, kCols columns each: two a tile of the task, so that a barrier is waited for by the four warps of one tile
// alone, one round after the other.  (Its parity cannot tell a warp that is a round ahead from one that is not.)
constexpr int kBuffers = 2 * kTiles;
constexpr int kShort = 4;                                             // chunks of a task that is short
constexpr int kSumWarps = 4 * kTiles, kFeeder = kSumWarps, kIssuer = kSumWarps + 1, kThreads = 32 * (kSumWarps + 2);
constexpr int kQueries = kSlots * kTileBytes, kSchedule = kQueries + kQuerySlots * kQuerySlot;
static_assert(kQuerySlot % 1024 == 0 && kBuffers * kCols == 512, "layout");

struct TcTask {
  int b, l, h;
  int len, before, used;  // rows; query row m sees rows up to before + m / G; query rows
  int first;
  int r0, tiles;          // tiles 0: there is none any more
  int pad;
};

struct TcBars {
  uint64_t k_full[kSlots], k_empty[kSlots];
  uint64_t q_full[kQuerySlots], q_empty[kQuerySlots];
  uint64_t s_full[kBuffers], s_empty[kBuffers];
  uint64_t t_full[2], t_empty[2];
  uint64_t drained;
  TcTask task[2];
  uint32_t tmem;
  int err;
};

// The chunk of queries from which on some of them see row r, of a task.
__device__ __forceinline__ int first_chunk(const WeighArgs& a, const TcTask& k, int r) { return max(0, r - k.before) * a.G / kCols; }
__device__ __forceinline__ int chunks(const TcTask& k) { return (k.used + kCols - 1) / kCols; }
// Columns of chunk c's product.
__device__ __forceinline__ int columns(const TcTask& k, int c) { return min(kCols, (k.used - c * kCols + 15) / 16 * 16); }

// The sequences, in shared memory: the tasks before each, and what it is.
struct TcSchedule {
  long long* start;  // [B + 1]
  WeighSeq* seq;     // [B]
  __device__ __forceinline__ TcSchedule(unsigned char* at, int B) : start(reinterpret_cast<long long*>(at)), seq(reinterpret_cast<WeighSeq*>(start + B + 1)) {}
  static size_t bytes(int B) { return sizeof(long long) * (B + 1) + sizeof(WeighSeq) * B; }
};

// Task `id` of the call, if there is one (tiles > 0): sequences in order, of each the first rows of all layers and heads before the next.
__device__ __forceinline__ TcTask task_at(const WeighArgs& a, const TcSchedule& sch, unsigned long long id) {
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
  k.len = s.len;
  k.before = s.len - s.n;
  k.used = s.n * a.G;
  k.first = s.first;
  k.r0 = j * kGroupRows;
  k.tiles = min(kTiles, (s.len - k.r0 + kTile - 1) / kTile);
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

__global__ void __launch_bounds__(kThreads, 1) weigh_tc_kernel(const __grid_constant__ WeighArgs a, const __grid_constant__ CUtensorMap map_k) {
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(16) TcBars bars;
  volatile int& s_err = bars.err;
  const TcSchedule sch(smem + kSchedule, a.B);
  long long* start = sch.start;
  const CacheDev& c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    s_err = 0;
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&bars.k_full[s], 1);
      mbar_init(&bars.k_empty[s], 1);
    }
    for (int s = 0; s < kQuerySlots; ++s) {
      mbar_init(&bars.q_full[s], 1);
      mbar_init(&bars.q_empty[s], 1 + kSumWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.t_full[s], 1);
      mbar_init(&bars.t_empty[s], 1 + kSumWarps);
    }
    for (int s = 0; s < kBuffers; ++s) {
      mbar_init(&bars.s_full[s], 1);
      mbar_init(&bars.s_empty[s], 4);
    }
    mbar_init(&bars.drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  for (int b = tid; b < a.B; b += kThreads) {
    bool ok;
    const WeighSeq s = weigh_seq(a, b, &ok);
    sch.seq[b] = s;
    start[b] = s.n == 0 ? 0 : static_cast<long long>((s.len + kGroupRows - 1) / kGroupRows) * c.L * c.H;
  }
  __syncthreads();
  if (warp == 0) {
    long long base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      const long long own = b < a.B ? start[b] : 0;
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
  }
  if (warp == kIssuer) tmem_alloc(&bars.tmem, kBuffers * kCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = bars.tmem, base = smem_addr(smem);
  wait_for_first();

  if (warp == kFeeder) {
    // =================================================================== feeder
    const int box = min(kTile, c.P);  // rows a copy
    // A task's number, in lane 0, and not waited for before it is used.  Taken early where tasks are short; where they are long
    // late, as one that waits for its block waits for nothing else.
    auto fetch = [&] { return lane == 0 ? atomicAdd(a.next, 1ull) : 0ull; };
    auto known = [&](unsigned long long id) { return task_at(a, sch, __shfl_sync(0xffffffffu, id, 0)); };
    auto page_of = [&](const TcTask& k) {  // of the lane-th page of the task's rows
      const int at = (k.r0 >> c.shift) + lane;
      return k.tiles > 0 && at < c.max_pages ? __ldg(c.table + static_cast<size_t>(k.b) * c.max_pages + at) : -1;
    };
    unsigned long long id = fetch();
    TcTask now = known(id), next = {};
    int page = page_of(now), next_page = 0;
    bool taken = false;  // id is the number of the task after the next that is known
    int tc = 0, kc = 0, qc = 0;
    uint32_t left_out = 0;  // slots that the test hook never fills
    bool stop = false;
    while (!stop) {
      if (!warp_wait(&bars.t_empty[tc & 1], ((tc >> 1) & 1) ^ 1, a.wait_ns, &s_err)) break;
      if (lane == 0) {
        bars.task[tc & 1] = now;
        mbar_arrive(&bars.t_full[tc & 1]);
      }
      __syncwarp();
      ++tc;
      if (now.tiles == 0) break;
      const size_t task = (static_cast<size_t>(now.l) * a.B + now.b) * c.H + now.h;
      const int c0 = first_chunk(a, now, now.r0), c1 = chunks(now);
      const bool is_short = c1 - c0 <= kShort;
      auto look_ahead = [&] {
        if (!taken) id = fetch();
        next = known(id);
        next_page = page_of(next);
        taken = false;
      };
      if (is_short) {  // the next one's pages, and the number of the one behind it, come while this one's copies wait for their slots
        look_ahead();
        if (next.tiles > 0) {
          id = fetch();
          taken = true;
        }
      }
      for (int ch = c0; ch < c1 && !stop; ++ch, ++qc) {
        const int slot = qc % kQuerySlots, n = columns(now, ch);
        if (!warp_wait(&bars.q_empty[slot], ((qc / kQuerySlots) & 1) ^ 1, a.wait_ns, &s_err)) {
          stop = true;
          break;
        }
        if (lane == 0) {
          unsigned char* to = smem + kQueries + slot * kQuerySlot;
          const size_t m = task * a.mpad + static_cast<size_t>(ch) * kCols;
          mbar_arrive_tx(&bars.q_full[slot], n / 8 * kGroupBytes + n * 4);
          bulk_g2s(to, a.parts + m / 8 * kGroupBytes, n / 8 * kGroupBytes, &bars.q_full[slot]);
          bulk_g2s(to + kQueryBytes, a.refs + m, n * 4, &bars.q_full[slot]);
        }
        __syncwarp();
        if (ch != c0) continue;
        for (int t = 0; t < now.tiles; ++t, ++kc) {
          const int ks = kc % kSlots, rows = min(kTile, now.len - now.r0 - t * kTile), boxes = (rows + box - 1) / box;
          if (!warp_wait(&bars.k_empty[ks], ((kc / kSlots) & 1) ^ 1, a.wait_ns, &s_err)) {
            stop = true;
            break;
          }
          // lane x copies box x: page (tile's first row + x box) / P of the task
          const int first = t * kTile + lane * box, id = __shfl_sync(0xffffffffu, page, (first >> c.shift) & 31);
          if (a.skip_copy && t == 0) {
            left_out |= 1u << ks;
            continue;
          }
          left_out &= ~(1u << ks);
          if (lane == 0) mbar_arrive_tx(&bars.k_full[ks], boxes * box * kD * 2);
          __syncwarp();
          if (lane < boxes) {
            const bool ok = id >= 0 && id < c.n_pages;
            if (!ok) atomicExch(a.status, kStatusDeviceAssert);
            tma_3d(base + ks * kTileBytes + lane * box * 128, &map_k, 0, (((ok ? id : 0) * c.H + now.h) << c.shift) + (first & (c.P - 1)), now.l,
                   &bars.k_full[ks]);
          }
          __syncwarp();
        }
      }
      if (!is_short && !stop) look_ahead();
      now = next;
      page = next_page;
    }
    if (s_err || stop) {
      s_err = 1;
      if (lane == 0) atomicExch(a.status, kStatusTimeout);
    }
    // nothing may be in flight when the block ends
    if (lane == 0) {
      for (int x = max(0, kc - kSlots); x < kc; ++x)
        if (!(left_out >> (x % kSlots) & 1)) mbar_wait(&bars.k_full[x % kSlots], (x / kSlots) & 1, kDrainNs);
      for (int x = max(0, qc - kQuerySlots); x < qc; ++x) mbar_wait(&bars.q_full[x % kQuerySlots], (x / kQuerySlots) & 1, kDrainNs);
    }
    __syncwarp();
  } else if (warp == kIssuer) {
    // =================================================================== products
    if (one_lane()) {
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (s_err) return false;
        if (mbar_wait(bar, parity, a.wait_ns)) return true;
        s_err = 1;
        atomicExch(a.status, kStatusTimeout);
        return false;
      };
      int tc = 0, kc = 0, qc = 0, done[kTiles] = {};  // done: products for each tile of the tasks
      bool go = true;
      while (go && wait(&bars.t_full[tc & 1], (tc >> 1) & 1)) {
        const TcTask k = bars.task[tc & 1];
        __threadfence_block();
        mbar_arrive(&bars.t_empty[tc & 1]);
        ++tc;
        if (k.tiles == 0) break;
        const int c0 = first_chunk(a, k, k.r0), c1 = chunks(k);
        int seen = 0;  // tiles whose copy has been waited for
        for (int ch = c0; ch < c1 && go; ++ch, ++qc) {
          go = wait(&bars.q_full[qc % kQuerySlots], (qc / kQuerySlots) & 1);
          if (!go) break;
          // descriptors' addresses count 16 bytes: 32 bytes on a k step, a part's 1024 on a part
          const uint64_t q = matrix_at(base + kQueries + qc % kQuerySlots * kQuerySlot, 16, kGroupBytes, 2);
          const uint32_t desc = product_of(kTile, columns(k, ch), false, false);
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            // (nor do later tiles' rows have a query that sees them)
            if (!go || t >= k.tiles || first_chunk(a, k, k.r0 + t * kTile) > ch) break;
            const int ks = (kc + t) % kSlots, buf = 2 * t + (done[t] & 1);
            if (t >= seen) {
              go = wait(&bars.k_full[ks], ((kc + t) / kSlots) & 1);
              if (!go) break;
              seen = t + 1;
            }
            go = wait(&bars.s_empty[buf], ((done[t] >> 1) & 1) ^ 1);
            if (!go) break;
            fence_after();
            const uint64_t rows = matrix_at(base + ks * kTileBytes, 16, 1024, 2);
            const uint32_t d = tmem + buf * kCols;
#pragma unroll
            for (int part = 2; part >= 0; --part)
#pragma unroll
              for (int x = 0; x < 4; ++x) mma_tc(d, rows + 2 * x, q + part * (kPartBytes / 16) + 2 * x, desc, part < 2 || x > 0);
            commit_tc(&bars.s_full[buf]);
            if (ch == c1 - 1) commit_tc(&bars.k_empty[ks]);
            ++done[t];
          }
          if (go) commit_tc(&bars.q_empty[qc % kQuerySlots]);
        }
        kc += k.tiles;
      }
      commit_tc(&bars.drained);  // nothing may be in flight when the block ends
      mbar_wait(&bars.drained, 0, kDrainNs);
    }
    __syncwarp();
  } else {
    // =================================================================== sums
    const int mine = warp >> 2, wq = warp & 3;  // the warp's tile of a task, and its 32 rows of that
    const uint32_t lanes = static_cast<uint32_t>(wq) << 21;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (warp_wait(bar, parity, a.wait_ns, &s_err)) return true;
      s_err = 1;
      if (lane == 0) atomicExch(a.status, kStatusTimeout);
      return false;
    };
    int tc = 0, qc = 0, done = 0;
    bool go = true;
    while (go && wait(&bars.t_full[tc & 1], (tc >> 1) & 1)) {
      const TcTask k = bars.task[tc & 1];
      __threadfence_block();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.t_empty[tc & 1]);
      ++tc;
      if (k.tiles == 0) break;
      float* out = a.weights + ((static_cast<size_t>(k.l) * c.S + k.b) * c.H + k.h) * a.rows;
      const int r = k.r0 + mine * kTile + wq * 32 + lane;  // the thread's row
      float sum = 0.f;
      const float old = r < k.first && r < k.len ? out[r] : 0.f;
      const int page = r < k.len ? __ldg(c.table + static_cast<size_t>(k.b) * c.max_pages + (r >> c.shift)) : -1;  // (looked at in the end)
      const int c0 = first_chunk(a, k, k.r0), c1 = chunks(k);
      for (int ch = c0; ch < c1 && go; ++ch, ++qc) {
        const int n = columns(k, ch), m0 = ch * kCols;
        const float* ref = reinterpret_cast<const float*>(smem + kQueries + qc % kQuerySlots * kQuerySlot + kQueryBytes);
        go = wait(&bars.q_full[qc % kQuerySlots], (qc / kQuerySlots) & 1);
        if (!go) break;
        if (mine < k.tiles && first_chunk(a, k, k.r0 + mine * kTile) <= ch) {  // some of these queries see rows of the tile
          const int buf = 2 * mine + (done & 1);
          go = wait(&bars.s_full[buf], (done >> 1) & 1);
          ++done;
          if (!go) break;
          fence_after();
          // whether every column is a query row that sees all rows of the tile
          const bool all = m0 + n <= k.used && k.before + m0 / a.G >= k.r0 + (mine + 1) * kTile - 1;
          const int lo = max(0, r - k.before) * a.G - m0, hi = k.used - m0;  // the columns that see row r
          float s[4] = {0.f, 0.f, 0.f, 0.f};
          auto use = [&]<bool ALL>(const uint32_t (&x)[16], int col) {
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 r4 = *reinterpret_cast<const float4*>(ref + col + e);
              float y[4] = {__uint_as_float(x[e]), __uint_as_float(x[e + 1]), __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])};
              add2(y[0], y[1], r4.x, r4.y);
              add2(y[2], y[3], r4.z, r4.w);
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                y[f] = ex2(y[f]);
                if (!ALL) y[f] = col + e + f >= lo && col + e + f < hi ? y[f] : 0.f;
              }
              add2(s[0], s[1], y[0], y[1]);
              add2(s[2], s[3], y[2], y[3]);
            }
          };
          const uint32_t from = tmem + buf * kCols + lanes;
          auto add = [&]<bool ALL>() {
            uint32_t x[16], y[16];
            ld16(from, x);
            wait16(x);
            for (int col = 0; col < n; col += 32) {
              const bool second = col + 16 < n;
              if (second) ld16(from + col + 16, y);
              use.template operator()<ALL>(x, col);
              if (!second) break;
              wait16(y);
              if (col + 32 < n) ld16(from + col + 32, x);
              use.template operator()<ALL>(y, col + 16);
              wait16(x);
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
          if (isnan(part) && r < k.len) part = add_infinite(a, k, r, max(m0, m0 + lo), min(m0 + n, k.used));
          sum += part;
        }
        __threadfence_block();  // the references have been read
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.q_empty[qc % kQuerySlots]);
      }
      if (!go) break;
      if (page >= 0 && page < c.n_pages) out[r] = old + sum;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kIssuer) tmem_free(tmem, kBuffers * kCols);
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

cudaError_t launch_weigh_tc(const WeighArgs& a, cudaStream_t stream) {
  cudaError_t e = allow_shared(weigh_tc_kernel, kSchedule + TcSchedule::bytes(kMaxSeqs));
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  e = map_layers(&map, a.c, a.c.P < kTile ? a.c.P : kTile);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(152);  // one block an SM
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSchedule + TcSchedule::bytes(a.B);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weigh_tc_kernel, a, map);
}

}  // namespace fibattn
