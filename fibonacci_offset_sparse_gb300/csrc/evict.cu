// Eviction from the paged cache by accumulated attention weight (sm_103a).
//
// Of a sequence's rows the first, the last and, of those between, the heaviest stay, for each layer and key head by itself; they move
// down in order, K turned from its old place to the new one (e^{-i (old - new) theta} a pair; a plan that does not rotate moves
// it as it is).  Two launches, the second a programmatic dependent of the first:
//   plan   one block: what each sequence keeps, the free pages that take the place of shared ones, tables, counts, lengths;
//   evict  a block (of few of them, a cluster) a sequence, layer and head: the weight of the last row that stays, the list of rows that stay, in order, and their
//          weights; then K and V by that list.  A row never moves up, so the rows that a step writes were all read in it or before, and
//          one barrier a step, between its reads and its writes, keeps them apart.  No order of blocks matters.
// What bounds it: the rows' bytes, read and written once; one block's search runs beside the others' moves (in launches of their own search
// and move took 449 us, together 365).  16 sequences of 2048 to 4096 rows cut to 2048, 16 layers, 8 heads, bf16 (2.05 GB): plan 9 us,
// evict 344 (6.0 TB/s); 65536 rows cut to 16384 (1.12 GB, 128 blocks): 220 (5.1 TB/s, after a search of some 45 us in which nothing moves);
// 16 beams that share prompts of 2048, cut to 1024 (0.82 GB, shared pages from L2): 120.
#include "cache_dev.cuh"

namespace fibattn {

namespace {

// What the plan leaves for the others; keep < 0: nothing to do.
struct EvictJob {
  int len, keep;
  int same;  // pages in front that stay as they are
  int unused;
};

struct EvictArgs {
  CacheDev c;
  int B, rows, sink, recent, n_max;
  const int32_t* keep;
  float* weights;    // [L, S, H, rows]
  int32_t* dropped;  // [B] or null
  const float2* rope_lo;
  const float2* rope_hi;
  float2 turn[kFreq];  // theta / 2 pi as a sum of two, whether the plan rotates or not
  EvictJob* jobs;
  int32_t* list;   // free pages taken
  int32_t* old;    // [S, max_pages]: the pages that a sequence held; ~page where a new one takes its place
  int32_t* taken;  // [S, max_pages / 32 up]: how many of 32 pages are replaced
  int32_t* stays;  // [L, S, H, rows]: the row that comes to place j
};

// ------------------------------------------------------------------------------------- plan --
// A thread a sequence for lengths and sums; 32 pages of one a warp at a time, from another warp on for each sequence, so that all
// warps share a long one and as many short ones go side by side.
constexpr int kShortList = 4096;

__global__ void __launch_bounds__(kPlanThreads) evict_plan_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int s_len[kMaxSeqs], s_keep[kMaxSeqs], s_off[kMaxSeqs];
  __shared__ int s_sums[33], s_low;
  __shared__ int32_t s_list[kShortList];
  let_second_start();
  const CacheDev& c = a.c;
  const int b = threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cursor = max(0, min(c.state[kStateCursor], c.n_pages));
  int counts[4];
  load_refs(c, (cursor & ~3) + 4 * static_cast<int>(threadIdx.x), cursor, counts);
  bool bad = false;
  int len = 0, keep = -1;
  if (b < a.B) {
    len = c.lens[b];
    const int k = a.keep[b];
    bad = k < 0 || len < 0 || len > static_cast<long long>(c.max_pages) * c.P;
    if (!bad && len > k) {
      bad = a.sink + a.recent > k || len > a.rows || len > a.n_max;
      keep = k;
    }
  }
  s_len[b] = len;
  s_keep[b] = keep;
  s_off[b] = 0;
  if (b == 0) s_low = c.n_pages;
  bool any_bad = __syncthreads_or(bad);
  bad = false;
  const int chunks = (c.max_pages + 31) / 32;
  if (!any_bad) {
    for (int s = 0; s < a.B; ++s) {
      if (s_keep[s] < 0) continue;
      const int had = pages_of(c, s_len[s]), has = pages_of(c, s_keep[s]), same = min(a.sink >> c.shift, has);
      const int32_t* row = c.table + static_cast<size_t>(s) * c.max_pages;
      int32_t* old = a.old + static_cast<size_t>(s) * c.max_pages;
      for (int at = (warp - s) & 31; at * 32 < had; at += kPlanThreads / 32) {
        const int j = at * 32 + lane, page = j < had ? row[j] : 0;
        const bool in = page >= 0 && page < c.n_pages;
        bad |= !in;
        const bool taken = in && j >= same && j < has && c.refs[page] > 1;
        if (j < had) old[j] = taken ? ~page : page;
        const int n = __popc(__ballot_sync(0xffffffffu, taken));
        if (lane == 0) {
          a.taken[static_cast<size_t>(s) * chunks + at] = n;
          if (n > 0) atomicAdd(&s_off[s], n);
        }
      }
    }
  }
  any_bad = __syncthreads_or(bad) || any_bad;
  int total;
  const int off = block_scan_1024(any_bad ? 0 : s_off[b], s_sums, &total);
  s_off[b] = off;
  int32_t* list = total <= kShortList ? s_list : a.list;
  const bool enough = any_bad || (total <= c.n_pages && find_free(c, cursor, counts, total, list, s_sums) == total);
  if (any_bad || !enough) {  // nothing changes
    if (b < a.B) a.jobs[b] = EvictJob{0, -1, 0, 0};
    if (b == 0) c.state[kStateStatus] = any_bad ? kStatusDeviceAssert : kStatusNoPages;
    return;
  }
  __syncthreads();  // every offset is there
  int lowest = c.n_pages;
  for (int s = 0; s < a.B; ++s) {
    if (s_keep[s] < 0) continue;
    const int had = pages_of(c, s_len[s]), has = pages_of(c, s_keep[s]);
    int32_t* row = c.table + static_cast<size_t>(s) * c.max_pages;
    const int32_t* old = a.old + static_cast<size_t>(s) * c.max_pages;
    for (int at = (warp - s) & 31; at * 32 < had; at += kPlanThreads / 32) {
      const int j = at * 32 + lane, page = j < had ? old[j] : 0;  // (this lane wrote it)
      const bool taken = page < 0, gone = j < had && j >= has;
      const unsigned mask = __ballot_sync(0xffffffffu, taken);
      if (mask != 0) {  // its place in the list: behind what the chunks in front take
        int before = 0;
        for (int i = lane; i < at; i += 32) before += __ldcg(a.taken + static_cast<size_t>(s) * chunks + i);
        before = s_off[s] + __reduce_add_sync(0xffffffffu, before);
        if (taken) {
          const int id = list[before + __popc(mask & ((1u << lane) - 1u))];
          row[j] = id;
          c.refs[id] = 1;
        }
      }
      if (gone) row[j] = -1;
      if (taken || gone) {
        const int left = taken ? ~page : page;
        if (atomicSub(&c.refs[left], 1) == 1) lowest = min(lowest, left);
      }
    }
  }
  lowest = __reduce_min_sync(0xffffffffu, lowest);
  if (lane == 0 && lowest < c.n_pages) atomicMin(&s_low, lowest);
  if (b < a.B) {
    a.jobs[b] = EvictJob{len, keep, keep < 0 ? 0 : min(a.sink >> c.shift, pages_of(c, keep)), 0};
    if (keep >= 0) c.lens[b] = keep;
    if (a.dropped != nullptr && keep >= 0) a.dropped[b] += len - keep;
  }
  __syncthreads();
  if (b == 0) c.state[kStateCursor] = min(s_low, total > 0 ? list[total - 1] + 1 : cursor);
}

// ----------------------------------------------------------------------------------- select --
// A block a sequence, layer and head: rows [sink, end) compete for `need` places.  The last weight that stays is found by passes over the
// weights, each of which counts keys in up to 2048 bins of the range that is left, at first that from the least key to the largest: weights
// have few exponents, and threads that meet in a bin go one after the other.  (Bins of the words' upper 11 bits: 157 us for 128 blocks
// of 65536 rows; two bits a pass by comparing and adding up: 88 us for 1920 blocks of 2048 to 4096 rows, which took 55 by the upper bits.)
constexpr int kBins = 2048;

// Weights in ascending order as unsigned words: the two zeros alike (their sum with 0 is +0), a NaN (the sum's, all ones but the sign) 0.  The
// largest is infinity's, 0xff800001.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u)) + 1u;
}

// The key of the last row that stays, and how many of the rows with that key do (the first ones).
struct Least {
  uint32_t key;
  int quota;
};

// What the block's threads share of it.
template <int THREADS>
struct Finder {
  int hist[kBins];
  int sums[32];
  uint32_t lows[32], highs[32];
  int bin, above;

  // The least and the largest of the block's keys.
  __device__ __forceinline__ void range(uint32_t& low, uint32_t& high) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    if (lane == 0) {
      lows[warp] = low;
      highs[warp] = high;
    }
    __syncthreads();
    low = __reduce_min_sync(0xffffffffu, lane < THREADS / 32 ? lows[lane] : 0xffffffffu);
    high = __reduce_max_sync(0xffffffffu, lane < THREADS / 32 ? highs[lane] : 0u);
  }

  // The highest bin with at least `need` keys in it and above; above: those above it.  Ends synchronised.
  __device__ __forceinline__ void find(int need) {
    constexpr int EACH = kBins / THREADS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, top = kBins - 1 - EACH * static_cast<int>(threadIdx.x);
    int own = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) own += hist[top - i];  // from the highest bin down
    int inc = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int before = __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0) + inc - own;
    if (before < need && before + own >= need) {  // one thread
      int i = 0;
      for (int x = hist[top]; before + x < need; x = hist[top - ++i]) before += x;
      bin = top - i;
      above = before;
    }
    __syncthreads();
  }

  // each(f): f(key) for every key of the thread that competes, the same ones at every call.
  template <typename Each>
  __device__ __forceinline__ Least least(int need, Each&& each) {
    uint32_t low = 0xffffffffu, high = 0;
    each([&](uint32_t key) {
      low = min(low, key);
      high = max(high, key);
    });
    range(low, high);
    uint32_t span = high - low;  // what is left: keys low .. low + span
    for (bool all = true;; all = false) {
      const int bits = 32 - __clz(span), shift = max(0, bits - 11);
      for (int i = threadIdx.x; i < kBins; i += THREADS) hist[i] = 0;
      __syncthreads();
      each([&](uint32_t key) {
        if (all || key - low <= span) atomicAdd(&hist[(key - low) >> shift], 1);
      });
      __syncthreads();
      find(need);
      low += static_cast<uint32_t>(bin) << shift;
      need -= above;
      if (shift == 0) return Least{low, need};
      span = (1u << shift) - 1;
      __syncthreads();  // (the bin has been read)
    }
  }
};

// The rows of a sequence, layer and head that stay, in order, into `stays`; their weights move.  The least weight needs the lengths alone, so it
// is looked for while the plan is made, with the length that there is; where the plan has been there before, it is looked for behind it.  (Behind
// it every time: 3 sequences of 200 rows 15.5 us, which take 12.2; the 16 beams 140, which take 137.)
template <int THREADS, int KEYS>
struct Select {
  static constexpr int WARPS = THREADS / 32, ROWS = THREADS * KEYS;
  static_assert(ROWS < 1 << 15, "two counts a word");
  Finder<THREADS> finder;
  int words[KEYS][WARPS], rows[KEYS], len;

  // False: nothing to do.
  __device__ __forceinline__ bool run(const EvictArgs& a, int b, float* w, int32_t* stays, EvictJob* its) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float x[KEYS];  // the weights of a step's rows: r0 + i THREADS + thread
    Least least{0xfffffffeu, 0};  // (above every weight's)
    auto load = [&](int r0, int most) {
      if (r0 + ROWS <= most) {
#pragma unroll
        for (int i = 0; i < KEYS; ++i) x[i] = w[r0 + i * THREADS + threadIdx.x];
      } else {
#pragma unroll
        for (int i = 0; i < KEYS; ++i) x[i] = r0 + i * THREADS + static_cast<int>(threadIdx.x) < most ? w[r0 + i * THREADS + threadIdx.x] : 0.f;
      }
    };
    EvictJob job{};
    if (threadIdx.x == 0) len = __ldcg(a.c.lens + b);  // (one thread: the plan may be about to change it)
    __syncthreads();
    job.len = len;
    job.keep = a.keep[b];
    bool planned = false;
    if (job.len > a.rows || job.len <= job.keep || a.sink + a.recent > job.keep) job.len = 0;  // the plan refuses it or has been there
    while (true) {
      const int end = job.len - a.recent, need = job.keep - a.sink - a.recent;
      if (job.len <= ROWS) {
        load(0, job.len);
        if (job.len > 0 && need > 0)
          least = finder.least(need, [&](auto&& f) {
#pragma unroll
            for (int i = 0; i < KEYS; ++i) {
              if (i * THREADS >= end) break;
              const int r = i * THREADS + threadIdx.x;
              if (r >= a.sink && r < end) f(order_of(x[i]));
            }
          });
      } else if (need > 0) {
        least = finder.least(need, [&](auto&& f) {
          for (int r0 = a.sink; r0 < end; r0 += ROWS) {
            load(r0, end);
            if (r0 + ROWS <= end) {
#pragma unroll
              for (int i = 0; i < KEYS; ++i) f(order_of(x[i]));
            } else {
#pragma unroll
              for (int i = 0; i < KEYS; ++i)
                if (r0 + i * THREADS + static_cast<int>(threadIdx.x) < end) f(order_of(x[i]));
            }
          }
        });
      }
      if (planned) break;
      wait_for_first();
      const int before = job.len;
      job = a.jobs[b];
      *its = job;
      if (job.keep < 0) return false;
      if (job.len == before) break;
      planned = true;
    }
    const int end = job.len - a.recent;
    // The list.  What stays before a row: the rows that stay for certain, and of those with the least key the first ones.  Both counts
    // in one word.
    int sure = 0, ties = 0;  // of the steps before
    for (int r0 = 0; r0 < job.len; r0 += ROWS) {
      if (job.len > ROWS) load(r0, job.len);
      auto key_of = [&](int i) {  // of a row that stays for certain above all; 1 + that of none
        const int r = r0 + i * THREADS + threadIdx.x;
        return r < a.sink || r >= end ? 0xffffffffu : order_of(x[i]);
      };
      auto in = [&](int i) { return r0 + i * THREADS + static_cast<int>(threadIdx.x) < job.len; };
#pragma unroll
      for (int i = 0; i < KEYS; ++i) {
        if (r0 + i * THREADS >= job.len) break;
        const uint32_t key = key_of(i);
        const int n = __popc(__ballot_sync(0xffffffffu, in(i) && key > least.key)) | __popc(__ballot_sync(0xffffffffu, key == least.key)) << 16;
        if (lane == 0) words[i][warp] = n;
      }
      __syncthreads();  // (and every weight of the step has been read)
      for (int i = warp; i < KEYS; i += WARPS) {  // exclusive sums over the warps
        if (r0 + i * THREADS >= job.len) break;
        const int own = lane < WARPS ? words[i][lane] : 0;
        int inc = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, d);
          if (lane >= d) inc += y;
        }
        if (lane < WARPS) words[i][lane] = inc - own;
        if (lane == 31) rows[i] = inc;
      }
      __syncthreads();
      int all = 0;  // before the run of THREADS rows
#pragma unroll
      for (int i = 0; i < KEYS; ++i) {
        if (r0 + i * THREADS >= job.len) break;
        const int r = r0 + i * THREADS + threadIdx.x;
        const uint32_t key = key_of(i);
        const bool stay = in(i) && key > least.key, tie = key == least.key;
        const unsigned below = (1u << lane) - 1u, stay_mask = __ballot_sync(0xffffffffu, stay), tie_mask = __ballot_sync(0xffffffffu, tie);
        const int word = all + words[i][warp], tied = ties + (word >> 16) + __popc(tie_mask & below);
        if (stay || (tie && tied < least.quota)) {
          const int at = sure + (word & 0xffff) + __popc(stay_mask & below) + min(tied, least.quota);
          stays[at] = r;
          if (at != r) w[at] = x[i];
        }
        all += rows[i];
      }
      sure += all & 0xffff;
      ties += all >> 16;
      __syncthreads();
    }
    return true;
  }
};

// ------------------------------------------------------------------------------------- move --
// e^{i d theta} of the pairs 8t .. 8t+7.  bf16: d theta in turns, its fraction exact to 2^-24, and the approximate sine and cosine, 1.2e-6 in
// all, far below a step of the type; float32: the tables', whose 256 bytes a row are as much to read as K and V (bf16 with them: 128 blocks of
// 16384 rows moved took 140 us more).
template <typename DT>
__device__ __forceinline__ void factors(const EvictArgs& a, int d, int t, float2 (&e)[8]) {
  if constexpr (sizeof(DT) == 2) {
    const float x = static_cast<float>(d);  // exact
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float2 turn = a.turn[8 * t + u];
      const float p = x * turn.x;
      const float f = ((p - rintf(p)) + fmaf(x, turn.x, -p)) + x * turn.y;
      __sincosf(6.283185307179586f * f, &e[u].y, &e[u].x);
    }
  } else {
    rope_row(a.rope_lo, a.rope_hi, d, t, e);
  }
}

// Whether the plan rotates, as its tables say now (a captured call follows them, not what was set at the capture): pair 0 turns by an angle of 1 a
// position, whatever the base, and by none in the tables of a plan that does not rotate.
__device__ __forceinline__ bool rotates(const EvictArgs& a) {
  return __ldg(&a.rope_lo[kFreq].y) != 0.f;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;\n" ::: "memory");
}

// The rows of K or V that `stays` lists come to places job.same * P ..: a quad a row, each thread dims 8t .. and 32+8t .. of it: two 16-byte
// words of bf16, four of float32.  By THREADS threads of each of `blocks` blocks, `rank` among them, with a barrier of their own (of several blocks: the
// cluster's).
template <typename DT, int THREADS, int ROWS, bool SHARED>
__device__ __forceinline__ void move_rows(const EvictArgs& a, const EvictJob& job, int v, int l, int b, int h, const int32_t* stays, int rank, int blocks) {
  const int thread = threadIdx.x % THREADS;
  constexpr int kWords = static_cast<int>(sizeof(DT)), kHalf = kWords / 2;  // 16-byte words a thread and row
  constexpr int kStep = THREADS / 4 * ROWS;
  const CacheDev& c = a.c;
  const int32_t* old = a.old + static_cast<size_t>(b) * c.max_pages;
  const int32_t* now = c.table + static_cast<size_t>(b) * c.max_pages;
  DT* pool = static_cast<DT*>(v ? c.v : c.k) + ((static_cast<size_t>(l) * c.n_pages * c.H + h) << c.shift) * kD;
  const size_t page_elems = (static_cast<size_t>(c.H) << c.shift) * kD;
  const int t = thread & 3, quad = thread >> 2, mask = c.P - 1;
  int turns = v == 0 && rotates(a);
  for (int start = job.same << c.shift; start < job.keep; start += kStep * blocks) {
    const int j0 = start + kStep * rank;
    uint4 x[ROWS][kWords];
    int src[ROWS];  // -1: none, or it is there already
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int j = j0 + i * (THREADS / 4) + quad;
      src[i] = j < job.keep ? stays[j] : -1;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (src[i] < 0) continue;
      const int page = old[src[i] >> c.shift];
      const uint4* p = reinterpret_cast<const uint4*>(pool + (page < 0 ? ~page : page) * page_elems + static_cast<size_t>(src[i] & mask) * kD);
      if (src[i] == j0 + i * (THREADS / 4) + quad && page >= 0) {
        src[i] = -1;
        continue;
      }
#pragma unroll
      for (int k = 0; k < kWords; ++k) x[i][k] = p[(k / kHalf) * 4 * kHalf + t * kHalf + k % kHalf];
    }
    // every row of the step has been read
    if (SHARED)
      cluster_sync();
    else
      asm volatile("barrier.cta.sync %0, %1;\n" ::"r"(1 + v), "n"(THREADS) : "memory");
    asm volatile("" : "+r"(turns));  // (no loop of its own for either value: 65536 rows cut to 16384 took 265 us with that, 251 so)
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int j = j0 + i * (THREADS / 4) + quad;
      if (src[i] < 0) continue;
      if (turns && src[i] != j) {
        float2 e[8];
        float y[16];
        factors<DT>(a, src[i] - j, t, e);
        if constexpr (sizeof(DT) == 2) {
          const uint32_t u[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            y[2 * k] = bf_lo(u[k]);
            y[2 * k + 1] = bf_hi(u[k]);
          }
          rotate_part(y, e, true);
          x[i][0] = make_uint4(pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3]), pack_bf2(y[4], y[5]), pack_bf2(y[6], y[7]));
          x[i][1] = make_uint4(pack_bf2(y[8], y[9]), pack_bf2(y[10], y[11]), pack_bf2(y[12], y[13]), pack_bf2(y[14], y[15]));
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            y[4 * k] = __uint_as_float(x[i][k].x);
            y[4 * k + 1] = __uint_as_float(x[i][k].y);
            y[4 * k + 2] = __uint_as_float(x[i][k].z);
            y[4 * k + 3] = __uint_as_float(x[i][k].w);
          }
          rotate_part(y, e, true);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x[i][k] = make_uint4(__float_as_uint(y[4 * k]), __float_as_uint(y[4 * k + 1]), __float_as_uint(y[4 * k + 2]), __float_as_uint(y[4 * k + 3]));
        }
      }
      uint4* p = reinterpret_cast<uint4*>(pool + now[j >> c.shift] * page_elems + static_cast<size_t>(j & mask) * kD);
#pragma unroll
      for (int k = 0; k < kWords; ++k) p[(k / kHalf) * 4 * kHalf + t * kHalf + k % kHalf] = x[i][k];
    }
  }
}

// SHARED: a cluster a sequence, layer and head, whose first block makes the list that all move by.
template <typename DT, int THREADS, int KEYS, bool SHARED>
__global__ void __launch_bounds__(THREADS, THREADS >= 1024 ? 1 : 4) evict_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int ROWS = sizeof(DT) == 2 ? 4 : 2;
  __shared__ Select<THREADS, KEYS> select;
  const CacheDev& c = a.c;
  int rank = 0, blocks = 1;
  if constexpr (SHARED) {
    asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(blocks));
  }
  const int per = c.L * c.H, at = blockIdx.x / blocks, b = at / per, lh = at % per, l = lh / c.H, h = lh % c.H;
  const size_t task = (static_cast<size_t>(l) * c.S + b) * c.H + h;
  int32_t* stays = a.stays + task * a.rows;
  EvictJob job;
  if (rank == 0) {
    if (!select.run(a, b, a.weights + task * a.rows, stays, &job)) return;
  } else {
    wait_for_first();
    job = a.jobs[b];
    if (job.keep < 0) return;  // (and so in every block of the cluster)
  }
  if (SHARED) cluster_sync();
  // One half of the threads K, the other V: one reads while the other writes.  (One after the other, 128 blocks of 65536 rows cut to 16384:
  // 264 us.)
  move_rows<DT, THREADS / 2, ROWS, SHARED>(a, job, threadIdx.x / (THREADS / 2), l, b, h, stays, rank, blocks);
}

template <typename DT, int THREADS, int KEYS>
cudaError_t launch_in(const EvictArgs& a, unsigned tasks, unsigned blocks, cudaStream_t stream) {
  return blocks == 1 ? launch_second(evict_kernel<DT, THREADS, KEYS, false>, dim3(tasks), THREADS, 0, stream, a)
                     : launch_second_in_clusters(evict_kernel<DT, THREADS, KEYS, true>, dim3(tasks * blocks), blocks, THREADS, 0, stream, a);
}

// By what the weights' rows can hold: up to 5120 rows a block of 256 threads, four of which share an SM; longer ones 1024 threads, which beyond
// 16384 rows read the weights anew in each pass.  (Lengths are on the device, so that room for more rows than there are takes the larger block: 2048 blocks
// of 4096 rows cut to 2048 take 387 us with room for 5121 or 131072, 363 with room for 5120; of 2048 to 1024 227, 189; of 600 to 500 61, 43.)  Where these leave SMs without one, 2, 4 or 8 blocks of 256 rows or more to each (15 of 30300 rows
// cut to 10211, bf16: 47 us, one block each 116; 32 of 2077 cut to 1782, float32: 22, 54).
template <typename DT>
cudaError_t launch(const EvictArgs& a, unsigned tasks, cudaStream_t stream) {
  const bool few = a.rows <= 256 * 20;
  unsigned blocks = 1;
  while (blocks < 8 && tasks * blocks * 2 <= (few ? 152 * 4 : 152) && a.rows > 256 * static_cast<int>(blocks)) blocks *= 2;
  return few ? launch_in<DT, 256, 20>(a, tasks, blocks, stream) : launch_in<DT, 1024, 16>(a, tasks, blocks, stream);
}

size_t rows_bytes(const fib_attn_cache& c, int rows) {
  return round_up(sizeof(int32_t) * static_cast<size_t>(c.n_layers) * c.max_seqs * c.heads * static_cast<size_t>(rows));
}
size_t tables_bytes(const fib_attn_cache& c) {
  return round_up(sizeof(int32_t) * static_cast<size_t>(c.max_seqs) * static_cast<size_t>(c.max_pages));
}
size_t taken_bytes(const fib_attn_cache& c) {
  return round_up(sizeof(int32_t) * static_cast<size_t>(c.max_seqs) * ((static_cast<size_t>(c.max_pages) + 31) / 32));
}

}  // namespace

// jobs, the free pages taken, the old tables and what is replaced of them, the rows that stay
size_t cache_evict_workspace_bytes(const fib_attn_cache& c, int rows) {
  return round_up(sizeof(EvictJob) * kMaxSeqs) + round_up(sizeof(int32_t) * static_cast<size_t>(c.n_pages)) + tables_bytes(c) +
         taken_bytes(c) + rows_bytes(c, rows);
}

cudaError_t launch_cache_evict(const fib_attn_cache& cache, int B, int rows, const int32_t* keep, int sink, int recent, int n_max,
                               float* weights, int32_t* dropped, const float2* lo_tab, const float2* hi_tab, const float2* turn, void* ws,
                               cudaStream_t stream) {
  EvictArgs a;
  a.c = device_view(cache);
  a.B = B;
  a.rows = rows;
  a.sink = sink;
  a.recent = recent;
  a.n_max = n_max;
  a.keep = keep;
  a.weights = weights;
  a.dropped = dropped;
  a.rope_lo = lo_tab;
  a.rope_hi = hi_tab;
  for (int m = 0; m < kFreq; ++m) a.turn[m] = turn[m];
  unsigned char* at = static_cast<unsigned char*>(ws);
  a.jobs = reinterpret_cast<EvictJob*>(at);
  at += round_up(sizeof(EvictJob) * kMaxSeqs);
  a.list = reinterpret_cast<int32_t*>(at);
  at += round_up(sizeof(int32_t) * static_cast<size_t>(cache.n_pages));
  a.old = reinterpret_cast<int32_t*>(at);
  at += tables_bytes(cache);
  a.taken = reinterpret_cast<int32_t*>(at);
  at += taken_bytes(cache);
  a.stays = reinterpret_cast<int32_t*>(at);
  evict_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned tasks = static_cast<unsigned>(B) * cache.n_layers * cache.heads;
  return cache.dtype == FIB_DTYPE_F32 ? launch<float>(a, tasks, stream) : launch<__nv_bfloat16>(a, tasks, stream);
}

}  // namespace fibattn
