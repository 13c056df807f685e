// The paged key/value cache's own operators (sm_103a): commit (allocate, copy on write, rotate
// and store accepted tokens), fork (share, reorder, free) and compact (move pages down).
//
// Each is two launches (the fork of a small table one): a small one that reads and rewrites the tables and counts, and
// one that moves rows (commit, compact) or finishes the tables (fork).  The second is a programmatic dependent of
// the first, so its launch overlaps it, and takes the work list that the first left in the
// workspace.  All choices are made in an order that no scheduling changes: sequences ascending, free pages
// ascending; the only atomics are integer sums and minima.
//
// What bounds them: the rows' bytes where there are many, else the plan's chain of reads (counts and lengths, tables, a
// scan, a list).  Commit of 64 sequences x 16 layers, 134 MB: 21 us, 4 of them the plan; of one token for 32 sequences
// 6.5; of a prompt of 2048 tokens (16 layers, 134 MB) 27, of 4 x 8192 (2.15 GB) 326 (6.6 TB/s, 97% of a measured copy).  Fork of
// 32 x 64 and of 256 x 512 table entries 8 us.  Compaction of 1.07 GB 168 us (6.4 TB/s, 94%), of 20 MB 7.
#include "cache.cuh"
#include "tc_common.cuh"

namespace fibattn {

namespace {

constexpr int kPlanThreads = 1024;

struct CacheDev {
  int L, H, P, shift, n_pages, S, max_pages;
  void* k;
  void* v;
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  int32_t* state;
};

CacheDev device_view(const fib_attn_cache& c) {
  CacheDev d;
  d.L = c.n_layers;
  d.H = c.heads;
  d.P = c.page_rows;
  d.shift = log2_of(c.page_rows);
  d.n_pages = c.n_pages;
  d.S = c.max_seqs;
  d.max_pages = c.max_pages;
  d.k = c.k;
  d.v = c.v;
  d.table = c.table;
  d.lens = c.lens;
  d.refs = c.refs;
  d.state = c.state;
  return d;
}

__device__ __forceinline__ void wait_for_first() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void let_second_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// A kernel as a programmatic dependent of the one before it on the stream.
template <typename... Params, typename... Args>
cudaError_t launch_second(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The counts of four pages from `id` (a multiple of 4) on; 0 behind the last page.
__device__ __forceinline__ void load_counts(const CacheDev& c, int id, int (&r)[4]) {
  r[0] = r[1] = r[2] = r[3] = 0;
  if (id + 3 < c.n_pages) {
    const int4 x = *reinterpret_cast<const int4*>(c.refs + id);
    r[0] = x.x; r[1] = x.y; r[2] = x.z; r[3] = x.w;
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (id + u < c.n_pages) r[u] = c.refs[id + u];
  }
}
// ... 1 (in use) for those outside [from, n_pages).
__device__ __forceinline__ void load_refs(const CacheDev& c, int id, int from, int (&r)[4]) {
  load_counts(c, id, r);
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (id + u < from || id + u >= c.n_pages) r[u] = 1;
}

// The ids of free pages from `from` on, ascending, into list[0 .. want); returns how many there
// are up to `want`.  4096 counts a step (r: those of the first, loaded by the caller ahead of its other reads);
// stops as soon as enough are found.
__device__ int find_free(const CacheDev& c, int from, int (&r)[4], int want, int32_t* list, int* sums) {
  int found = 0;
  for (int base = from & ~3; base < c.n_pages && found < want; base += 4 * kPlanThreads) {
    const int id = base + 4 * static_cast<int>(threadIdx.x);
    if (base > from) load_refs(c, id, from, r);
    const int n = (r[0] == 0) + (r[1] == 0) + (r[2] == 0) + (r[3] == 0);
    int total;
    int at = found + block_scan_1024(n, sums, &total);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (r[u] == 0) {
        if (at < want) list[at] = id + u;
        ++at;
      }
    found += total;
  }
  __syncthreads();
  return min(found, want);
}

// ------------------------------------------------------------------------------- commit --
// Work list of a commit, in the workspace: one entry a sequence, then the free pages taken.
struct CommitJob {
  int len;  // rows before the call
  int n;    // rows gained (0: nothing to do)
  int src;  // page whose first len % P rows are copied, or -1
  int dst;  // ... into this one
};

struct CommitArgs {
  CacheDev c;
  int B, T, n_max;
  const int32_t* n_new;
  const int32_t* path;
  const void* k_new;
  const void* v_new;
  const float2* rope_lo;
  const float2* rope_hi;
  CommitJob* jobs;
  int32_t* list;
};

// One block, a thread a sequence.  What it waits for is a chain of reads, so those that depend on nothing come first, and
// the pages taken stay in shared memory unless they are many.
constexpr int kShortList = 4096;

__global__ void __launch_bounds__(kPlanThreads) commit_plan_kernel(const __grid_constant__ CommitArgs a) {
  __shared__ __align__(16) int s_page[kMaxSeqs], s_len[kMaxSeqs];
  __shared__ int s_first[kMaxSeqs], s_count[kMaxSeqs], s_off[kMaxSeqs];
  __shared__ int s_sums[33];
  __shared__ int32_t s_list[kShortList];
  let_second_start();
  const CacheDev& c = a.c;
  const int b = threadIdx.x;
  // the first step of the search for free pages, on its way while the sequences are read
  const int cursor = max(0, min(c.state[kStateCursor], c.n_pages));
  int counts[4];
  load_refs(c, (cursor & ~3) + 4 * static_cast<int>(threadIdx.x), cursor, counts);
  // ... and the first 1024 entries of the paths, with the numbers that say which of them count
  const long long nodes = a.path == nullptr ? 0 : static_cast<long long>(a.B) * a.T;
  int node = 0, seq = 0, gains = 0;
  if (threadIdx.x < nodes) {
    seq = static_cast<int>(threadIdx.x) / a.T;
    node = a.path[threadIdx.x];
    gains = a.n_new[seq];
  }
  int n = 0, len = 0, page = -1, refs = 0;
  bool bad = static_cast<int>(threadIdx.x) - seq * a.T < gains && (node < 0 || node >= a.T), part = false;
  if (b < a.B) {
    n = a.n_new[b];
    len = c.lens[b];
    bad |= n < 0 || n > a.T || len < 0 || static_cast<long long>(len) + n > static_cast<long long>(c.max_pages) * c.P ||
          (n > 0 && static_cast<long long>(len) + n > a.n_max);
    if (bad) n = 0;  // (nothing changes then)
    part = n > 0 && (len & (c.P - 1)) != 0;
    if (part) {
      page = c.table[static_cast<size_t>(b) * c.max_pages + (len >> c.shift)];
      if (page < 0 || page >= c.n_pages)
        bad = true;
      else
        refs = c.refs[page];
    }
  }
  for (long long i = threadIdx.x + kPlanThreads; i < nodes; i += kPlanThreads) {
    seq = static_cast<int>(i / a.T);
    node = a.path[i];
    bad |= i - static_cast<long long>(seq) * a.T < a.n_new[seq] && (node < 0 || node >= a.T);
  }
  // shared last pages: who else writes into the same one.  The longest keeps it (the last of those), where all
  // holders write: what the others copy from it lies in front of its new rows.
  s_page[b] = part && refs > 1 ? page : -1;
  s_len[b] = len;
  const bool any_bad = __syncthreads_or(bad);
  bool copy = false;
  if (!any_bad && part && refs > 1) {
    int writers = 0;
    bool keeps = true;
    for (int o = 0; o < a.B; o += 4) {
      const int4 p = *reinterpret_cast<const int4*>(s_page + o), l = *reinterpret_cast<const int4*>(s_len + o);
      const int ps[4] = {p.x, p.y, p.z, p.w}, ls[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool same = ps[u] == page;  // (-1 behind the last sequence)
        writers += same;
        keeps &= !same | (ls[u] < len) | ((ls[u] == len) & (o + u <= b));
      }
    }
    copy = !(writers == refs && keeps);
  }
  const int first = (len + c.P - 1) >> c.shift;
  const int fresh = n > 0 ? ((len + n + c.P - 1) >> c.shift) - first : 0;
  int total;
  const int off = block_scan_1024(any_bad ? 0 : fresh + (copy ? 1 : 0), s_sums, &total);
  int32_t* list = total <= kShortList ? s_list : a.list;
  const bool enough = any_bad || find_free(c, cursor, counts, total, list, s_sums) == total;
  if (any_bad || !enough) {  // nothing changes
    if (b < a.B) a.jobs[b] = CommitJob{0, 0, -1, -1};
    if (b == 0) c.state[kStateStatus] = any_bad ? kStatusDeviceAssert : kStatusNoPages;
    return;
  }
  s_first[b] = first;
  s_count[b] = fresh;
  s_off[b] = off + (copy ? 1 : 0);
  if (b < a.B) {
    CommitJob j{len, n, -1, -1};
    if (copy) {
      j.src = page;
      j.dst = list[off];
      c.table[static_cast<size_t>(b) * c.max_pages + (len >> c.shift)] = j.dst;
      c.refs[j.dst] = 1;
      atomicSub(&c.refs[page], 1);
    }
    a.jobs[b] = j;
    if (n > 0) c.lens[b] = len + n;
  }
  if (b == 0 && total > 0) c.state[kStateCursor] = list[total - 1] + 1;
  __syncthreads();
  for (int s = threadIdx.x >> 5; s < a.B; s += kPlanThreads / 32)
    for (int i = threadIdx.x & 31; i < s_count[s]; i += 32) {
      const int id = list[s_off[s] + i];
      c.table[static_cast<size_t>(s) * c.max_pages + s_first[s] + i] = id;
      c.refs[id] = 1;
    }
}

constexpr int kWriteThreads = 128;
constexpr int kWriteTokens = 64;  // tokens of a sequence a block
// Words of a copied page's K and V that a thread has in flight: 64 sequences of 16 layers with up to 8 new rows and 40 copied
// ones, 134 MB read and written: 1 25.5 us, 2 23.9, 4 23.8, 6 25.7.
constexpr int kCopyVecs = 2;

// Block (sequence and layer, group of heads, chunk of tokens): copies the shared page's rows, then a quad
// of threads writes the rows of one token and head (lane layout of common.cuh).
template <typename DT>
__global__ void __launch_bounds__(kWriteThreads) commit_write_kernel(const __grid_constant__ CommitArgs a, int heads) {
  wait_for_first();
  const CacheDev& c = a.c;
  const int b = blockIdx.x / c.L, l = blockIdx.x % c.L;
  const int h0 = blockIdx.y * heads, h1 = min(c.H, h0 + heads);
  const CommitJob job = a.jobs[b];
  const int i0 = blockIdx.z * kWriteTokens, i1 = min(job.n, i0 + kWriteTokens);
  DT* K = static_cast<DT*>(c.k);
  DT* V = static_cast<DT*>(c.v);
  const size_t layer = static_cast<size_t>(l) * c.n_pages;
  if (blockIdx.z == 0 && job.src >= 0) {
    const int vecs = (job.len & (c.P - 1)) * kD * static_cast<int>(sizeof(DT)) / 16;
    const size_t from = ((layer + job.src) * c.H + h0) * c.P * kD, to = ((layer + job.dst) * c.H + h0) * c.P * kD;
    const size_t step = static_cast<size_t>(c.P) * kD;
    for (int at = threadIdx.x; at < vecs * (h1 - h0); at += kWriteThreads * kCopyVecs) {
      uint4 kx[kCopyVecs], vx[kCopyVecs];
#pragma unroll
      for (int u = 0; u < kCopyVecs; ++u) {
        const int i = at + u * kWriteThreads, h = i / vecs, x = i % vecs;
        if (h >= h1 - h0) break;
        kx[u] = reinterpret_cast<const uint4*>(K + from + h * step)[x];
        vx[u] = reinterpret_cast<const uint4*>(V + from + h * step)[x];
      }
#pragma unroll
      for (int u = 0; u < kCopyVecs; ++u) {
        const int i = at + u * kWriteThreads, h = i / vecs, x = i % vecs;
        if (h >= h1 - h0) break;
        reinterpret_cast<uint4*>(K + to + h * step)[x] = kx[u];
        reinterpret_cast<uint4*>(V + to + h * step)[x] = vx[u];
      }
    }
  }
  const int t = threadIdx.x & 3;
  for (int item = threadIdx.x >> 2; item < (i1 - i0) * (h1 - h0); item += kWriteThreads / 4) {
    const int i = i0 + item / (h1 - h0), h = h0 + item % (h1 - h0);
    const int node = a.path != nullptr ? a.path[static_cast<size_t>(b) * a.T + i] : i;
    const int pos = job.len + i;
    const int page = c.table[static_cast<size_t>(b) * c.max_pages + (pos >> c.shift)];
    const size_t from = (((static_cast<size_t>(l) * a.B + b) * c.H + h) * a.T + node) * kD;
    const size_t to = (((layer + page) * c.H + h) * c.P + (pos & (c.P - 1))) * kD;
    float x[16], y[16];
    load_part(static_cast<const DT*>(a.k_new) + from, t, x);
    load_part(static_cast<const DT*>(a.v_new) + from, t, y);
    float2 e[8];
    rope_row(a.rope_lo, a.rope_hi, pos, t, e);
    rotate_part(x, e, false);
    store_part(K + to, t, x);
    store_part(V + to, t, y);
  }
}

// --------------------------------------------------------------------------------- fork --
struct ForkArgs {
  CacheDev c;
  const int32_t* src;
  int32_t* rows;  // [S, max_pages]: what the sequences' rows become
  int32_t* lens;  // [S]; -1: the whole call is refused
};

__device__ __forceinline__ int pages_of(const CacheDev& c, int len) { return (len + c.P - 1) >> c.shift; }

// Whether the call is refused (the same in every block).
__device__ __forceinline__ bool fork_refused(const ForkArgs& a) {
  const CacheDev& c = a.c;
  bool bad = false;
  for (int i = threadIdx.x; i < c.S; i += blockDim.x) {
    const int s = a.src[i], len = c.lens[i];
    bad |= s < -1 || s >= c.S || len < 0 || len > static_cast<long long>(c.max_pages) * c.P;
  }
  return __syncthreads_or(bad);
}

// Sequence b, by `threads` threads of number t: the new row into the workspace, +1 for each page it holds now, -1
// for each that it held.  Sums of integers: the order does not matter.
__device__ __forceinline__ void fork_count(const ForkArgs& a, int b, int t, int threads) {
  const CacheDev& c = a.c;
  const int s = a.src[b];
  const int len = s < 0 ? 0 : c.lens[s];
  if (t == 0) a.lens[b] = len;
  if (s == b) return;
  const int now = pages_of(c, len), old = pages_of(c, c.lens[b]);
  const int32_t* from = c.table + static_cast<size_t>(max(s, 0)) * c.max_pages;
  const int32_t* mine = c.table + static_cast<size_t>(b) * c.max_pages;
  for (int j = t; j < max(now, old); j += threads) {
    const int in = j < now ? from[j] : 0, out = j < old ? mine[j] : 0;
    if (j < now) {
      a.rows[static_cast<size_t>(b) * c.max_pages + j] = in;
      if (in >= 0 && in < c.n_pages)
        atomicAdd(&c.refs[in], 1);
      else
        c.state[kStateStatus] = kStatusDeviceAssert;
    }
    if (j < old) {
      if (out >= 0 && out < c.n_pages)
        atomicSub(&c.refs[out], 1);
      else
        c.state[kStateStatus] = kStatusDeviceAssert;
    }
  }
}

// Then its row into the table; returns the lowest of its old pages that has lost its last holder.  Its length is
// the caller's to write, when all its threads are past this.
__device__ __forceinline__ int fork_write(const ForkArgs& a, int b, int t, int threads) {
  const CacheDev& c = a.c;
  int lowest = c.n_pages;
  if (a.src[b] == b) return lowest;
  const int now = pages_of(c, __ldcg(a.lens + b)), old = pages_of(c, c.lens[b]);
  for (int j = t; j < max(now, old); j += threads) {
    int32_t* e = c.table + static_cast<size_t>(b) * c.max_pages + j;
    if (j < old) {
      const int page = *e;
      if (page >= 0 && page < c.n_pages && __ldcg(c.refs + page) == 0) lowest = min(lowest, page);
    }
    *e = j < now ? __ldcg(a.rows + static_cast<size_t>(b) * c.max_pages + j) : -1;
  }
  return lowest;
}

// Small tables: both halves in one launch, by one cluster of blocks; a warp a sequence.
constexpr int kForkCluster = 8;
constexpr int kForkWarps = 16;

__global__ void __launch_bounds__(32 * kForkWarps) fork_cluster_kernel(const __grid_constant__ ForkArgs a) {
  const CacheDev& c = a.c;
  if (fork_refused(a)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) c.state[kStateStatus] = kStatusDeviceAssert;
    return;  // (every block of the cluster)
  }
  const int first = blockIdx.x * kForkWarps + (threadIdx.x >> 5), step = gridDim.x * kForkWarps, lane = threadIdx.x & 31;
  for (int b = first; b < c.S; b += step) fork_count(a, b, lane, 32);
  __threadfence();
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  int lowest = c.n_pages;
  for (int b = first; b < c.S; b += step) {
    lowest = min(lowest, fork_write(a, b, lane, 32));
    __syncwarp();  // every lane has read the old length
    if (lane == 0) c.lens[b] = __ldcg(a.lens + b);
  }
  lowest = __reduce_min_sync(0xffffffffu, lowest);
  if (lane == 0 && lowest < c.n_pages) atomicMin(&c.state[kStateCursor], lowest);
}

// Large ones: a block a sequence, the second half in a launch of its own.
constexpr int kForkThreads = 256;

__global__ void __launch_bounds__(kForkThreads) fork_count_kernel(const __grid_constant__ ForkArgs a) {
  let_second_start();
  const int b = blockIdx.x;
  if (fork_refused(a)) {
    if (threadIdx.x == 0) {
      a.lens[b] = -1;
      if (b == 0) a.c.state[kStateStatus] = kStatusDeviceAssert;
    }
    return;
  }
  fork_count(a, b, threadIdx.x, kForkThreads);
}

__global__ void __launch_bounds__(kForkThreads) fork_write_kernel(const __grid_constant__ ForkArgs a) {
  wait_for_first();
  const CacheDev& c = a.c;
  const int b = blockIdx.x, len = a.lens[b];
  if (len < 0) return;
  const int lowest = fork_write(a, b, threadIdx.x, kForkThreads);
  if (lowest < c.n_pages) atomicMin(&c.state[kStateCursor], lowest);
  __syncthreads();  // every thread has read the old length
  if (threadIdx.x == 0) c.lens[b] = len;
}

// ------------------------------------------------------------------------------ compact --
struct CompactArgs {
  CacheDev c;
  int32_t* remap;
  int32_t* moves;  // number of moves
  int32_t* src;
  int32_t* dst;
};

// One block: counts the used pages (n), then lists the free ones below n and the used ones
// from n on; the i-th of these moves into the i-th of those.  4096 counts a step; those of the first step, all
// of a pool of up to 4096 pages, are read once.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ int s_sums[33];
  let_second_start();
  const CacheDev& c = a.c;
  constexpr int kStep = 4 * kPlanThreads;
  const int t4 = 4 * static_cast<int>(threadIdx.x);
  int head[4];
  load_counts(c, t4, head);
  int mine = (head[0] > 0) + (head[1] > 0) + (head[2] > 0) + (head[3] > 0);
  for (int base = kStep; base < c.n_pages; base += kStep) {
    int r[4];
    load_counts(c, base + t4, r);
    mine += (r[0] > 0) + (r[1] > 0) + (r[2] > 0) + (r[3] > 0);
  }
  int live;
  block_scan_1024(mine, s_sums, &live);
  int holes = 0, moved = 0;
  for (int base = 0; base < c.n_pages; base += kStep) {
    int r[4] = {head[0], head[1], head[2], head[3]};
    if (base > 0) load_counts(c, base + t4, r);
    // holes in the lower half of the sum, movers in the upper (4096 of each at most)
    int both = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int id = base + t4 + u;
      if (id < c.n_pages) both += r[u] > 0 ? (id >= live ? 1 << 16 : 0) : (id < live ? 1 : 0);
    }
    int total;
    const int at = block_scan_1024(both, s_sums, &total);
    int at_hole = holes + (at & 0xffff), at_out = moved + (at >> 16);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int id = base + t4 + u;
      if (id < live && id < c.n_pages && r[u] <= 0) a.dst[at_hole++] = id;
    }
    __syncthreads();
    // every hole lies below `live`, so as many as the movers so far are listed by now
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int id = base + t4 + u;
      if (id >= c.n_pages) break;
      int to = r[u] > 0 ? id : -1;
      if (r[u] > 0 && id >= live) {
        to = a.dst[at_out];
        a.src[at_out++] = id;
      }
      a.remap[id] = to;
    }
    holes += total & 0xffff;
    moved += total >> 16;
  }
  if (threadIdx.x == 0) {
    *a.moves = moved;
    c.state[kStateLive] = live;
    c.state[kStateCursor] = live;
  }
}

constexpr int kMoveThreads = 256;
// 16-byte words a thread has in flight.  Half of 1024 pages of 16 layers, 1.07 GB read and written: 4 182 us, 8 171, 16 168
// (6.4 TB/s).
constexpr int kMoveVecs = 16;

__global__ void __launch_bounds__(kMoveThreads) compact_move_kernel(const __grid_constant__ CompactArgs a, int page_vecs) {
  wait_for_first();
  const CacheDev& c = a.c;
  const int moves = *a.moves;
  if (moves == 0) return;
  // tables
  for (int b = blockIdx.x; b < c.S; b += gridDim.x) {
    const int len = c.lens[b];
    const int held = len < 0 ? 0 : min(pages_of(c, len), c.max_pages);
    for (int j = threadIdx.x; j < held; j += kMoveThreads) {
      int32_t* e = c.table + static_cast<size_t>(b) * c.max_pages + j;
      const int page = *e;
      if (page >= 0 && page < c.n_pages) *e = a.remap[page];
      else c.state[kStateStatus] = kStatusDeviceAssert;
    }
  }
  for (int m = blockIdx.x * kMoveThreads + threadIdx.x; m < moves; m += gridDim.x * kMoveThreads) {
    const int from = a.src[m];
    c.refs[a.dst[m]] = c.refs[from];
    c.refs[from] = 0;
  }
  // rows: units of kMoveThreads * kMoveVecs 16-byte words of one page of one layer's K or V
  const int per = (page_vecs + kMoveThreads * kMoveVecs - 1) / (kMoveThreads * kMoveVecs);
  const long long units = static_cast<long long>(moves) * c.L * 2 * per;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int piece = static_cast<int>(u % per);
    const long long w = u / per;
    const int m = static_cast<int>(w / (2 * c.L)), s = static_cast<int>(w % (2 * c.L));
    uint4* pool = static_cast<uint4*>(s & 1 ? c.v : c.k);
    const size_t layer = static_cast<size_t>(s >> 1) * c.n_pages;
    const uint4* from = pool + (layer + a.src[m]) * page_vecs;
    uint4* to = pool + (layer + a.dst[m]) * page_vecs;
    uint4 x[kMoveVecs];
#pragma unroll
    for (int v = 0; v < kMoveVecs; ++v) {
      const int at = (piece * kMoveVecs + v) * kMoveThreads + threadIdx.x;
      if (at < page_vecs) x[v] = from[at];
    }
#pragma unroll
    for (int v = 0; v < kMoveVecs; ++v) {
      const int at = (piece * kMoveVecs + v) * kMoveThreads + threadIdx.x;
      if (at < page_vecs) to[at] = x[v];
    }
  }
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// commit: jobs and the pages taken (n_pages at most); fork: rows and lengths; compact: a count
// and two lists of n_pages.
size_t cache_workspace_bytes(const fib_attn_cache& c) {
  const size_t pages = round_up(sizeof(int32_t) * static_cast<size_t>(c.n_pages));
  const size_t commit = round_up(sizeof(CommitJob) * kMaxSeqs) + pages;
  const size_t fork = round_up(sizeof(int32_t) * kMaxSeqs) +
                      round_up(sizeof(int32_t) * static_cast<size_t>(c.max_seqs) * static_cast<size_t>(c.max_pages));
  const size_t compact = 256 + 2 * pages;
  size_t m = commit > fork ? commit : fork;
  return m > compact ? m : compact;
}

cudaError_t launch_cache_commit(const fib_attn_cache& cache, int B, int T, int n_max, const int32_t* n_new,
                                const int32_t* path, const void* k_new, const void* v_new, const float2* lo_tab,
                                const float2* hi_tab, void* ws, cudaStream_t stream) {
  CommitArgs a;
  a.c = device_view(cache);
  a.B = B;
  a.T = T;
  a.n_max = n_max;
  a.n_new = n_new;
  a.path = path;
  a.k_new = k_new;
  a.v_new = v_new;
  a.rope_lo = lo_tab;
  a.rope_hi = hi_tab;
  a.jobs = static_cast<CommitJob*>(ws);
  a.list = reinterpret_cast<int32_t*>(static_cast<unsigned char*>(ws) + round_up(sizeof(CommitJob) * kMaxSeqs));
  commit_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // heads a block: so many that a block's 32 quads all have a row of its tokens
  const int tokens = T < kWriteTokens ? T : kWriteTokens;
  int heads = kWriteThreads / 4 / tokens;
  heads = heads < 1 ? 1 : heads > cache.heads ? cache.heads : heads;
  const dim3 grid(static_cast<unsigned>(B) * cache.n_layers, (cache.heads + heads - 1) / heads,
                  (T + kWriteTokens - 1) / kWriteTokens);
  return cache.dtype == FIB_DTYPE_F32
             ? launch_second(commit_write_kernel<float>, grid, kWriteThreads, stream, a, heads)
             : launch_second(commit_write_kernel<__nv_bfloat16>, grid, kWriteThreads, stream, a, heads);
}

cudaError_t launch_cache_fork(const fib_attn_cache& cache, const int32_t* src, void* ws, cudaStream_t stream) {
  ForkArgs a;
  a.c = device_view(cache);
  a.src = src;
  a.lens = static_cast<int32_t*>(ws);
  a.rows = reinterpret_cast<int32_t*>(static_cast<unsigned char*>(ws) + round_up(sizeof(int32_t) * kMaxSeqs));
  // One launch while the table is small.  32 x 64 entries: 12.3 us a call among others, 15.9 us in two (7.3 and 5.8 us in
  // a graph, where launches cost little); 256 x 512: 51 us by one cluster, 7.6 us in two.
  if (static_cast<long long>(cache.max_seqs) * cache.max_pages <= 1 << 13) {
    const int blocks = (cache.max_seqs + kForkWarps - 1) / kForkWarps;
    int size = 1;
    while (size < blocks && size < kForkCluster) size *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(size));
    cfg.blockDim = dim3(32 * kForkWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(size);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fork_cluster_kernel, a);
  }
  fork_count_kernel<<<cache.max_seqs, kForkThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_second(fork_write_kernel, dim3(static_cast<unsigned>(cache.max_seqs)), kForkThreads, stream, a);
}

cudaError_t launch_cache_compact(const fib_attn_cache& cache, int32_t* remap, void* ws, cudaStream_t stream) {
  CompactArgs a;
  a.c = device_view(cache);
  a.remap = remap;
  a.moves = static_cast<int32_t*>(ws);
  a.src = reinterpret_cast<int32_t*>(static_cast<unsigned char*>(ws) + 256);
  a.dst = reinterpret_cast<int32_t*>(static_cast<unsigned char*>(ws) + 256 +
                                     round_up(sizeof(int32_t) * static_cast<size_t>(cache.n_pages)));
  compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int row_vecs = kD * (cache.dtype == FIB_DTYPE_F32 ? 4 : 2) / 16;
  const int page_vecs = cache.heads * cache.page_rows * row_vecs;
  return launch_second(compact_move_kernel, dim3(152 * 8), kMoveThreads, stream, a, page_vecs);
}

}  // namespace fibattn
