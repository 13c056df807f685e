// Eviction from the paged cache by accumulated attention weight (sm_103a).
//
// Of a sequence's rows the first, the last and, of those between, the heaviest stay, for each layer and key head by itself; they move
// down in order, K turned from its old place to the new one (e^{-i (old - new) theta} a pair; a plan that does not rotate moves
// it as it is).  Three launches in a chain, each a programmatic dependent of the one before:
//   plan    one block: what each sequence keeps, the free pages that take the place of shared ones, tables, counts, lengths;
//   select  a block a sequence, layer and head: the weight of the last row that stays, by three passes over the weights' bits (11, 11,
//           10), then the list of rows that stay, in order; the weights move here;
//   move    a block for K and one for V: a row never moves up, so the rows that a step writes were all read in it or before, and one
//           barrier a step, between its reads and its writes, keeps them apart.  No order of blocks matters.
// What bounds it: the rows' bytes, read and written once.
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
  bool turns;
  EvictJob* jobs;
  int32_t* list;   // free pages taken
  int32_t* old;    // [S, max_pages]: the pages that a sequence held; ~page where a new one takes its place
  int32_t* stays;  // [L, S, H, rows]: the row that comes to place j
};

// ------------------------------------------------------------------------------------- plan --
// A thread a sequence for lengths and sums, a warp a sequence for its pages.
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
  if (!any_bad) {
    for (int s = warp; s < a.B; s += kPlanThreads / 32) {
      if (s_keep[s] < 0) continue;
      const int had = pages_of(c, s_len[s]), has = pages_of(c, s_keep[s]), same = min(a.sink >> c.shift, has);
      const int32_t* row = c.table + static_cast<size_t>(s) * c.max_pages;
      int32_t* old = a.old + static_cast<size_t>(s) * c.max_pages;
      int shared = 0;
#pragma unroll 4
      for (int j = lane; j < had; j += 32) {
        const int page = row[j];
        const bool in = page >= 0 && page < c.n_pages;
        bad |= !in;
        const bool taken = in && j >= same && j < has && c.refs[page] > 1;
        shared += taken;
        old[j] = taken ? ~page : page;
      }
      shared = __reduce_add_sync(0xffffffffu, shared);
      if (lane == 0) s_off[s] = shared;
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
  for (int s = warp; s < a.B; s += kPlanThreads / 32) {
    if (s_keep[s] < 0) continue;
    const int had = pages_of(c, s_len[s]), has = pages_of(c, s_keep[s]);
    int32_t* row = c.table + static_cast<size_t>(s) * c.max_pages;
    const int32_t* old = a.old + static_cast<size_t>(s) * c.max_pages;
    int at = s_off[s];
    for (int j0 = 0; j0 < had; j0 += 32) {
      const int j = j0 + lane, page = j < had ? old[j] : 0;  // (this lane wrote it)
      const bool taken = page < 0, gone = j < had && j >= has;
      const unsigned mask = __ballot_sync(0xffffffffu, taken);
      if (taken) {
        const int id = list[at + __popc(mask & ((1u << lane) - 1u))];
        row[j] = id;
        c.refs[id] = 1;
      }
      if (gone) row[j] = -1;
      if (taken || gone) {
        const int left = taken ? ~page : page;
        if (atomicSub(&c.refs[left], 1) == 1) lowest = min(lowest, left);
      }
      at += __popc(mask);
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
constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32, kSelRows = 4;  // rows a thread and step
constexpr int kBins = 2048;

// Weights in ascending order as unsigned words: the two zeros alike, NaN below all.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Counts of `n` bins in `hist`: the highest bin with at least `need` keys in it and above; *above gets those above it.  The whole
// block; ends synchronised.
__device__ __forceinline__ int find_bin(const int* hist, int n, int need, int* sums, int* s_out, int* above) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, each = n / kSelThreads;  // 4 or 2 bins a thread, from the highest down
  const int top = n - 1 - each * static_cast<int>(threadIdx.x);
  int own = 0;
  for (int i = 0; i < each; ++i) own += hist[top - i];
  int inc = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  int before = inc - own;
  for (int w = 0; w < warp; ++w) before += sums[w];
  if (before < need && before + own >= need) {  // one thread
    for (int i = 0; i < each; ++i) {
      const int x = hist[top - i];
      if (before + x >= need) {
        s_out[0] = top - i;
        s_out[1] = before;
        break;
      }
      before += x;
    }
  }
  __syncthreads();
  *above = s_out[1];
  return s_out[0];
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int s_hist[kBins];
  __shared__ int s_sums[kSelWarps * kSelRows + 1], s_out[2];
  let_second_start();
  wait_for_first();
  const CacheDev& c = a.c;
  const int per = c.L * c.H, b = blockIdx.x / per, lh = blockIdx.x % per, l = lh / c.H, h = lh % c.H;
  const EvictJob job = a.jobs[b];
  if (job.keep < 0) return;
  const size_t task = (static_cast<size_t>(l) * c.S + b) * c.H + h;
  float* w = a.weights + task * a.rows;
  int32_t* stays = a.stays + task * a.rows;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int end = job.len - a.recent, need = job.keep - a.sink - a.recent;  // rows [sink, end) compete for `need` places
  // the last row that stays among them: its key, and how many of the rows with that key stay (the first ones)
  uint32_t least = 0xffffffffu;  // (no row has it)
  int quota = 0;
  if (need > 0) {
    int left = need;
    uint32_t prefix = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
      for (int i = threadIdx.x; i < bins; i += kSelThreads) s_hist[i] = 0;
      __syncthreads();
#pragma unroll 8
      for (int r = a.sink + static_cast<int>(threadIdx.x); r < end; r += kSelThreads) {
        const uint32_t key = order_of(w[r]);
        if (pass == 0 || key >> (pass == 1 ? 21 : 10) == prefix) atomicAdd(&s_hist[(key >> shift) & (bins - 1)], 1);
      }
      __syncthreads();
      int above;
      const int bin = find_bin(s_hist, bins, left, s_sums, s_out, &above);
      prefix = pass == 0 ? bin : prefix << (pass == 1 ? 11 : 10) | bin;
      left -= above;
      __syncthreads();
    }
    least = prefix;
    quota = left;
  }
  // The list.  What stays before a row: the rows that stay for certain, and of those with the least key the first ones.  Both counts
  // in one word: 2048 rows a step.
  int sure = 0, ties = 0;  // of the steps before
  for (int r0 = 0; r0 < job.len; r0 += kSelThreads * kSelRows) {
    float x[kSelRows];
    unsigned sure_mask[kSelRows], tie_mask[kSelRows];
#pragma unroll
    for (int i = 0; i < kSelRows; ++i) {
      const int r = r0 + i * kSelThreads + threadIdx.x;
      x[i] = r < job.len ? w[r] : 0.f;
      const uint32_t key = order_of(x[i]);
      const bool edge = r < a.sink || (r >= end && r < job.len), mid = r >= a.sink && r < end && need > 0;
      sure_mask[i] = __ballot_sync(0xffffffffu, edge || (mid && key > least));
      tie_mask[i] = __ballot_sync(0xffffffffu, mid && key == least);
      if (lane == 0) s_sums[i * kSelWarps + warp] = __popc(sure_mask[i]) | __popc(tie_mask[i]) << 16;
    }
    __syncthreads();  // (and every weight of the step has been read)
    if (warp == 0) {  // exclusive sums of the 64 words
      const int x0 = s_sums[2 * lane], x1 = s_sums[2 * lane + 1];
      int inc = x0 + x1;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
      }
      s_sums[2 * lane] = inc - x0 - x1;
      s_sums[2 * lane + 1] = inc - x1;
      if (lane == 31) s_sums[64] = inc;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSelRows; ++i) {
      const int r = r0 + i * kSelThreads + threadIdx.x, word = s_sums[i * kSelWarps + warp];
      const unsigned below = (1u << lane) - 1u;
      const int sures = sure + (word & 0xffff) + __popc(sure_mask[i] & below), tied = ties + (word >> 16) + __popc(tie_mask[i] & below);
      const bool tie = tie_mask[i] >> lane & 1;
      if ((sure_mask[i] >> lane & 1) || (tie && tied < quota)) {
        const int at = sures + min(tied, quota);
        stays[at] = r;
        if (at != r) w[at] = x[i];
      }
    }
    const int all = s_sums[64];
    sure += all & 0xffff;
    ties += all >> 16;
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------------- move --
constexpr int kMoveThreads = 512;

// A quad a row, each thread dims 8t .. and 32+8t .. of it: two 16-byte words of bf16, four of float32.
template <typename DT, int ROWS>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int kWords = static_cast<int>(sizeof(DT)), kHalf = kWords / 2;  // 16-byte words a thread and row
  constexpr int kStep = kMoveThreads / 4 * ROWS;
  wait_for_first();
  const CacheDev& c = a.c;
  const int v = blockIdx.x & 1, per = c.L * c.H, task = blockIdx.x >> 1, b = task / per, lh = task % per, l = lh / c.H, h = lh % c.H;
  const EvictJob job = a.jobs[b];
  if (job.keep < 0) return;
  const int32_t* stays = a.stays + ((static_cast<size_t>(l) * c.S + b) * c.H + h) * a.rows;
  const int32_t* old = a.old + static_cast<size_t>(b) * c.max_pages;
  const int32_t* now = c.table + static_cast<size_t>(b) * c.max_pages;
  DT* pool = static_cast<DT*>(v ? c.v : c.k) + ((static_cast<size_t>(l) * c.n_pages * c.H + h) << c.shift) * kD;
  const size_t page_elems = (static_cast<size_t>(c.H) << c.shift) * kD;
  const int t = threadIdx.x & 3, quad = threadIdx.x >> 2, mask = c.P - 1;
  for (int j0 = job.same << c.shift; j0 < job.keep; j0 += kStep) {
    uint4 x[ROWS][kWords];
    int src[ROWS];
    bool moves[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int j = j0 + i * (kMoveThreads / 4) + quad;
      src[i] = j < job.keep ? stays[j] : -1;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int j = j0 + i * (kMoveThreads / 4) + quad;
      moves[i] = false;
      if (src[i] >= 0) {
        const int page = old[src[i] >> c.shift];
        moves[i] = src[i] != j || page < 0;
        if (moves[i]) {
          const uint4* p = reinterpret_cast<const uint4*>(pool + (page < 0 ? ~page : page) * page_elems + static_cast<size_t>(src[i] & mask) * kD);
#pragma unroll
          for (int k = 0; k < kWords; ++k) x[i][k] = p[(k / kHalf) * 4 * kHalf + t * kHalf + k % kHalf];
        }
      }
    }
    __syncthreads();  // every row of the step has been read
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int j = j0 + i * (kMoveThreads / 4) + quad;
      if (!moves[i]) continue;
      if (v == 0 && a.turns && src[i] != j) {
        float2 e[8];
        float y[16];
        rope_row(a.rope_lo, a.rope_hi, src[i] - j, t, e);
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

size_t rows_bytes(const fib_attn_cache& c, int rows) {
  return round_up(sizeof(int32_t) * static_cast<size_t>(c.n_layers) * c.max_seqs * c.heads * static_cast<size_t>(rows));
}
size_t tables_bytes(const fib_attn_cache& c) {
  return round_up(sizeof(int32_t) * static_cast<size_t>(c.max_seqs) * static_cast<size_t>(c.max_pages));
}

}  // namespace

// jobs, the free pages taken, the old tables, the rows that stay
size_t cache_evict_workspace_bytes(const fib_attn_cache& c, int rows) {
  return round_up(sizeof(EvictJob) * kMaxSeqs) + round_up(sizeof(int32_t) * static_cast<size_t>(c.n_pages)) + tables_bytes(c) + rows_bytes(c, rows);
}

cudaError_t launch_cache_evict(const fib_attn_cache& cache, int B, int rows, const int32_t* keep, int sink, int recent, int n_max,
                               float* weights, int32_t* dropped, const float2* lo_tab, const float2* hi_tab, bool turns, void* ws,
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
  a.turns = turns;
  unsigned char* at = static_cast<unsigned char*>(ws);
  a.jobs = reinterpret_cast<EvictJob*>(at);
  at += round_up(sizeof(EvictJob) * kMaxSeqs);
  a.list = reinterpret_cast<int32_t*>(at);
  at += round_up(sizeof(int32_t) * static_cast<size_t>(cache.n_pages));
  a.old = reinterpret_cast<int32_t*>(at);
  at += tables_bytes(cache);
  a.stays = reinterpret_cast<int32_t*>(at);
  evict_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned tasks = static_cast<unsigned>(B) * cache.n_layers * cache.heads;
  e = launch_second(evict_select_kernel, dim3(tasks), kSelThreads, stream, a);
  if (e != cudaSuccess) return e;
  return cache.dtype == FIB_DTYPE_F32 ? launch_second(evict_move_kernel<float, 2>, dim3(2 * tasks), kMoveThreads, stream, a)
                                      : launch_second(evict_move_kernel<__nv_bfloat16, 4>, dim3(2 * tasks), kMoveThreads, stream, a);
}

}  // namespace fibattn
