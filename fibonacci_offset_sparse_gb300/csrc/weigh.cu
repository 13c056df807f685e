// The attention weight that new tokens give to each row of the paged cache, added up (sm_103a):
//   weights[r] = (r < first ? weights[r] : 0) + sum over query rows m with r <= p_m of exp(q'_m . K_r / 8 - lse_m).
// A row's sum needs no other row once lse is known, so a row belongs to one warp (or one thread, weigh_tc.cu): no partials, no atomics,
// one order of sums.  Two launches: the queries rotated, scaled and split once; then one pass over K.
//
// What bounds it: the read of K.  Here, for up to 8 query rows a key head (and float32 of any number): keys as the 16 rows of
// mma.sync's tile, queries as its 8 columns.  A warp has units of 4 KB of K to itself and a ring of three of them in shared memory, filled by
// bulk copies, so 16 warps have 192 KB an SM on their way and no warp waits for another.  A lane's 16-byte words are the tile's fragments
// (the order of the dims is the same for both).  A token of 32 sequences of up to 2048 rows, 16 layers, 8 heads, bf16 (792 MB): 141 us with
// the queries' 6 (5.6 TB/s, 83% of a measured copy); loads straight to registers took 172.  In float32 (1538 MB), of one token or of eight: 277 us (5.6 TB/s).
// Precision: scores are float32.  The query is split in three bf16 (24 bits; cached bf16 rows enter as stored), float32 query and
// rows each in two tf32 to nearest (22 bits); the small parts are added up first, as the pipes round toward zero.
#include "weigh.cuh"

namespace fibattn {

namespace {

// ------------------------------------------------------------------------------------- queries --
constexpr int kPrepThreads = 128, kPrepHeads = 4;

__device__ __forceinline__ float tf32_of(float x) {
  uint32_t y;
  asm("cvt.rna.tf32.f32 %0, %1;\n" : "=r"(y) : "f"(x));
  return __uint_as_float(y);
}

// A quad a query row (of mpad, those behind the last one as 0) of HEADS key heads, whose factors are the same and whose loads go side by side: block
// (layer and sequence, 32 rows of its heads after one another).
template <typename DT, int HEADS>
__global__ void __launch_bounds__(kPrepThreads) weigh_prep_kernel(const __grid_constant__ WeighArgs a) {
  let_second_start();
  const int t = threadIdx.x & 3, l = blockIdx.x / a.B, b = blockIdx.x % a.B;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.next = 0;
  bool ok;
  const WeighSeq s = weigh_seq(a, b, &ok);
  if (!ok && threadIdx.x == 0) atomicExch(a.status, kStatusDeviceAssert);
  if (s.n == 0) return;
  const int used = s.n * a.G, most = (used + 63) / 64 * 64;  // (no tile reaches behind these)
  const long long rows = static_cast<long long>((a.c.H + HEADS - 1) / HEADS) * a.mpad, step = static_cast<long long>(gridDim.y) * (kPrepThreads / 4);
  for (long long item = static_cast<long long>(blockIdx.y) * (kPrepThreads / 4) + (threadIdx.x >> 2); item < rows; item += step) {
    const int h0 = static_cast<int>(item / a.mpad) * HEADS, m = static_cast<int>(item % a.mpad), r = m & 7;
    if (m >= most) continue;
    const int i = m / a.G, g = m - i * a.G;
    int node = i;
    bool live = m < used;
    if (live && a.path != nullptr) {
      node = a.path[static_cast<size_t>(b) * a.T + i];
      if (node < 0 || node >= a.T) {
        live = false;
        atomicExch(a.status, kStatusDeviceAssert);
      }
    }
    float values[HEADS][16], refs[HEADS];
    float2 e[8];
    if (live) {
#pragma unroll
      for (int k = 0; k < HEADS; ++k) {
        const int h = min(h0 + k, a.c.H - 1);
        const size_t row = ((static_cast<size_t>(l) * a.B + b) * a.Hq + h * a.G + g) * a.T + node;
        load_part(static_cast<const DT*>(a.q) + row * kD, t, values[k]);
        refs[k] = -a.lse[row] * kLog2e;
      }
      rope_row(a.rope_lo, a.rope_hi, s.len - s.n + i, t, e);
    }
#pragma unroll
    for (int k = 0; k < HEADS; ++k) {
      const int h = h0 + k;
      if (h >= a.c.H) break;
      const size_t task = (static_cast<size_t>(l) * a.B + b) * a.c.H + h;
      float(&x)[16] = values[k];
      float ref = -INFINITY;
      if (live) {
        rotate_part(x, e, false);
        ref = refs[k];
#pragma unroll
        for (int u = 0; u < 16; ++u) x[u] *= kLog2e / 8.0f;
      } else {
#pragma unroll
        for (int u = 0; u < 16; ++u) x[u] = 0.f;
      }
      if (t == 0) a.refs[task * a.mpad + m] = ref;
      if constexpr (sizeof(DT) == 2) {
        if (t < 2) {  // an infinite one has no rest
          const float hi = __bfloat162float(__float2bfloat16_rn(ref)), left = isfinite(hi) ? ref - hi : 0.f;
          const float mid = __bfloat162float(__float2bfloat16_rn(left));
          const size_t group = task * (a.mpad / 8) + m / 8;
          if (a.G * a.T > kSpreadRows) {
            *reinterpret_cast<uint4*>(a.ref_parts + group * kRefGroupBytes + t * 128 + r * 16) =
                t == 0 ? make_uint4(pack_bf2_rn(hi, mid), pack_bf2_rn(left - mid, 0.f), 0, 0) : make_uint4(0, 0, 0, 0);
          } else {
            const float parts[3] = {hi, mid, left - mid};
#pragma unroll
            for (int part = 0; part < 3; ++part)
              *reinterpret_cast<uint4*>(a.ref_parts + (group * 3 + part) * kRefGroupBytes + t * 128 + r * 16) =
                  make_uint4(t == 0 ? pack_bf2_rn(parts[part], 0.f) : 0, 0, 0, 0);
          }
        }
        unsigned char* at = a.parts + (task * (a.mpad / 8) + m / 8) * kGroupBytes + r * 128;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          uint32_t w[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            w[u] = pack_bf2_rn(x[2 * u], x[2 * u + 1]);
            x[2 * u] -= bf_lo(w[u]);
            x[2 * u + 1] -= bf_hi(w[u]);
          }
          *reinterpret_cast<uint4*>(at + part * kPartBytes + ((t ^ r) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(at + part * kPartBytes + (((t + 4) ^ r) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
        }
      } else {
        float* at = reinterpret_cast<float*>(a.parts + (task * (a.mpad / 8) + m / 8) * kGroupBytes32) + r * kD;
        float hi[16], lo[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          hi[u] = tf32_of(x[u]);
          lo[u] = tf32_of(x[u] - hi[u]);
        }
        store_part(at, t, hi);
        store_part(at + 8 * kD, t, lo);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------- rows --
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kUnitBytes = 4096, kSlots = 3;  // of a warp's ring

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's fragments.  Lane (g, t) = (lane / 4, lane % 4).
// kOne: 8 query rows at most, whose fragments stay in registers; kFew: 2 at most, whose parts are columns of one product; kMany, kTeam: any
// number, which pass by the unit's rows, split once, the next eight on their way while eight are used (one block of 8 warps an SM for the
// registers; float32, 32 tokens over 2 sequences of 3149 rows, 16 layers, 8 heads: 57 us; rows split for each eight, 16 warps an SM, 71); with kTeam
// several warps share a unit where there are few (a prompt of 328, 5 layers, 3 heads, 6 of queries: 24 us, one warp a unit 39; its barrier
// costs the 32 tokens 3 us).
enum Rows { kFew, kOne, kMany, kTeam };
template <typename DT, Rows ROWS>
struct Frag;
template <Rows ROWS>
struct Frag<__nv_bfloat16, ROWS> {
  static constexpr int kTiles = 2, kWords = 2;  // 16-byte words of a row that a lane holds: dims 8t .., 32+8t ..
  static constexpr int kGroup = kGroupBytes, kPer = 2;  // queries of a lane's scores
  uint4 q[3][2];
  __device__ __forceinline__ static int word(int t, int k) { return t + 4 * k; }
  __device__ __forceinline__ void load(const unsigned char* group, int g, int t) {
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
      for (int k = 0; k < 2; ++k) q[p][k] = *reinterpret_cast<const uint4*>(group + p * kPartBytes + g * 128 + ((word(t, k) ^ g) << 4));
  }
  __device__ __forceinline__ static int query(int t, int j) { return 2 * t + j; }
  __device__ __forceinline__ static float add_up(float x) { return quad_sum(x); }  // over a quad's queries
  // Scores of 16 rows (x0: row g, x1: row g + 8) and 8 queries, y[row][query]; upper: of the queries' upper part alone.
  __device__ __forceinline__ void scores(const uint4 (&x0)[2], const uint4 (&x1)[2], float (&y)[2][2], bool upper) const {
    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 2; p >= 0; --p) {
      if (upper && p > 0) continue;
      mma_bf16(c, x0[0].x, x1[0].x, x0[1].x, x1[1].x, q[p][0].x, q[p][1].x);
      mma_bf16(c, x0[0].y, x1[0].y, x0[1].y, x1[1].y, q[p][0].y, q[p][1].y);
      mma_bf16(c, x0[0].z, x1[0].z, x0[1].z, x1[1].z, q[p][0].z, q[p][1].z);
      mma_bf16(c, x0[0].w, x1[0].w, x0[1].w, x1[1].w, q[p][0].w, q[p][1].w);
    }
    y[0][0] = c[0]; y[0][1] = c[1]; y[1][0] = c[2]; y[1][1] = c[3];
  }
};
// Columns 0, 1, 2 of the product are the first query's hi, mid, lo, 4, 5, 6 the second's: a third of the products, and one score a row and
// lane (of query t / 2) where there are two.  The token above: 133 us without the queries' launch, as eight columns 141.
template <>
struct Frag<__nv_bfloat16, kFew> {
  static constexpr int kTiles = 2, kWords = 2;
  static constexpr int kGroup = kGroupBytes, kPer = 1;
  uint4 q[2];
  __device__ __forceinline__ static int word(int t, int k) { return t + 4 * k; }
  __device__ __forceinline__ void load(const unsigned char* group, int g, int t) {
    const int part = g & 3, row = g >> 2;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      q[k] = part < 3 ? *reinterpret_cast<const uint4*>(group + part * kPartBytes + row * 128 + ((word(t, k) ^ row) << 4)) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ static int query(int t, int) { return t >> 1; }
  __device__ __forceinline__ static float add_up(float x) { return x + __shfl_xor_sync(0xffffffffu, x, 2); }
  __device__ __forceinline__ void scores(const uint4 (&x0)[2], const uint4 (&x1)[2], float (&y)[2][1], bool upper) const {
    float c[4] = {0.f, 0.f, 0.f, 0.f};
    mma_bf16(c, x0[0].x, x1[0].x, x0[1].x, x1[1].x, q[0].x, q[1].x);
    mma_bf16(c, x0[0].y, x1[0].y, x0[1].y, x1[1].y, q[0].y, q[1].y);
    mma_bf16(c, x0[0].z, x1[0].z, x0[1].z, x1[1].z, q[0].z, q[1].z);
    mma_bf16(c, x0[0].w, x1[0].w, x0[1].w, x1[1].w, q[0].w, q[1].w);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float part = c[2 * e] + c[2 * e + 1];  // hi + mid, or lo + 0
      y[e][0] = upper ? __shfl_sync(0xffffffffu, c[2 * e], threadIdx.x & 30) : part + __shfl_xor_sync(0xffffffffu, part, 1);
    }
  }
};
template <Rows ROWS>
struct Frag<float, ROWS> {
  static constexpr int kTiles = 1, kWords = 4;  // dims 16k + 4t .., k = 0 .. 3
  static constexpr int kGroup = kGroupBytes32, kPer = 2;
  uint4 q[2][4];
  __device__ __forceinline__ static int word(int t, int k) { return t + 4 * k; }
  __device__ __forceinline__ void load(const unsigned char* group, int g, int t) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int k = 0; k < 4; ++k) q[p][k] = reinterpret_cast<const uint4*>(group)[(p * 8 + g) * 16 + word(t, k)];
  }
  __device__ __forceinline__ static int query(int t, int j) { return 2 * t + j; }
  __device__ __forceinline__ static float add_up(float x) { return quad_sum(x); }
  // Rows split: word k of both.
  struct Split {
    uint32_t h0[4], h1[4], l0[4], l1[4];
    __device__ __forceinline__ void set(const uint4& x0, const uint4& x1) {
      const uint32_t u0[4] = {x0.x, x0.y, x0.z, x0.w}, u1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f0 = __uint_as_float(u0[e]), f1 = __uint_as_float(u1[e]), g0 = tf32_of(f0), g1 = tf32_of(f1);
        h0[e] = __float_as_uint(g0);
        h1[e] = __float_as_uint(g1);
        l0[e] = __float_as_uint(tf32_of(f0 - g0));
        l1[e] = __float_as_uint(tf32_of(f1 - g1));
      }
    }
  };
  static constexpr bool kOnce = ROWS >= kMany;
  Split rows[kOnce ? 4 : 1];  // of many queries: all of them, once a unit
  __device__ __forceinline__ void take_rows(const uint4 (&x0)[4], const uint4 (&x1)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) rows[k].set(x0[k], x1[k]);
  }
  __device__ __forceinline__ void scores(const uint4 (&x0)[4], const uint4 (&x1)[4], float (&y)[2][2], bool upper) {
    float c[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
    float d[4] = {0.f, 0.f, 0.f, 0.f};  // the large products
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (!kOnce) rows[0].set(x0[k], x1[k]);
      const Split& r = rows[kOnce ? k : 0];
      const uint32_t qh[4] = {q[0][k].x, q[0][k].y, q[0][k].z, q[0][k].w}, ql[4] = {q[1][k].x, q[1][k].y, q[1][k].z, q[1][k].w};
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        if (!upper) {
          mma_tf32(c, r.l0[e], r.l1[e], r.l0[e + 1], r.l1[e + 1], qh[e], qh[e + 1]);
          mma_tf32(b, r.h0[e], r.h1[e], r.h0[e + 1], r.h1[e + 1], ql[e], ql[e + 1]);
        }
        mma_tf32(d, r.h0[e], r.h1[e], r.h0[e + 1], r.h1[e + 1], qh[e], qh[e + 1]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e >> 1][e & 1] = (c[e] + b[e]) + d[e];
  }
};

// A warp's units: a run of 4 KB pieces of K (32 rows of bf16, 16 of float32) of tasks (sequence, layer, head) after one another.
struct Cursor {
  long long u, end;  // the next task's first unit in the run; the run's end
  int i, last;       // the present task's next unit, and the one behind its last in the run
  int b, l, h;
  WeighSeq s;

  // Moves to the next unit, unit `i` of the task; false at the run's end.
  template <int UNIT>
  __device__ __forceinline__ bool next(const WeighArgs& a, const long long* start, bool* fresh) {
    *fresh = ++i >= last;
    if (!*fresh) return true;
    if (u >= end) return false;
    int lo = 0, hi = a.B;  // start[lo] <= u < start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= u)
        lo = mid;
      else
        hi = mid;
    }
    bool ok;
    b = lo;
    s = weigh_seq(a, b, &ok);
    const int units = (s.len + UNIT - 1) / UNIT;
    const long long off = u - start[b];
    const int lh = off < 1LL << 31 ? static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(units)) : static_cast<int>(off / units);
    l = lh / a.c.H;
    h = lh - l * a.c.H;
    i = static_cast<int>(off - static_cast<long long>(lh) * units);
    last = static_cast<int>(min(static_cast<long long>(units), i + (end - u)));
    u += last - i;
    return true;
  }
};

template <typename DT, Rows ROWS>
__global__ void __launch_bounds__(kThreads, ROWS >= kMany ? 1 : 2) weigh_kernel(const __grid_constant__ WeighArgs a) {
  using F = Frag<DT, ROWS>;
  constexpr bool ONE = ROWS < kMany;
  constexpr int TILES = F::kTiles, UNIT = 16 * TILES, ROW = kD * static_cast<int>(sizeof(DT));
  static_assert(UNIT * ROW == kUnitBytes, "a unit");
  extern __shared__ __align__(128) unsigned char s_ring[];  // [kWarps][kSlots][kUnitBytes]
  __shared__ uint64_t s_full[kWarps][kSlots];
  __shared__ float s_part[ROWS == kTeam ? 2 : 1][kWarps][16];  // what a team's warps have of a unit's rows
  __shared__ int s_there[kWarps][kSlots];  // bit x: box x of the slot's unit lies in the pool
  __shared__ long long s_start[kMaxSeqs + 1];  // units before each sequence's (of all layers and heads)
  const CacheDev& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  for (int b = threadIdx.x; b < a.B; b += kThreads) {
    bool ok;
    const WeighSeq s = weigh_seq(a, b, &ok);
    s_start[b] = s.n == 0 ? 0 : static_cast<long long>((s.len + UNIT - 1) / UNIT) * c.L * c.H;
  }
  if (threadIdx.x < kWarps * kSlots) mbar_init(&s_full[0][0] + threadIdx.x, 1);
  asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  __syncthreads();
  if (threadIdx.x < 32) {
    long long base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      const long long own = b < a.B ? s_start[b] : 0;
      long long x = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      if (b < a.B) s_start[b] = base + x - own;
      base += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) s_start[a.B] = base;
  }
  __syncthreads();
  // kTeam: where there are warps without a unit, 2, 4 or 8 of a block have each, and of its queries every second, fourth or eighth group.
  const long long total = s_start[a.B];
  int team = 1;
  if constexpr (ROWS == kTeam)
    while (team < kWarps && total * (2 * team) <= static_cast<long long>(gridDim.x) * kWarps) team *= 2;
  const int slice = warp % team;
  const long long warps = static_cast<long long>(gridDim.x) * (kWarps / team), w = (static_cast<long long>(blockIdx.x) * kWarps + warp) / team;
  const long long each = total / warps, rest = total % warps, first = w * each + min(w, rest);
  const Cursor begin{first, first + each + (w < rest ? 1 : 0), 0, 0, 0, 0, 0, {}};
  unsigned char* ring = s_ring + warp * kSlots * kUnitBytes;
  const int box = min(UNIT, c.P);  // rows a copy

  // Copies: lane x those of box x.  The page of the unit after the one that is copied is on its way.
  Cursor feed = begin;
  int page = 0, fed = 0;
  bool fresh, more = feed.next<UNIT>(a, s_start, &fresh);
  auto look = [&] {
    const int r = feed.i * UNIT + lane * box;
    page = more && lane * box < UNIT && r < feed.s.len ? __ldg(c.table + static_cast<size_t>(feed.b) * c.max_pages + (r >> c.shift)) : 0;
  };
  auto copy = [&] {
    if (!more) return;
    const int slot = fed % kSlots, r = feed.i * UNIT + lane * box;
    const bool mine = lane * box < UNIT && r < feed.s.len, ok = page >= 0 && page < c.n_pages;
    const unsigned there = __ballot_sync(0xffffffffu, mine && ok), boxes = __ballot_sync(0xffffffffu, mine);
    if (there != boxes && lane == 0) atomicExch(a.status, kStatusDeviceAssert);
    if (lane == 0) {
      s_there[warp][slot] = static_cast<int>(there);
      mbar_arrive_tx(&s_full[warp][slot], __popc(there) * box * ROW);
    }
    __syncwarp();
    if (mine && ok) {
      const long long row = (((static_cast<long long>(feed.l) * c.n_pages + page) * c.H + feed.h) << c.shift) + (r & (c.P - 1));
      bulk_g2s(ring + slot * kUnitBytes + lane * box * ROW, static_cast<const unsigned char*>(c.k) + row * ROW, box * ROW, &s_full[warp][slot]);
    }
    __syncwarp();
    ++fed;
    more = feed.next<UNIT>(a, s_start, &fresh);
    look();
  };
  look();
  for (int x = 0; x < kSlots; ++x) copy();
  wait_for_first();

  Cursor k = begin;
  F q;
  float ref[F::kPer];
  int sees[F::kPer];  // the last row that the lane's queries see
  const unsigned char* parts = nullptr;
  const float* refs = nullptr;
  float* out = nullptr;
  int used = 0, before = 0;  // query row m sees rows up to before + m / G
  auto take = [&](F& to, float (&to_ref)[F::kPer], int group) {
    to.load(parts + static_cast<size_t>(group) * F::kGroup, g, t);
#pragma unroll
    for (int j = 0; j < F::kPer; ++j) to_ref[j] = refs[group * 8 + F::query(t, j)];
  };
  bool lost = false;
  for (int n = 0; k.next<UNIT>(a, s_start, &fresh); ++n) {
    if (fresh) {
      const size_t task = (static_cast<size_t>(k.l) * a.B + k.b) * c.H + k.h;
      parts = a.parts + task * (a.mpad / 8) * F::kGroup;
      refs = a.refs + task * a.mpad;
      out = a.weights + ((static_cast<size_t>(k.l) * c.S + k.b) * c.H + k.h) * a.rows;
      used = k.s.n * a.G;
      before = k.s.len - k.s.n;
      if constexpr (ONE) {
        take(q, ref, 0);
#pragma unroll
        for (int j = 0; j < F::kPer; ++j) sees[j] = F::query(t, j) < used ? before + F::query(t, j) / a.G : -1;
      }
    }
    const int r0 = k.i * UNIT, slot = n % kSlots, row = r0 + 8 * t + g;  // the row that the lane writes (float32: of t < 2)
    const bool writes = 8 * t < UNIT && row < k.s.len && slice == 0;
    const float old = writes && row < k.s.first ? out[row] : 0.f;
    const bool landed = !lost && mbar_wait(&s_full[warp][slot], (n / kSlots) & 1, a.wait_ns);
    if (!__all_sync(0xffffffffu, landed)) {
      if (lane == 0) atomicExch(a.status, kStatusTimeout);
      if (team == 1) break;
      lost = true;  // the others wait for this warp's part all the same
    }
    const bool there = s_there[warp][slot] >> ((8 * t & (UNIT - 1)) / box) & 1;
    uint4 x[TILES][2][F::kWords];
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const unsigned char* at = ring + slot * kUnitBytes + (16 * i + 8 * e + g) * ROW;
        if constexpr (sizeof(DT) == 2) {
          lds_row_part(at, t, g & 1, x[i][e][0], x[i][e][1]);
        } else {
#pragma unroll
          for (int z = 0; z < F::kWords; ++z) x[i][e][z] = reinterpret_cast<const uint4*>(at)[F::word(t, z)];
        }
      }
    float sum[2 * TILES];
#pragma unroll
    for (int v = 0; v < 2 * TILES; ++v) sum[v] = 0.f;
    const int groups = (used + 7) / 8;
    int from[2 * TILES];  // the first query that sees row 8v + g
    if constexpr (!ONE) {
      q.take_rows(x[0][0], x[0][1]);
#pragma unroll
      for (int v = 0; v < 2 * TILES; ++v) from[v] = max(0, r0 + 8 * v + g - before) * a.G;
    }
    const int edge = max(0, r0 + UNIT - 1 - before) * a.G;  // the first that sees every row of the unit
    const int group0 = ONE ? 0 : max(0, r0 - before) * a.G / 8;
    F next;
    float next_ref[F::kPer];
    if constexpr (!ONE) take(next, next_ref, min(group0 + slice, groups - 1));
    for (int group = group0 + slice; group < groups; group += team) {
      if constexpr (!ONE) {  // the next queries are on their way while these are used
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int k = 0; k < 4; ++k) q.q[p][k] = next.q[p][k];
#pragma unroll
        for (int j = 0; j < F::kPer; ++j) ref[j] = next_ref[j];
        take(next, next_ref, min(group + team, groups - 1));
      }
      // whether every query that the product has room for is one, and sees every row of the unit
      const bool all = group * 8 + (ROWS == kFew ? 2 : 8) <= used && group * 8 >= edge;
      float part[2 * TILES];
      // A NaN may come of an infinite key, where the parts' products are infinities of opposite signs: the upper
      // part's alone keep the sign, and a second round takes them.
#pragma unroll 1
      for (int round = 0; round < 2; ++round) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
          float y[2][F::kPer];
          q.scores(x[i][0], x[i][1], y, false);
          if (round == 1) {
            float z[2][F::kPer];
            q.scores(x[i][0], x[i][1], z, true);
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int j = 0; j < F::kPer; ++j) y[e][j] = isnan(y[e][j]) ? z[e][j] : y[e][j];
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float given = 0.f;
#pragma unroll
            for (int j = 0; j < F::kPer; ++j) {
              const float p = ex2(y[e][j] + ref[j]);
              if constexpr (ONE)
                given += all || r0 + 16 * i + 8 * e + g <= sees[j] ? p : 0.f;
              else
                given += all || (group * 8 + F::query(t, j) < used && group * 8 + F::query(t, j) >= from[2 * i + e]) ? p : 0.f;
            }
            part[2 * i + e] = given;
            bad |= isnan(given);
          }
        }
        if (!__any_sync(0xffffffffu, bad)) break;
      }
#pragma unroll
      for (int v = 0; v < 2 * TILES; ++v) sum[v] += part[v];
    }
    // value v of a quad's four lanes, added up, is row 8v + g's; lane t takes that of value t
#pragma unroll
    for (int v = 0; v < 2 * TILES; ++v) sum[v] = F::add_up(sum[v]);
    float y = t == 0 ? sum[0] : sum[1];
    if constexpr (TILES == 2) y = t == 2 ? sum[2] : t == 3 ? sum[3] : y;
    if constexpr (ROWS == kTeam) {
      if (team > 1) {
        static_assert(TILES == 1, "a part: 16 rows");
        if (t < 2) s_part[n & 1][warp][8 * t + g] = y;
        asm volatile("barrier.cta.sync %0, %1;\n" ::"r"(1 + warp / team), "r"(32 * team) : "memory");
        for (int i = 1; i < team && writes; ++i) y += s_part[n & 1][warp + i][8 * t + g];
      }
    }
    if (writes && there) out[row] = old + y;
    __threadfence_block();  // the slot has been read
    __syncwarp();
    if (!lost) copy();  // (a slot whose rows have not come is not filled again)
  }
  // nothing may be in flight when the block ends
  for (int x = max(0, fed - kSlots); x < fed; ++x) mbar_wait(&s_full[warp][x % kSlots], (x / kSlots) & 1, kWeighDrainNs);
}

cudaError_t launch_rows(void (*kernel)(WeighArgs), const WeighArgs& a, int blocks, cudaStream_t stream) {
  constexpr size_t kRing = static_cast<size_t>(kWarps) * kSlots * kUnitBytes;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRing));
  return e == cudaSuccess ? launch_second(kernel, dim3(152 * blocks), kThreads, kRing, stream, a) : e;  // 152 SMs
}

template <typename DT>
cudaError_t launch(const WeighArgs& a, cudaStream_t stream) {
  // Several heads a thread where one would be more blocks than the device holds: prompts of 2048, 4 layers, 8 heads, 51.3 us in all, with two
  // heads 51.9, with one 53.6.
  const bool several = a.c.H > 1 && static_cast<long long>(a.c.L) * a.B * a.c.H * (a.mpad / (kPrepThreads / 4)) > 152 * 16;
  const int runs = several ? (a.c.H + kPrepHeads - 1) / kPrepHeads : a.c.H;
  const long long blocks = (static_cast<long long>(runs) * a.mpad + kPrepThreads / 4 - 1) / (kPrepThreads / 4);
  const dim3 grid(static_cast<unsigned>(a.c.L) * a.B, static_cast<unsigned>(blocks < 32768 ? blocks : 32768));
  if (several)
    weigh_prep_kernel<DT, kPrepHeads><<<grid, kPrepThreads, 0, stream>>>(a);
  else
    weigh_prep_kernel<DT, 1><<<grid, kPrepThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if constexpr (sizeof(DT) == 2) {
    if (a.G * a.T <= 2) return launch_rows(weigh_kernel<DT, kFew>, a, 2, stream);
    return a.G * a.T <= 8 ? launch_rows(weigh_kernel<DT, kOne>, a, 2, stream) : launch_weigh_tc(a, stream);
  } else {
    if (a.G * a.T <= 8) return launch_rows(weigh_kernel<DT, kOne>, a, 2, stream);
    return a.G * a.T <= 64 ? launch_rows(weigh_kernel<DT, kMany>, a, 1, stream) : launch_rows(weigh_kernel<DT, kTeam>, a, 1, stream);
  }
}

int padded(int rows) { return rows <= 8 ? 8 : (rows + 63) / 64 * 64; }

}  // namespace

size_t weigh_workspace_bytes(const fib_attn_cache& c, int B, int Hq, int T) {
  const int query_rows = Hq / c.heads * T;
  const size_t tasks = static_cast<size_t>(c.n_layers) * B * c.heads, mpad = padded(query_rows);
  return 256 + round_up(tasks * mpad * sizeof(float)) +
         tasks * (mpad / 8) * (c.dtype == FIB_DTYPE_F32 ? kGroupBytes32 : kGroupBytes + (query_rows <= kSpreadRows ? 3 : 1) * kRefGroupBytes);
}

cudaError_t launch_cache_weigh(const fib_attn_cache& cache, int B, int Hq, int T, int rows, int n_max, const int32_t* n_new, const int32_t* path,
                               const int32_t* first, const void* q, const float* lse, float* weights, const float2* lo_tab,
                               const float2* hi_tab, int* status, unsigned long long wait_ns, int skip_copy, void* ws,
                               cudaStream_t stream) {
  WeighArgs a;
  a.c = device_view(cache);
  a.B = B;
  a.Hq = Hq;
  a.G = Hq / cache.heads;
  a.T = T;
  a.rows = rows;
  a.n_max = n_max;
  a.mpad = padded(a.G * T);
  a.n_new = n_new;
  a.path = path;
  a.first = first;
  a.q = q;
  a.lse = lse;
  a.weights = weights;
  a.rope_lo = lo_tab;
  a.rope_hi = hi_tab;
  a.status = status;
  unsigned char* at = static_cast<unsigned char*>(ws);
  a.next = reinterpret_cast<unsigned long long*>(at);
  at += 256;
  a.refs = reinterpret_cast<float*>(at);
  at += round_up(static_cast<size_t>(cache.n_layers) * B * cache.heads * a.mpad * sizeof(float));
  a.parts = at;
  a.ref_parts = at + static_cast<size_t>(cache.n_layers) * B * cache.heads * (a.mpad / 8) * kGroupBytes;
  a.wait_ns = wait_ns;
  a.task_ns = wait_ns + static_cast<unsigned long long>((a.G * a.T + 127) / 128) * 20000;  // (128 queries take a task 2 us)
  a.skip_copy = skip_copy;
  return cache.dtype == FIB_DTYPE_F32 ? launch<float>(a, stream) : launch<__nv_bfloat16>(a, stream);
}

}  // namespace fibattn
