// Rotary positions by themselves (sm_103a): pairs of dims turned by position * frequency, the rest copied.
//
// y = amplitude * R(p) x; R is orthogonal a pair, so the transposed map (the backward pass) is the same kernel with the sine
// negated.  e^{i p theta} is one complex product of two table entries (p = 64 hi + lo, both built in binary64), 1.2e-7 of error.
//
// What bounds it: the rows' bytes.  So four threads (float32: eight) take a row as wide loads, each both halves of its pairs, read their
// factors once and use them for several heads of the token; what is on its way at a time is HEADS rows a thread.  131072 tokens of 8 + 8
// bf16 heads: 85 us (6.3 TB/s, 94% of a measured copy); 8 x 4096 out of a fused projection: 22 us (91%); 2 x 74198 tokens of 4 + 2 float32
// heads, interleaved, back into one: 68 us (the copy's rate; with four threads a row 98).  One head alone: 131072 tokens 12 us, 2.8 TB/s, as its
// factors' reads are four times the row's.  Element by element 2 x 60000 tokens of 16 heads take 223 us, by words 79.
#include "rotary.cuh"
#include "tc_common.cuh"

namespace fibattn {

namespace {

// Position of row n of sequence b; false (reported) where the tables do not hold it.
__device__ __forceinline__ bool position(const RotaryArgs& a, int b, int n, int* p) {
  const long long at = a.pos != nullptr     ? a.pos[static_cast<long long>(b) * a.N + n]
                       : a.start != nullptr ? static_cast<long long>(a.start[b]) + n
                                            : n;
  *p = static_cast<int>(at);
  if (at >= 0 && at < a.n_max) return true;
  atomicExch(a.status, kStatusDeviceAssert);
  return false;
}

// 16 bytes of a row, as they lie in memory.
template <typename DT>
struct Word;
template <>
struct Word<__nv_bfloat16> {
  static constexpr int kValues = 8;
  uint4 x;
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = bf_lo(x.x); v[1] = bf_hi(x.x); v[2] = bf_lo(x.y); v[3] = bf_hi(x.y);
    v[4] = bf_lo(x.z); v[5] = bf_hi(x.z); v[6] = bf_lo(x.w); v[7] = bf_hi(x.w);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    x = make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7]));
  }
};
template <>
struct Word<float> {
  static constexpr int kValues = 4;
  uint4 x;
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = __uint_as_float(x.x); v[1] = __uint_as_float(x.y); v[2] = __uint_as_float(x.z); v[3] = __uint_as_float(x.w);
  }
  __device__ __forceinline__ void set(const float (&v)[4]) {
    x = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};

// e^{i p theta_m} of N pairs from m on (a multiple of 2), times the amplitude, the sine with its sign.
template <int N>
__device__ __forceinline__ void factors(const RotaryArgs& a, int p, int m, float2* e) {
  const float4* h4 = reinterpret_cast<const float4*>(a.rope_hi + (p / kSplit) * kFreq + m);
  const float4* l4 = reinterpret_cast<const float4*>(a.rope_lo + (p % kSplit) * kFreq + m);
#pragma unroll
  for (int u = 0; u < N / 2; ++u) {
    const float4 x = __ldg(h4 + u), y = __ldg(l4 + u);
    e[2 * u] = make_float2((x.x * y.x - x.y * y.y) * a.amp, (x.x * y.y + x.y * y.x) * (a.amp * a.sign));
    e[2 * u + 1] = make_float2((x.z * y.z - x.w * y.w) * a.amp, (x.z * y.w + x.w * y.z) * (a.amp * a.sign));
  }
}

constexpr int kThreads = 128;

// Pointer-and-stride arithmetic of head `h` (queries, then keys) at row n of sequence b.
template <typename DT>
__device__ __forceinline__ const DT* row_in(const RotaryArgs& a, int b, int h, int n) {
  const int s = h >= a.heads[0], at = h - (s ? a.heads[0] : 0);
  return static_cast<const DT*>(a.x[s]) + (b * a.xs[s][0] + at * a.xs[s][1] + n * a.xs[s][2]);
}
template <typename DT>
__device__ __forceinline__ DT* row_out(const RotaryArgs& a, int b, int h, int n) {
  const int s = h >= a.heads[0], at = h - (s ? a.heads[0] : 0);
  return static_cast<DT*>(a.y[s]) + (b * a.ys[s][0] + at * a.ys[s][1] + n * a.ys[s][2]);
}

// 4 (float32: 8) threads a token, HEADS heads; thread t holds two 16-byte words of each row: of rotate-half pairs (rot_dim a multiple of two
// words) its t-th word of first dims and that of their partners, of what is only copied the next two that no thread before it holds; of
// interleaved pairs word t of either half of the row.
template <typename DT, int HEADS, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  constexpr int V = Word<DT>::kValues, LANES = kD / (2 * V);
  const int t = threadIdx.x % LANES;
  const long long item = static_cast<long long>(blockIdx.x) * (kThreads / LANES) + threadIdx.x / LANES;
  if (item >= static_cast<long long>(a.B) * a.N) return;
  const int b = static_cast<int>(item / a.N), n = static_cast<int>(item - static_cast<long long>(b) * a.N);
  const int heads = a.heads[0] + a.heads[1], h0 = blockIdx.y * HEADS, turned = a.rot_dim / (2 * V);  // threads with rotate-half pairs
  int at[2] = {V * t, kD / 2 + V * t};
  if (!INTERLEAVED) {
    at[0] = t < turned ? V * t : a.rot_dim + 2 * V * (t - turned);
    at[1] = t < turned ? a.rot_dim / 2 + V * t : at[0] + V;
  }
  Word<DT> v[HEADS][2];
#pragma unroll
  for (int i = 0; i < HEADS; ++i)
    if (h0 + i < heads) {
      const DT* x = row_in<DT>(a, b, h0 + i, n);
#pragma unroll
      for (int k = 0; k < 2; ++k) v[i][k].x = *reinterpret_cast<const uint4*>(x + at[k]);
    }
  int p;
  if (!position(a, b, n, &p)) return;
  float2 e[V];
  if (INTERLEAVED) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (at[k] >= a.rot_dim) break;
      factors<V / 2>(a, p, at[k] / 2, e + k * V / 2);
#pragma unroll
      for (int i = 0; i < HEADS; ++i) {
        float x[V];
        v[i][k].get(x);
#pragma unroll
        for (int u = 0; u < V / 2; ++u) {
          if (at[k] + 2 * u >= a.rot_dim) break;
          const float2 f = e[k * V / 2 + u];
          const float c = x[2 * u], d = x[2 * u + 1];
          x[2 * u] = c * f.x - d * f.y;
          x[2 * u + 1] = c * f.y + d * f.x;
        }
        v[i][k].set(x);
      }
    }
  } else if (t < turned) {
    factors<V>(a, p, V * t, e);
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      float x[V], y[V];
      v[i][0].get(x);
      v[i][1].get(y);
#pragma unroll
      for (int u = 0; u < V; ++u) {
        const float c = x[u], d = y[u];
        x[u] = c * e[u].x - d * e[u].y;
        y[u] = c * e[u].y + d * e[u].x;
      }
      v[i][0].set(x);
      v[i][1].set(y);
    }
  }
#pragma unroll
  for (int i = 0; i < HEADS; ++i)
    if (h0 + i < heads) {
      DT* y = row_out<DT>(a, b, h0 + i, n);
#pragma unroll
      for (int k = 0; k < 2; ++k) *reinterpret_cast<uint4*>(y + at[k]) = v[i][k].x;
    }
}

// Any layout and alignment: a warp a row, a lane a pair (or two dims that are copied).
template <typename DT>
__global__ void __launch_bounds__(kThreads) rotary_any_kernel(const __grid_constant__ RotaryArgs a) {
  const int m = threadIdx.x & 31, heads = a.heads[0] + a.heads[1], half = a.rot_dim / 2;
  const long long item = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (item >= static_cast<long long>(a.B) * a.N) return;
  const int b = static_cast<int>(item / a.N), n = static_cast<int>(item - static_cast<long long>(b) * a.N);
  int p;
  if (!position(a, b, n, &p)) return;
  const bool turn = m < half;
  const int at0 = a.layout == FIB_ROPE_HALF && turn ? m : 2 * m, at1 = a.layout == FIB_ROPE_HALF && turn ? m + half : 2 * m + 1;
  float2 e = rope_factor(a.rope_lo, a.rope_hi, p, m);
  e.x *= a.amp;
  e.y *= a.amp * a.sign;
  for (int h = blockIdx.y; h < heads; h += gridDim.y) {
    const DT* x = row_in<DT>(a, b, h, n);
    const DT c = x[at0], d = x[at1];
    const float cf = static_cast<float>(c), df = static_cast<float>(d);
    __syncwarp();  // (in place: every lane has read its pair; lanes' pairs are their own)
    DT* y = row_out<DT>(a, b, h, n);
    y[at0] = turn ? static_cast<DT>(cf * e.x - df * e.y) : c;
    y[at1] = turn ? static_cast<DT>(cf * e.y + df * e.x) : d;
  }
}

// Whether every row is made of aligned words that a thread has both halves of pairs of.
bool wide(const RotaryArgs& a, int es) {
  if (a.layout == FIB_ROPE_HALF && a.rot_dim % (32 / es) != 0) return false;
  for (int s = 0; s < 2; ++s) {
    if (a.heads[s] == 0) continue;
    if (reinterpret_cast<uintptr_t>(a.x[s]) % 16 != 0 || reinterpret_cast<uintptr_t>(a.y[s]) % 16 != 0) return false;
    for (int d = 0; d < 3; ++d)
      if (a.xs[s][d] * es % 16 != 0 || a.ys[s][d] * es % 16 != 0) return false;
  }
  return true;
}

template <typename DT, int HEADS>
cudaError_t launch(const RotaryArgs& a, cudaStream_t stream) {
  const long long items = static_cast<long long>(a.B) * a.N;
  const int heads = a.heads[0] + a.heads[1];
  if (wide(a, sizeof(DT))) {
    constexpr int kTokens = kThreads / (kD / (2 * Word<DT>::kValues));
    const dim3 grid(static_cast<unsigned>((items + kTokens - 1) / kTokens), (heads + HEADS - 1) / HEADS);
    if (a.layout == FIB_ROPE_HALF)
      rotary_kernel<DT, HEADS, false><<<grid, kThreads, 0, stream>>>(a);
    else
      rotary_kernel<DT, HEADS, true><<<grid, kThreads, 0, stream>>>(a);
  } else {
    const dim3 grid(static_cast<unsigned>((items + kThreads / 32 - 1) / (kThreads / 32)), (heads + 3) / 4);
    rotary_any_kernel<DT><<<grid, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t stream) {
  return dtype == FIB_DTYPE_F32 ? launch<float, 4>(a, stream) : launch<__nv_bfloat16, 4>(a, stream);
}

}  // namespace fibattn
