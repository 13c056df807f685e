// Rotary positions by themselves (sm_103a): pairs of dims turned by position * frequency, the rest copied.
//
// y = amplitude * R(p) x; R is orthogonal a pair, so the transposed map (the backward pass) is the same kernel with the sine
// negated.  e^{i p theta} is one complex product of two table entries (p = 64 hi + lo, both built in binary64), 1.2e-7 of error.
//
// What bounds it: the rows' bytes.  So a quad of threads takes a row as wide loads (each thread both halves of its pairs), reads
// its eight factors once and uses them for several heads of the token; what is on its way at a time is kHeads rows a quad.
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

template <typename DT>
struct Vec8;  // eight values, as they lie in memory
template <>
struct Vec8<__nv_bfloat16> {
  uint4 x;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { x = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = x; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = bf_lo(x.x); v[1] = bf_hi(x.x); v[2] = bf_lo(x.y); v[3] = bf_hi(x.y);
    v[4] = bf_lo(x.z); v[5] = bf_hi(x.z); v[6] = bf_lo(x.w); v[7] = bf_hi(x.w);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    x = make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7]));
  }
};
template <>
struct Vec8<float> {
  float4 x, y;
  __device__ __forceinline__ void load(const float* p) {
    x = reinterpret_cast<const float4*>(p)[0];
    y = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = x;
    reinterpret_cast<float4*>(p)[1] = y;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    x = make_float4(v[0], v[1], v[2], v[3]);
    y = make_float4(v[4], v[5], v[6], v[7]);
  }
};

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

// A quad a token, HEADS heads; thread t of it holds 16 dims of each row, as two runs of eight: of INTERLEAVED pairs
// 16t .. 16t+15, of rotate-half ones (rot_dim a multiple of 16) 8t .. and their partners, of what is only copied the
// next 16 that no thread before it holds.
template <typename DT, int HEADS, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  const int t = threadIdx.x & 3;
  const long long item = static_cast<long long>(blockIdx.x) * (kThreads / 4) + (threadIdx.x >> 2);
  if (item >= static_cast<long long>(a.B) * a.N) return;
  const int b = static_cast<int>(item / a.N), n = static_cast<int>(item - static_cast<long long>(b) * a.N);
  const int heads = a.heads[0] + a.heads[1], h0 = blockIdx.y * HEADS, turned = a.rot_dim / 16;
  int at0, at1;
  if (INTERLEAVED || t >= turned) {
    at0 = 16 * t;
    at1 = at0 + 8;
  } else {
    at0 = 8 * t;
    at1 = a.rot_dim / 2 + 8 * t;
  }
  Vec8<DT> v[HEADS][2];
#pragma unroll
  for (int i = 0; i < HEADS; ++i)
    if (h0 + i < heads) {
      const DT* x = row_in<DT>(a, b, h0 + i, n);
      v[i][0].load(x + at0);
      v[i][1].load(x + at1);
    }
  int p;
  if (!position(a, b, n, &p)) return;
  // pairs 8t .. 8t+7, of which the first `pairs` are rotated
  const int pairs = INTERLEAVED ? max(0, min(8, a.rot_dim / 2 - 8 * t)) : t < turned ? 8 : 0;
  if (pairs > 0) {
    float2 e[8];
    rope_row(a.rope_lo, a.rope_hi, p, t, e);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      e[u].x *= a.amp;
      e[u].y *= a.amp * a.sign;
    }
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      float x[8], y[8];
      v[i][0].get(x);
      v[i][1].get(y);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        float& c = INTERLEAVED ? (u < 4 ? x[2 * (u & 3)] : y[2 * (u & 3)]) : x[u];
        float& d = INTERLEAVED ? (u < 4 ? x[2 * (u & 3) + 1] : y[2 * (u & 3) + 1]) : y[u];
        const float c0 = c, d0 = d;
        if (!INTERLEAVED || u < pairs) {
          c = c0 * e[u].x - d0 * e[u].y;
          d = c0 * e[u].y + d0 * e[u].x;
        }
      }
      v[i][0].set(x);
      v[i][1].set(y);
    }
  }
#pragma unroll
  for (int i = 0; i < HEADS; ++i)
    if (h0 + i < heads) {
      DT* y = row_out<DT>(a, b, h0 + i, n);
      v[i][0].store(y + at0);
      v[i][1].store(y + at1);
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

// Whether every row is made of aligned runs of eight.
bool wide(const RotaryArgs& a, int es) {
  if (a.layout == FIB_ROPE_HALF && a.rot_dim % 16 != 0) return false;
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
    const dim3 grid(static_cast<unsigned>((items + kThreads / 4 - 1) / (kThreads / 4)), (heads + HEADS - 1) / HEADS);
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
  return dtype == FIB_DTYPE_F32 ? launch<float, 2>(a, stream) : launch<__nv_bfloat16, 4>(a, stream);
}

}  // namespace fibattn
