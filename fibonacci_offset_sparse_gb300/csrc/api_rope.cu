// C ABI of the rotary positions (declared in include/fib_attn.h): the handle, argument checks and the launch; and whether a
// plan's own calls rotate.
#include <algorithm>
#include <new>
#include <utility>
#include <vector>

#include "plan.h"
#include "planner.h"
#include "rotary.cuh"

struct fib_attn_rope_s {
  fib_attn_rope_spec spec;
  int N_max = 0, device = -1;
  float2* d_lo = nullptr;
  float2* d_hi = nullptr;
  int* d_status = nullptr;
};

using namespace fibattn;

namespace {

void release(fib_attn_rope_s* r) {
  cudaFree(r->d_lo);
  cudaFree(r->d_hi);
  cudaFree(r->d_status);
  delete r;
}

// Rows of 64 at strides s over extents n (b, h, n): whether no two of them overlap.
bool rows_apart(const int64_t* s, const int* n) {
  std::pair<int64_t, int> d[3] = {{s[0], n[0]}, {s[1], n[1]}, {s[2], n[2]}};
  std::sort(d, d + 3);
  int64_t inner = kD;
  for (const auto& [stride, extent] : d) {
    if (extent == 1) continue;
    if (stride < inner) return false;
    inner += stride * (extent - 1);
  }
  return true;
}

constexpr int64_t kFar = 1LL << 58;  // elements: no tensor reaches as far, and neither a sum of three such extents nor the bytes of one leaves 63 bits

// One tensor pair of a call.
int check_rows(int B, int H, int N, int es, const void* x, const int64_t* xs, const void* y, const int64_t* ys) {
  if (x == nullptr || y == nullptr || xs == nullptr || ys == nullptr || !aligned(x, es) || !aligned(y, es)) return FIB_ERR_INVALID_ARG;
  const int n[3] = {B, H, N};
  uint64_t x_end = kD, y_end = kD;
  bool same = x == y;
  for (int d = 0; d < 3; ++d) {
    if (xs[d] < 0 || ys[d] < 0 || xs[d] >= 1LL << 40 || ys[d] >= 1LL << 40) return FIB_ERR_INVALID_ARG;
    if (n[d] > 1) {
      if (std::max(xs[d], ys[d]) > (kFar - 1) / (n[d] - 1)) return FIB_ERR_INVALID_ARG;  // (before the product is made)
      x_end += static_cast<uint64_t>(xs[d]) * (n[d] - 1);
      y_end += static_cast<uint64_t>(ys[d]) * (n[d] - 1);
      same = same && xs[d] == ys[d];
    }
  }
  if (x_end >= kFar || y_end >= kFar || !rows_apart(ys, n)) return FIB_ERR_INVALID_ARG;
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(x), y0 = reinterpret_cast<uintptr_t>(y);
  if (!same && x0 < y0 + y_end * es && y0 < x0 + x_end * es) return FIB_ERR_INVALID_ARG;
  return FIB_OK;
}

// Rows of 64 of a tensor that check_rows has passed: where the first lies, strides, extents.
struct Rows {
  uintptr_t at;
  const int64_t* s;
  int n[3];
  int64_t end() const {
    int64_t e = kD;
    for (int d = 0; d < 3; ++d) e += s[d] * (n[d] - 1);
    return e;
  }
  bool packed() const { return rows_apart(s, n) && end() == static_cast<int64_t>(kD) * n[0] * n[1] * n[2]; }
};

// Whether some index differences d_i in [low_i, high_i] take `behind` + sum of s_i d_i into (-kD, kD); strides descend, in `more` of them.
struct Steps {
  int64_t s, low, high;
};
bool meets(const Steps* step, int more, int64_t behind) {
  if (more == 0) return behind > -kD && behind < kD;
  int64_t below = kD - 1, above = kD - 1;  // what the smaller strides can still take off and add
  for (int i = 1; i < more; ++i) {
    below -= step[i].s * step[i].low;
    above += step[i].s * step[i].high;
  }
  const int64_t s = step->s;
  // the differences that leave the rest in reach; more than a few only where an input's rows overlap one another, which is not looked into
  const int64_t first = std::max(step->low, -((behind + above) / s) - 1), last = std::min(step->high, (below - behind) / s + 1);
  if (last - first > 16) return false;
  for (int64_t d = first; d <= last; ++d)
    if (meets(step + 1, more - 1, behind + s * d)) return true;
  return false;
}

// Whether an output shares memory with another tensor of the call.  Found for tensors of the same strides, as parts of one projection are
// (a stride of one row only counts for nothing), and for two without gaps; of others, which may lie in one another's gaps, only by their first rows.
bool overlap(const Rows& x, const Rows& y, int es) {
  if (x.at == y.at) return true;
  if (x.at >= y.at + y.end() * es || y.at >= x.at + x.end() * es) return false;
  if (x.packed() && y.packed()) return true;
  Steps step[3];
  int steps = 0;
  for (int d = 0; d < 3; ++d) {
    if (x.n[d] > 1 && y.n[d] > 1 && x.s[d] != y.s[d]) return false;
    const int64_t s = x.n[d] > 1 ? x.s[d] : y.s[d];
    if ((x.n[d] > 1 || y.n[d] > 1) && s > 0) step[steps++] = {s, 1 - x.n[d], y.n[d] - 1};
  }
  std::sort(step, step + steps, [](const Steps& a, const Steps& b) { return a.s > b.s; });
  return meets(step, steps, (static_cast<int64_t>(y.at) - static_cast<int64_t>(x.at)) / es);
}

}  // namespace

extern "C" {

int fib_attn_rope_frequencies(const fib_attn_rope_spec* spec, double* theta_out) {
  if (spec == nullptr || theta_out == nullptr) return FIB_ERR_INVALID_ARG;
  double theta[kFreq];
  if (!rope_frequencies(*spec, theta)) return FIB_ERR_INVALID_ARG;
  std::copy(theta, theta + spec->rot_dim / 2, theta_out);
  return FIB_OK;
}

int fib_attn_rope_create(fib_attn_rope_t* out, const fib_attn_rope_spec* spec, int N_max) {
  if (out == nullptr) return FIB_ERR_INVALID_ARG;
  *out = nullptr;
  double theta[kFreq] = {};
  if (spec == nullptr || N_max < 1 || N_max > (1 << 20) || !rope_frequencies(*spec, theta)) return FIB_ERR_INVALID_ARG;
  std::vector<float> lo, hi;
  try {
    rope_tables(N_max, theta, &lo, &hi);
  } catch (...) {
    return FIB_ERR_NOMEM;
  }
  fib_attn_rope_s* r = new (std::nothrow) fib_attn_rope_s();
  if (r == nullptr) return FIB_ERR_NOMEM;
  r->spec = *spec;
  r->N_max = N_max;
  cudaError_t e = cudaGetDevice(&r->device);
  if (e == cudaSuccess) e = cudaMalloc(&r->d_lo, lo.size() * sizeof(float));
  if (e == cudaSuccess) e = cudaMalloc(&r->d_hi, hi.size() * sizeof(float));
  if (e == cudaSuccess) e = cudaMalloc(&r->d_status, sizeof(int));
  if (e == cudaSuccess) e = cudaMemcpy(r->d_lo, lo.data(), lo.size() * sizeof(float), cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaMemcpy(r->d_hi, hi.data(), hi.size() * sizeof(float), cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaMemset(r->d_status, 0, sizeof(int));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();  // (the clearing, before a call on a stream that does not wait for it)
  if (e != cudaSuccess) {
    release(r);
    return cuda_status(e);
  }
  *out = r;
  return FIB_OK;
}

int fib_attn_rope_destroy(fib_attn_rope_t r) {
  if (r == nullptr) return FIB_OK;
  int prev = -1;
  cudaGetDevice(&prev);
  if (r->device >= 0) cudaSetDevice(r->device);
  cudaDeviceSynchronize();
  release(r);
  if (prev >= 0) cudaSetDevice(prev);
  return FIB_OK;
}

int fib_attn_rotary(fib_attn_rope_t r, int dtype, int B, int N, int Hq, int Hk, const void* q, const int64_t* q_strides, void* q_out,
                    const int64_t* q_out_strides, const void* k, const int64_t* k_strides, void* k_out, const int64_t* k_out_strides,
                    const int32_t* pos, const int32_t* start, int transpose, void* stream) {
  if (r == nullptr || (dtype != FIB_DTYPE_F32 && dtype != FIB_DTYPE_BF16)) return FIB_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || static_cast<long long>(B) * N > 0x7fffffffLL) return FIB_ERR_INVALID_ARG;
  if (Hq < 1 || Hq > FIB_MAX_HEADS || Hk < 0 || Hk > FIB_MAX_HEADS) return FIB_ERR_INVALID_ARG;
  const int es = dtype == FIB_DTYPE_F32 ? 4 : 2;
  if (check_rows(B, Hq, N, es, q, q_strides, q_out, q_out_strides)) return FIB_ERR_INVALID_ARG;
  if (Hk > 0 && check_rows(B, Hk, N, es, k, k_strides, k_out, k_out_strides)) return FIB_ERR_INVALID_ARG;
  if (Hk > 0) {
    const auto rows = [&](const void* at, const int64_t* s, int H) { return Rows{reinterpret_cast<uintptr_t>(at), s, {B, H, N}}; };
    const Rows to = rows(q_out, q_out_strides, Hq), k_to = rows(k_out, k_out_strides, Hk);
    if (overlap(rows(k, k_strides, Hk), to, es) || overlap(rows(q, q_strides, Hq), k_to, es) || overlap(to, k_to, es)) return FIB_ERR_INVALID_ARG;
  }
  if ((pos != nullptr && start != nullptr) || !aligned(pos, 4) || !aligned(start, 4)) return FIB_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return FIB_ERR_CUDA;
  if (dev != r->device) return FIB_ERR_INVALID_ARG;
  RotaryArgs a = {};
  a.B = B;
  a.N = N;
  a.n_max = r->N_max;
  a.heads[0] = Hq;
  a.heads[1] = Hk;
  a.x[0] = q;
  a.y[0] = q_out;
  a.x[1] = k;
  a.y[1] = k_out;
  for (int d = 0; d < 3; ++d) {
    a.xs[0][d] = q_strides[d];
    a.ys[0][d] = q_out_strides[d];
    if (Hk > 0) {
      a.xs[1][d] = k_strides[d];
      a.ys[1][d] = k_out_strides[d];
    }
  }
  a.pos = pos;
  a.start = start;
  a.rope_lo = r->d_lo;
  a.rope_hi = r->d_hi;
  a.layout = r->spec.layout;
  a.rot_dim = r->spec.rot_dim;
  a.amp = static_cast<float>(r->spec.amplitude);
  a.sign = transpose ? -1.f : 1.f;
  a.status = r->d_status;
  return cuda_status(launch_rotary(a, dtype, static_cast<cudaStream_t>(stream)));
}

int fib_attn_rope_status(fib_attn_rope_t r) {
  if (r == nullptr) return FIB_ERR_INVALID_ARG;
  if (cudaDeviceSynchronize() != cudaSuccess) return FIB_ERR_CUDA;
  int h = 0;
  if (cudaMemcpy(&h, r->d_status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return FIB_ERR_CUDA;
  if (h != FIB_OK && (cudaMemset(r->d_status, 0, sizeof(int)) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess)) return FIB_ERR_CUDA;
  return h;
}

int fib_attn_plan_set_rotation(fib_attn_plan_t p, int rotate) {
  if (p == nullptr) return FIB_ERR_INVALID_ARG;
  const int st = check_device(p);
  if (st != FIB_OK) return st;
  if (p->rotates == (rotate != 0)) return FIB_OK;
  std::vector<float> lo, hi;
  try {
    const double none[kFreq] = {};
    if (rotate)
      rope_tables(p->N_max, p->rope_base, &lo, &hi);
    else
      rope_tables(p->N_max, none, &lo, &hi);
  } catch (...) {
    return FIB_ERR_NOMEM;
  }
  cudaError_t e = cudaDeviceSynchronize();  // no call that reads the tables is under way
  if (e == cudaSuccess) e = cudaMemcpy(p->d_lo, lo.data(), lo.size() * sizeof(float), cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaMemcpy(p->d_hi, hi.data(), hi.size() * sizeof(float), cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e == cudaSuccess) p->rotates = rotate != 0;
  return cuda_status(e);
}

}  // extern "C"
