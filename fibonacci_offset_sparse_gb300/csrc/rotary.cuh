// Launch interface of the rotary positions' kernels (rotary.cu).
#pragma once
#include "../../include/fib_attn.h"
#include "common.cuh"

namespace fibattn {

// Queries (0) and keys (1): rows of 64 at x + b * xs[0] + h * xs[1] + n * xs[2] (elements), to y likewise.
struct RotaryArgs {
  int B, N, n_max;
  int heads[2];
  const void* x[2];
  void* y[2];
  long long xs[2][3], ys[2][3];
  const int32_t* pos;
  const int32_t* start;
  const float2* rope_lo;
  const float2* rope_hi;
  int layout, rot_dim;
  float amp, sign;  // of the factors; sign: -1 transposed
  int* status;
};
cudaError_t launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t stream);

}  // namespace fibattn
