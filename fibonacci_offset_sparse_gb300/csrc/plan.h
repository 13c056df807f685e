// The plan behind fib_attn_plan_t and the argument checks that the entry points share.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <vector>

#include "../../include/fib_attn.h"
#include "common.cuh"

struct fib_attn_plan_s {
  int base_kind = 0;
  std::vector<int32_t> custom;
  std::vector<double> alpha;
  int W = 0, N_max = 0, D = 0, mode = 0;
  double rope_base = 10000.0;
  int device = -1;
  float2* d_lo = nullptr;
  float2* d_hi = nullptr;
  int* d_status = nullptr;
  unsigned long long wait_ns = 1000000000ULL;  // bound of every device-side wait (1 s)
  int skip_first_rung_copy = 0;                // test hooks, see fib_attn_plan_set_debug
  int corrupt_rung_table = 0;
  // At N_max: every layer's table, and the one that a device alpha completes (INTERP; its status).
  std::vector<fibattn::LayerTable> tables;
  fibattn::LayerTable dev_table = {};
  int dev_status = FIB_ERR_UNSUPPORTED;
  fibattn::BwdStreams side;                             // the bf16 backward's second-half stream
  std::mutex side_mu;                          // one backward at a time forks onto it
};

namespace fibattn {

// Per-layer key table for a call at sequence length N (api.cu).
int make_table(const fib_attn_plan_s* p, int layer, int N, const float* alpha_dev, LayerTable* t);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int check_device(const fib_attn_plan_s* p) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return FIB_ERR_CUDA;
  if (dev != p->device) return FIB_ERR_INVALID_ARG;
  return FIB_OK;
}

inline int check_tensor(const void* ptr) {
  if (ptr == nullptr || !aligned(ptr, 16)) return FIB_ERR_INVALID_ARG;
  return FIB_OK;
}

inline int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return FIB_OK;
  if (e == cudaErrorMemoryAllocation) return FIB_ERR_NOMEM;
  return FIB_ERR_CUDA;
}

}  // namespace fibattn
