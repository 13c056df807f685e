// The accumulated attention weight of cached rows: what its kernels share (weigh.cu, weigh_tc.cu).
#pragma once
#include "cache_dev.cuh"
#include "tree.cuh"

namespace fibattn {

struct WeighArgs {
  CacheDev c;
  int B, Hq, G, T, rows, n_max;
  int mpad;  // query rows a key head (token-major, its G heads after one another), rounded up
  const int32_t* n_new;
  const int32_t* path;
  const int32_t* first;
  const void* q;
  const float* lse;
  float* weights;  // [L, S, H, rows]
  const float2* rope_lo;
  const float2* rope_hi;
  int* status;
  // Workspace.  parts: for each layer, sequence and key head, and 8 query rows after one another, the rotated rows times
  // log2(e)/8, split: bf16 hi, mid, lo, each [8][64] with its 16-byte words swizzled as the tensor pipes' 128-byte pattern, word w of
  // row r at w ^ r; float32 hi, lo (tf32), each [8][64].  refs: -lse * log2(e), -inf where there is no row.
  // ref_parts (weigh_tc.cu alone): the same split in bf16 hi, mid, lo, as rows of 16 of which the others are 0, for 8 query rows [2][8][8]; for
  // kSpreadRows or less a key head three of these, of the first hi alone, of the second mid, of the third lo.
  unsigned char* parts;
  float* refs;
  unsigned char* ref_parts;
  unsigned long long* next;  // weigh_tc.cu: the next task to be taken
  unsigned long long wait_ns;
  unsigned long long task_ns;  // weigh_tc.cu: ... of a wait that may take as long as a task
  int skip_copy;  // test hook: the first rows of every task of weigh_tc.cu are never copied
};

constexpr int kPartBytes = 8 * kD * 2;        // 8 rows of one bf16 part
constexpr int kGroupBytes = 3 * kPartBytes;   // 8 query rows, bf16
constexpr int kGroupBytes32 = 2 * 8 * kD * 4;  // ... float32
constexpr int kRefGroupBytes = 8 * 16 * 2;     // the references of 8 query rows
constexpr int kSpreadRows = 32;                // query rows a key head up to which weigh_tc.cu has the parts as columns

// For what is in flight when a warp gives up: its wait is not the caller's, which may be too short for a copy.
constexpr unsigned long long kWeighDrainNs = 2000000000ull;

// Sequence b of a call: rows, new ones (0: nothing to do), the first row whose weight begins with this call.
struct WeighSeq {
  int len, n, first;
};
__device__ __forceinline__ WeighSeq weigh_seq(const WeighArgs& a, int b, bool* ok) {
  WeighSeq s;
  s.len = a.c.lens[b];
  s.n = a.n_new[b];
  s.first = a.first == nullptr ? s.len - s.n : a.first[b];
  *ok = s.n >= 0 && s.n <= a.T && (s.n == 0 || (s.len >= s.n && s.len <= static_cast<long long>(a.c.max_pages) * a.c.P && s.len <= a.rows && s.len <= a.n_max));
  if (!*ok) s.n = 0;
  return s;
}

// weigh_tc.cu: bf16, more than 8 query rows a key head
cudaError_t launch_weigh_tc(const WeighArgs& a, cudaStream_t stream);

}  // namespace fibattn
