// C ABI of the paged cache and the tree decodes over it (declared in include/fib_attn.h):
// argument checks and launches.  As in api.cu, every entry point only enqueues work.
#include "cache.cuh"
#include "plan.h"

using namespace fibattn;

namespace {

// The struct's own rules; no device call.
int check_cache(const fib_attn_cache* c) {
  if (c == nullptr) return FIB_ERR_INVALID_ARG;
  if (c->dtype != FIB_DTYPE_F32 && c->dtype != FIB_DTYPE_BF16) return FIB_ERR_INVALID_ARG;
  if (c->n_layers < 1 || c->n_layers > FIB_MAX_LAYERS || c->heads < 1 || c->heads > FIB_MAX_HEADS) return FIB_ERR_INVALID_ARG;
  if (c->page_rows < 16 || c->page_rows > 256 || (c->page_rows & (c->page_rows - 1)) != 0) return FIB_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->max_seqs < 1 || c->max_seqs > FIB_MAX_SEQS || c->max_pages < 1) return FIB_ERR_INVALID_ARG;
  if (static_cast<long long>(c->max_pages) * c->page_rows > (1LL << 30)) return FIB_ERR_INVALID_ARG;
  if (static_cast<long long>(c->heads) * c->page_rows > 0x7fffffffLL / c->n_pages) return FIB_ERR_INVALID_ARG;
  if (check_tensor(c->k) || check_tensor(c->v) || check_tensor(c->refs) || check_tensor(c->state)) return FIB_ERR_INVALID_ARG;
  if (c->k == c->v) return FIB_ERR_INVALID_ARG;
  if (c->table == nullptr || !aligned(c->table, 4) || c->lens == nullptr || !aligned(c->lens, 4)) return FIB_ERR_INVALID_ARG;
  return FIB_OK;
}

int check_cache_device(const fib_attn_cache* c) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return FIB_ERR_CUDA;
  return dev == c->device ? FIB_OK : FIB_ERR_INVALID_ARG;
}

int check_ints(const int32_t* p) { return p == nullptr || !aligned(p, 4) ? FIB_ERR_INVALID_ARG : FIB_OK; }

int check_workspace(const void* ws, size_t bytes, size_t need) {
  return ws == nullptr || !aligned(ws, 256) || bytes < need ? FIB_ERR_INVALID_ARG : FIB_OK;
}

// The layer's key table: at N_max, where most calls are, the plan's own.  make_table allocates on the host; nothing may
// escape a C entry point.
int table_of(const fib_attn_plan_s* p, int layer, int N, const float* alpha_dev, LayerTable* t) noexcept {
  if (N == p->N_max) {
    *t = alpha_dev == nullptr ? p->tables[layer] : p->dev_table;
    t->layer = layer;
    t->alpha_dev = alpha_dev;
    return alpha_dev == nullptr ? FIB_OK : p->dev_status;
  }
  try {
    return make_table(p, layer, N, alpha_dev, t);
  } catch (...) {
    return FIB_ERR_NOMEM;
  }
}

// What both decodes check; fills everything of `a` but the key table.
int tree_args(fib_attn_plan_t p, int layer, const fib_attn_cache* c, int B, int Hq, int T, int N, const void* q,
              const void* k_new, const void* v_new, const int32_t* parent, const int32_t* n_nodes, void* o, float* lse,
              TreeArgs* a) {
  if (p == nullptr) return FIB_ERR_INVALID_ARG;
  const int st = check_cache(c);
  if (st != FIB_OK) return st;
  if (layer < 0 || layer >= c->n_layers) return FIB_ERR_INVALID_ARG;
  if (B < 1 || B > c->max_seqs || T < 1 || T > FIB_MAX_DRAFTS || N < 1 || N > p->N_max) return FIB_ERR_INVALID_ARG;
  if (Hq < 1 || Hq > FIB_MAX_HEADS || Hq % c->heads != 0) return FIB_ERR_INVALID_ARG;
  if (check_tensor(q) || check_tensor(k_new) || check_tensor(v_new) || check_tensor(o)) return FIB_ERR_INVALID_ARG;
  if (o == q || o == k_new || o == v_new || o == c->k || o == c->v) return FIB_ERR_INVALID_ARG;
  if (lse != nullptr && !aligned(lse, 4)) return FIB_ERR_INVALID_ARG;
  if (parent != nullptr && check_ints(parent)) return FIB_ERR_INVALID_ARG;
  if (n_nodes != nullptr && check_ints(n_nodes)) return FIB_ERR_INVALID_ARG;
  a->N = N;
  a->B = B;
  a->Hq = Hq;
  a->H = c->heads;
  a->G = Hq / c->heads;
  a->T = T;
  a->n_pages = c->n_pages;
  a->max_pages = c->max_pages;
  a->page_shift = log2_of(c->page_rows);
  a->q = q;
  a->kn = k_new;
  a->vn = v_new;
  const size_t layer_bytes = static_cast<size_t>(c->n_pages) * c->heads * c->page_rows * kD *
                             (c->dtype == FIB_DTYPE_F32 ? 4 : 2) * static_cast<size_t>(layer);
  a->kc = static_cast<const unsigned char*>(c->k) + layer_bytes;
  a->vc = static_cast<const unsigned char*>(c->v) + layer_bytes;
  a->table = c->table;
  a->lens = c->lens;
  a->parent = parent;
  a->nodes = n_nodes;
  a->o = o;
  a->lse = lse;
  a->rope_lo = p->d_lo;
  a->rope_hi = p->d_hi;
  a->status = p->d_status;
  return FIB_OK;
}

}  // namespace

extern "C" {

size_t fib_attn_cache_workspace_size(const fib_attn_cache* c) {
  return check_cache(c) == FIB_OK ? cache_workspace_bytes(*c) : 0;
}

int fib_attn_cache_commit(fib_attn_plan_t p, const fib_attn_cache* c, int B, int T, const int32_t* n_new,
                          const int32_t* path, const void* k_new, const void* v_new, void* workspace, size_t ws_bytes,
                          void* stream) {
  int st = check_cache(c);
  if (st != FIB_OK) return st;
  if (p == nullptr || B < 1 || B > c->max_seqs || T < 1 || T > (1 << 20)) return FIB_ERR_INVALID_ARG;
  if (check_ints(n_new) || (path != nullptr && check_ints(path))) return FIB_ERR_INVALID_ARG;
  if (check_tensor(k_new) || check_tensor(v_new)) return FIB_ERR_INVALID_ARG;
  if (k_new == c->k || k_new == c->v || v_new == c->k || v_new == c->v) return FIB_ERR_INVALID_ARG;
  if (check_workspace(workspace, ws_bytes, cache_workspace_bytes(*c))) return FIB_ERR_INVALID_ARG;
  st = check_device(p);
  if (st == FIB_OK) st = check_cache_device(c);
  if (st != FIB_OK) return st;
  return cuda_status(launch_cache_commit(*c, B, T, p->N_max, n_new, path, k_new, v_new, p->d_lo, p->d_hi, workspace,
                                         static_cast<cudaStream_t>(stream)));
}

int fib_attn_cache_fork(const fib_attn_cache* c, const int32_t* src, void* workspace, size_t ws_bytes, void* stream) {
  int st = check_cache(c);
  if (st != FIB_OK) return st;
  if (check_ints(src) || src == c->lens || src == c->table) return FIB_ERR_INVALID_ARG;
  if (check_workspace(workspace, ws_bytes, cache_workspace_bytes(*c))) return FIB_ERR_INVALID_ARG;
  st = check_cache_device(c);
  if (st != FIB_OK) return st;
  return cuda_status(launch_cache_fork(*c, src, workspace, static_cast<cudaStream_t>(stream)));
}

int fib_attn_cache_compact(const fib_attn_cache* c, int32_t* remap, void* workspace, size_t ws_bytes, void* stream) {
  int st = check_cache(c);
  if (st != FIB_OK) return st;
  if (check_ints(remap) || remap == c->refs || remap == c->table || remap == c->lens) return FIB_ERR_INVALID_ARG;
  if (check_workspace(workspace, ws_bytes, cache_workspace_bytes(*c)) || workspace == remap) return FIB_ERR_INVALID_ARG;
  st = check_cache_device(c);
  if (st != FIB_OK) return st;
  return cuda_status(launch_cache_compact(*c, remap, workspace, static_cast<cudaStream_t>(stream)));
}

// What a call of these sizes needs; 0 where they break the rules.  (Query rows are held to 2^40 values, so that no size here leaves 64 bits.)
static size_t weigh_bytes(const fib_attn_cache* c, int B, int Hq, int T) {
  if (B < 1 || B > c->max_seqs || T < 1 || T > (1 << 20) || Hq < 1 || Hq > FIB_MAX_HEADS || Hq % c->heads != 0) return 0;
  if (static_cast<long long>(c->n_layers) * B * Hq > (1LL << 40) / kD / T) return 0;
  return weigh_workspace_bytes(*c, B, Hq, T);
}

size_t fib_attn_cache_weigh_workspace_size(const fib_attn_cache* c, int B, int Hq, int T) {
  return check_cache(c) == FIB_OK ? weigh_bytes(c, B, Hq, T) : 0;
}

int fib_attn_cache_weigh(fib_attn_plan_t p, const fib_attn_cache* c, int B, int Hq, int T, int rows, const int32_t* n_new,
                         const int32_t* path, const int32_t* first, const void* q, const float* lse, float* weights, void* workspace,
                         size_t ws_bytes, void* stream) {
  int st = check_cache(c);
  if (st != FIB_OK) return st;
  const size_t need = weigh_bytes(c, B, Hq, T);
  if (p == nullptr || need == 0 || rows < 1 || rows > (1 << 30)) return FIB_ERR_INVALID_ARG;
  if (check_ints(n_new) || !aligned(path, 4) || !aligned(first, 4) || check_tensor(q)) return FIB_ERR_INVALID_ARG;
  if (lse == nullptr || !aligned(lse, 4) || weights == nullptr || !aligned(weights, 4) || weights == lse) return FIB_ERR_INVALID_ARG;
  if (check_workspace(workspace, ws_bytes, need)) return FIB_ERR_INVALID_ARG;
  if (workspace == q || workspace == lse || workspace == weights) return FIB_ERR_INVALID_ARG;
  st = check_device(p);
  if (st == FIB_OK) st = check_cache_device(c);
  if (st != FIB_OK) return st;
  return cuda_status(launch_cache_weigh(*c, B, Hq, T, rows, p->N_max, n_new, path, first, q, lse, weights, p->d_lo, p->d_hi, p->d_status,
                                        p->wait_ns, p->skip_first_rung_copy, workspace, static_cast<cudaStream_t>(stream)));
}

size_t fib_attn_cache_evict_workspace_size(const fib_attn_cache* c, int rows) {
  if (check_cache(c) != FIB_OK || rows < 1 || rows > (1 << 30)) return 0;
  return cache_evict_workspace_bytes(*c, rows);
}

int fib_attn_cache_evict(fib_attn_plan_t p, const fib_attn_cache* c, int B, int rows, const int32_t* keep, int sink, int recent,
                         float* weights, int32_t* dropped, void* workspace, size_t ws_bytes, void* stream) {
  int st = check_cache(c);
  if (st != FIB_OK) return st;
  if (p == nullptr || B < 1 || B > c->max_seqs || rows < 1 || rows > (1 << 30)) return FIB_ERR_INVALID_ARG;
  if (sink < 0 || recent < 0 || sink > (1 << 29) || recent > (1 << 29)) return FIB_ERR_INVALID_ARG;
  if (check_ints(keep) || weights == nullptr || !aligned(weights, 4) || !aligned(dropped, 4)) return FIB_ERR_INVALID_ARG;
  if (dropped != nullptr && (dropped == keep || dropped == c->lens || dropped == c->table || dropped == c->refs)) return FIB_ERR_INVALID_ARG;
  if (check_workspace(workspace, ws_bytes, cache_evict_workspace_bytes(*c, rows)) || workspace == weights) return FIB_ERR_INVALID_ARG;
  st = check_device(p);
  if (st == FIB_OK) st = check_cache_device(c);
  if (st != FIB_OK) return st;
  return cuda_status(launch_cache_evict(*c, B, rows, keep, sink, recent, p->N_max, weights, dropped, p->d_lo, p->d_hi, p->turn,
                                        workspace, static_cast<cudaStream_t>(stream)));
}

int fib_attn_tree_decode(fib_attn_plan_t p, int layer, const fib_attn_cache* c, int B, int Hq, int T, int N,
                         const void* q, const void* k_new, const void* v_new, const int32_t* parent,
                         const int32_t* n_nodes, void* o, float* lse, const float* alpha_dev, void* stream) {
  TreeArgs a;
  int st = tree_args(p, layer, c, B, Hq, T, N, q, k_new, v_new, parent, n_nodes, o, lse, &a);
  if (st != FIB_OK) return st;
  if (layer >= static_cast<int>(p->alpha.size())) return FIB_ERR_INVALID_ARG;
  if (alpha_dev != nullptr && !aligned(alpha_dev, 4)) return FIB_ERR_INVALID_ARG;
  st = check_device(p);
  if (st == FIB_OK) st = check_cache_device(c);
  if (st != FIB_OK) return st;
  st = table_of(p, layer, N, p->mode == FIB_MODE_INTERP ? alpha_dev : nullptr, &a.t);
  if (st != FIB_OK) return st;
  return cuda_status(launch_tree(a, c->dtype, static_cast<cudaStream_t>(stream)));
}

size_t fib_attn_dense_tree_workspace_size(fib_attn_plan_t p, const fib_attn_cache* c, int B, int Hq, int T) {
  if (p == nullptr || check_cache(c) != FIB_OK || B < 1 || B > c->max_seqs || T < 1 || T > FIB_MAX_DRAFTS || Hq < 1 ||
      Hq > FIB_MAX_HEADS || Hq % c->heads != 0)
    return 0;
  return dense_tree_workspace_bytes(Hq, c->heads, T, c->dtype);
}

int fib_attn_dense_tree_decode(fib_attn_plan_t p, int layer, const fib_attn_cache* c, int B, int Hq, int T,
                               const void* q, const void* k_new, const void* v_new, const int32_t* parent,
                               const int32_t* n_nodes, void* o, float* lse, void* workspace, size_t ws_bytes,
                               void* stream) {
  TreeArgs a;
  int st = tree_args(p, layer, c, B, Hq, T, p == nullptr ? 0 : p->N_max, q, k_new, v_new, parent, n_nodes, o, lse, &a);
  if (st != FIB_OK) return st;
  if (check_workspace(workspace, ws_bytes, dense_tree_workspace_bytes(Hq, c->heads, T, c->dtype)))
    return FIB_ERR_INVALID_ARG;
  if (workspace == q || workspace == o || workspace == k_new || workspace == v_new) return FIB_ERR_INVALID_ARG;
  st = check_device(p);
  if (st == FIB_OK) st = check_cache_device(c);
  if (st != FIB_OK) return st;
  a.t = LayerTable{};
  return cuda_status(launch_dense_tree(a, c->dtype, p->wait_ns, p->skip_first_rung_copy, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
