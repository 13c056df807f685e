"""Thin Python binding of libfibattn.so (argument marshalling only).

Function names mirror the C ABI in include/fib_attn.h.  Tensors are torch tensors on the
plan's CUDA device, contiguous [B, H, N, 64]; the binding passes their data pointers and
the current torch stream.  Every computation runs in the library's CUDA kernels: there is
no CPU fallback, and a missing or unloadable library raises immediately.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfibattn.so")

FIB_OK, FIB_ERR_INVALID_ARG, FIB_ERR_UNSUPPORTED, FIB_ERR_CUDA, FIB_ERR_NOMEM, \
    FIB_ERR_TIMEOUT, FIB_ERR_DEVICE_ASSERT, FIB_ERR_RANGE, FIB_ERR_NO_PAGES = range(9)
FIB_DEBUG_SKIP_COPY, FIB_DEBUG_CORRUPT_TABLE = 1, 2
FIB_BASE_FIBONACCI, FIB_BASE_POW2, FIB_BASE_CUSTOM = 0, 1, 2
FIB_SCHED_FIXED, FIB_SCHED_LINEAR, FIB_SCHED_COPRIME = 0, 1, 2
FIB_MODE_MASK, FIB_MODE_INTERP = 0, 1
FIB_DTYPE_F32, FIB_DTYPE_BF16 = 0, 1
FIB_HEAD_DIM, FIB_MAX_RUNGS, FIB_MAX_WINDOW, FIB_MAX_LAYERS = 64, 32, 64, 256
FIB_MAX_DRAFTS, FIB_MAX_SEQS, FIB_MAX_HEADS = 64, 1024, 1024

EXPORTS = [
    "fib_attn_error_string", "fib_attn_base", "fib_attn_schedule", "fib_attn_mask_distances",
    "fib_attn_interp_rungs", "fib_attn_plan_create", "fib_attn_plan_destroy",
    "fib_attn_plan_distances", "fib_attn_fwd_workspace_size", "fib_attn_fwd",
    "fib_attn_fwd_prepare_kv", "fib_attn_fwd_attend", "fib_attn_bwd_workspace_size", "fib_attn_bwd",
    "fib_attn_debug_indices", "fib_attn_last_device_status", "fib_attn_plan_set_debug",
    "fib_attn_bwd_noalloc", "fib_attn_decode", "fib_attn_dense_fwd_workspace_size", "fib_attn_dense_fwd",
    "fib_attn_debug_fill_shared", "fib_attn_bwd_prepared", "fib_attn_cache_workspace_size",
    "fib_attn_cache_commit", "fib_attn_cache_fork", "fib_attn_cache_compact", "fib_attn_tree_decode",
    "fib_attn_dense_tree_workspace_size", "fib_attn_dense_tree_decode",
]

_i32p = ctypes.POINTER(ctypes.c_int32)
_f32p = ctypes.POINTER(ctypes.c_float)
_f64p = ctypes.POINTER(ctypes.c_double)
_vp = ctypes.c_void_p
_i = ctypes.c_int


class CacheStruct(ctypes.Structure):
    """fib_attn_cache of include/fib_attn.h."""
    _fields_ = [("dtype", _i), ("n_layers", _i), ("heads", _i), ("page_rows", _i), ("n_pages", _i),
                ("max_seqs", _i), ("max_pages", _i), ("device", _i), ("k", _vp), ("v", _vp), ("table", _vp),
                ("lens", _vp), ("refs", _vp), ("state", _vp)]


_cachep = ctypes.POINTER(CacheStruct)

_SIGS = {
    "fib_attn_error_string": (ctypes.c_char_p, [_i]),
    "fib_attn_base": (_i, [_i, _i, _i32p, _i, ctypes.POINTER(_i)]),
    "fib_attn_schedule": (_i, [_i, _i, _i, _f64p]),
    "fib_attn_mask_distances": (_i, [_i32p, _i, ctypes.c_double, _i, _i, _i32p, _i, ctypes.POINTER(_i)]),
    "fib_attn_interp_rungs": (_i, [_i32p, _i, ctypes.c_double, _i, _i, _i32p, _i32p, _f32p, _i,
                                   ctypes.POINTER(_i)]),
    "fib_attn_plan_create": (_i, [ctypes.POINTER(_vp), _i, _i32p, _i, _f64p, _i, _i, _i, _i, _i,
                                  ctypes.c_double]),
    "fib_attn_plan_destroy": (_i, [_vp]),
    "fib_attn_plan_distances": (_i, [_vp, _i, _i, _i32p, _i, ctypes.POINTER(_i)]),
    "fib_attn_fwd_workspace_size": (ctypes.c_size_t, [_vp, _i, _i, _i, _i]),
    "fib_attn_fwd_prepare_kv": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "fib_attn_fwd_attend": (_i, [_vp, _i, _i, _i, _i, _i, _vp, _vp, ctypes.c_size_t, _vp, _vp, _vp, _vp]),
    "fib_attn_fwd": (_i, [_vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                          _vp]),
    "fib_attn_bwd_workspace_size": (ctypes.c_size_t, [_vp, _i, _i, _i]),
    "fib_attn_bwd": (_i, [_vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                          _vp, _vp, ctypes.c_size_t, _vp]),
    "fib_attn_debug_indices": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp]),
    "fib_attn_last_device_status": (_i, [_vp]),
    "fib_attn_debug_fill_shared": (_i, [ctypes.c_uint32, _vp]),
    "fib_attn_plan_set_debug": (_i, [_vp, _i, ctypes.c_longlong]),
    "fib_attn_decode": (_i, [_vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fib_attn_dense_fwd_workspace_size": (ctypes.c_size_t, [_vp, _i, _i, _i, _i]),
    "fib_attn_dense_fwd": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "fib_attn_bwd_noalloc": (_i, [_vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                  _vp, _vp, _vp, _vp]),
    "fib_attn_bwd_prepared": (_i, [_vp, _i, _i, _i, _i, _i, _vp, _vp, ctypes.c_size_t, _vp, _vp, _vp, _vp,
                                   _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "fib_attn_cache_workspace_size": (ctypes.c_size_t, [_cachep]),
    "fib_attn_cache_commit": (_i, [_vp, _cachep, _i, _i, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "fib_attn_cache_fork": (_i, [_cachep, _vp, _vp, ctypes.c_size_t, _vp]),
    "fib_attn_cache_compact": (_i, [_cachep, _vp, _vp, ctypes.c_size_t, _vp]),
    "fib_attn_tree_decode": (_i, [_vp, _i, _cachep, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fib_attn_dense_tree_workspace_size": (ctypes.c_size_t, [_vp, _cachep, _i, _i, _i]),
    "fib_attn_dense_tree_decode": (_i, [_vp, _i, _cachep, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                        ctypes.c_size_t, _vp]),
}

_lib = None


class FibAttnError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {error_string(code)} (status {code})")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load libfibattn.so (built in-tree by build.py); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


def error_string(code: int) -> str:
    return lib().fib_attn_error_string(int(code)).decode()


def _check(fn: str, code: int):
    if code != FIB_OK:
        raise FibAttnError(fn, code)


def _arr(ctype, values):
    a = (ctype * max(1, len(values)))(*values)
    return a


# ----------------------------------------------------------------------- host-only planner
def fib_attn_base(base_kind: int, N: int = 2) -> list[int]:
    n = _i(0)
    _check("fib_attn_base", lib().fib_attn_base(base_kind, N, None, 0, ctypes.byref(n)))
    out = (ctypes.c_int32 * max(1, n.value))()
    _check("fib_attn_base", lib().fib_attn_base(base_kind, N, out, n.value, ctypes.byref(n)))
    return list(out[: n.value])


def fib_attn_schedule(kind: int, n_layers: int, stride: int = 7) -> list[float]:
    out = (ctypes.c_double * n_layers)()
    _check("fib_attn_schedule", lib().fib_attn_schedule(kind, n_layers, stride, out))
    return list(out)


def fib_attn_mask_distances(base, alpha: float, W: int, N: int) -> list[int]:
    b = _arr(ctypes.c_int32, list(base))
    cap = FIB_MAX_RUNGS * 4
    out = (ctypes.c_int32 * cap)()
    n = _i(0)
    _check("fib_attn_mask_distances", lib().fib_attn_mask_distances(
        b, len(base), float(alpha), W, N, out, cap, ctypes.byref(n)))
    return list(out[: min(n.value, cap)])


def fib_attn_interp_rungs(base, alpha: float, W: int, N: int):
    b = _arr(ctypes.c_int32, list(base))
    cap = FIB_MAX_RUNGS * 4
    f, lo, w = (ctypes.c_int32 * cap)(), (ctypes.c_int32 * cap)(), (ctypes.c_float * cap)()
    n = _i(0)
    _check("fib_attn_interp_rungs", lib().fib_attn_interp_rungs(
        b, len(base), float(alpha), W, N, f, lo, w, cap, ctypes.byref(n)))
    return [(f[r], lo[r], w[r]) for r in range(min(n.value, cap))]


# ----------------------------------------------------------------------------- plan
class Plan:
    """Owns a fib_attn_plan_t (destroyed with the object)."""

    def __init__(self, handle, n_layers, W, N_max, mode, device):
        self.handle, self.n_layers, self.W, self.N_max, self.mode = handle, n_layers, W, N_max, mode
        self.device = device

    def close(self):
        if self.handle:
            lib().fib_attn_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def fib_attn_plan_create(base_kind: int, alpha, W: int, N_max: int, mode: int,
                         custom_base=None, D: int = 64, rope_base: float = 10000.0) -> Plan:
    alpha = [float(a) for a in alpha]
    cb = list(custom_base) if custom_base is not None else []
    h = _vp()
    _check("fib_attn_plan_create", lib().fib_attn_plan_create(
        ctypes.byref(h), base_kind, _arr(ctypes.c_int32, cb) if cb else None, len(cb),
        _arr(ctypes.c_double, alpha), len(alpha), W, N_max, D, mode, float(rope_base)))
    return Plan(h, len(alpha), W, N_max, mode, torch.cuda.current_device())


def fib_attn_plan_distances(plan: Plan, layer: int, N: int) -> list[int]:
    out = (ctypes.c_int32 * FIB_MAX_RUNGS)()
    n = _i(0)
    _check("fib_attn_plan_distances", lib().fib_attn_plan_distances(
        plan.handle, layer, N, out, FIB_MAX_RUNGS, ctypes.byref(n)))
    return list(out[: n.value])


# ---------------------------------------------------------------------------- device ops
_DT = {torch.float32: FIB_DTYPE_F32, torch.bfloat16: FIB_DTYPE_BF16}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _shape(q):
    if q.dim() != 4 or q.shape[-1] != FIB_HEAD_DIM:
        raise ValueError("expected [B, H, N, 64]")
    for t in (q,):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")
    return q.shape[0], q.shape[1], q.shape[2]


def _same(q, *ts):
    for t in ts:
        if t is not None and (t.shape != q.shape or t.dtype != q.dtype or not t.is_cuda
                              or not t.is_contiguous()):
            raise ValueError("q/k/v/o/dO/dq/dk/dv must share shape, dtype and be contiguous CUDA")


def fib_attn_fwd_workspace_size(plan: Plan, B: int, H: int, N: int, dtype) -> int:
    return int(lib().fib_attn_fwd_workspace_size(plan.handle, B, H, N, _DT.get(dtype, dtype)))


def fib_attn_fwd(plan: Plan, layer: int, q, k, v, o=None, lse=None, alpha_dev=None,
                 want_lse: bool = True, workspace=None, stream=None):
    """Returns (o, lse).  o/lse and the workspace are allocated (by torch) when not given."""
    B, H, N = _shape(q)
    _same(q, k, v, o)
    if o is None:
        o = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    need = fib_attn_fwd_workspace_size(plan, B, H, N, q.dtype)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("fib_attn_fwd", lib().fib_attn_fwd(
        plan.handle, layer, B, H, N, _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
        _ptr(alpha_dev), _ptr(workspace), ws_bytes, _stream(stream)))
    return o, lse


def fib_attn_fwd_prepare_kv(plan: Plan, k, v, workspace=None, stream=None):
    """K rotated at its own positions and V, as float16, into a workspace (allocated by torch
    when not given), for fib_attn_fwd_attend; returns the workspace."""
    B, H, N = _shape(k)
    _same(k, v)
    need = fib_attn_fwd_workspace_size(plan, B, H, N, k.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=k.device)
    _check("fib_attn_fwd_prepare_kv", lib().fib_attn_fwd_prepare_kv(
        plan.handle, B, H, N, _DT[k.dtype], _ptr(k), _ptr(v), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return workspace


def fib_attn_fwd_attend(plan: Plan, layer: int, q, workspace, o=None, lse=None, alpha_dev=None,
                        want_lse: bool = True, stream=None):
    """Attention of q against a workspace filled by fib_attn_fwd_prepare_kv; returns (o, lse)."""
    B, H, N = _shape(q)
    _same(q, o)
    if o is None:
        o = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check("fib_attn_fwd_attend", lib().fib_attn_fwd_attend(
        plan.handle, layer, B, H, N, _DT[q.dtype], _ptr(q), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(o), _ptr(lse), _ptr(alpha_dev),
        _stream(stream)))
    return o, lse


def fib_attn_dense_fwd(plan: Plan, q, k, v, o=None, lse=None, want_lse: bool = True, workspace=None,
                       stream=None):
    """Dense causal attention with the plan's RoPE (bf16); returns (o, lse)."""
    B, H, N = _shape(q)
    _same(q, k, v, o)
    if o is None:
        o = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    need = int(lib().fib_attn_dense_fwd_workspace_size(plan.handle, B, H, N, _DT[q.dtype]))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _check("fib_attn_dense_fwd", lib().fib_attn_dense_fwd(
        plan.handle, B, H, N, _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return o, lse


def fib_attn_decode(plan: Plan, layer: int, pos: int, q, k_cache, v_cache, o=None, lse=None,
                    alpha_dev=None, want_lse: bool = True, stream=None):
    """One token at position pos: q [B, H, 64], caches [B, H, N, 64]; returns (o, lse)."""
    if q.dim() != 3 or q.shape[-1] != FIB_HEAD_DIM or not q.is_cuda or not q.is_contiguous():
        raise ValueError("q must be a contiguous CUDA [B, H, 64] tensor")
    B, H, N = _shape(k_cache)
    _same(k_cache, v_cache)
    if q.shape[:2] != k_cache.shape[:2] or q.dtype != k_cache.dtype:
        raise ValueError("q and the caches must share B, H and dtype")
    o = torch.empty_like(q) if o is None else o
    if lse is None and want_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    _check("fib_attn_decode", lib().fib_attn_decode(
        plan.handle, layer, B, H, N, pos, _DT[q.dtype], _ptr(q), _ptr(k_cache), _ptr(v_cache),
        _ptr(o), _ptr(lse), _ptr(alpha_dev), _stream(stream)))
    return o, lse


# ------------------------------------------------------------------------ paged cache, tree decode
class Cache:
    """A paged key/value cache (fib_attn_cache): torch tensors and the struct that describes them.

    k, v: pools [n_layers, n_pages, heads, page_rows, 64]; table [max_seqs, max_pages], lens
    [max_seqs], refs [n_pages] and state [4], int32, are views of one tensor ``meta`` (a copy of
    it is a snapshot of everything but the rows)."""

    def __init__(self, k, v, meta, max_seqs, max_pages):
        self.k, self.v, self.meta = k, v, meta
        self.n_layers, self.n_pages, self.heads, self.page_rows = k.shape[:4]
        self.max_seqs, self.max_pages, self.dtype, self.device = max_seqs, max_pages, k.dtype, k.device
        at = _cache_meta(self.n_pages, max_seqs, max_pages)
        self.state, self.refs = meta[:4], meta[4:4 + self.n_pages]
        self.lens, self.table = meta[at[0]:at[0] + max_seqs], meta[at[1]:at[2]].view(max_seqs, max_pages)
        self.struct = CacheStruct(_DT[k.dtype], self.n_layers, self.heads, self.page_rows, self.n_pages, max_seqs,
                                  max_pages, k.device.index, k.data_ptr(), v.data_ptr(), self.table.data_ptr(),
                                  self.lens.data_ptr(), self.refs.data_ptr(), self.state.data_ptr())
        self.pointer, self.index = ctypes.pointer(self.struct), k.device.index


def _cache_meta(n_pages: int, max_seqs: int, max_pages: int):
    """(first of lens, first of table, end) in a cache's meta tensor; state and refs precede."""
    lens = 4 + n_pages
    return lens, lens + max_seqs, lens + max_seqs + max_seqs * max_pages


def fib_attn_cache_create(n_layers: int, heads: int, page_rows: int, n_pages: int, max_seqs: int, max_pages: int,
                          dtype, k=None, v=None, device="cuda") -> Cache:
    """An empty cache; its memory is allocated by torch, the pools only where not given."""
    shape = (n_layers, n_pages, heads, page_rows, FIB_HEAD_DIM)
    device = torch.device(device)
    if k is not None:
        device = k.device
    if device.type != "cuda":
        raise ValueError("the cache lives on a CUDA device")
    if dtype not in _DT:
        raise ValueError("the cache holds float32 or bfloat16")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    k = torch.zeros(shape, dtype=dtype, device=device) if k is None else k
    v = torch.zeros(shape, dtype=dtype, device=device) if v is None else v
    for t in (k, v):
        if tuple(t.shape) != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
            raise ValueError("k and v must be contiguous [n_layers, n_pages, heads, page_rows, 64] of dtype on one device")
    at = _cache_meta(n_pages, max_seqs, max_pages)
    meta = torch.zeros(at[2], dtype=torch.int32, device=device)
    meta[at[1]:] = -1
    c = Cache(k, v, meta, max_seqs, max_pages)
    if lib().fib_attn_cache_workspace_size(c.pointer) == 0:
        raise FibAttnError("fib_attn_cache_create", FIB_ERR_INVALID_ARG)
    return c


def fib_attn_cache_workspace_size(cache: Cache) -> int:
    return int(lib().fib_attn_cache_workspace_size(cache.pointer))


def fib_attn_cache_status(cache: Cache) -> int:
    """The status that the cache's calls recorded (synchronises), cleared."""
    st = int(cache.state[1].item())
    cache.state[1] = 0
    return st


# A decode step makes a few of the calls below a layer, each of a few microseconds on the GPU: their
# checks read each attribute of a tensor once, and addresses go to ctypes as plain integers.
def _bad(t, dtype, index) -> bool:
    """Whether t is not a contiguous `dtype` tensor on CUDA device `index`."""
    return t.dtype is not dtype or t.get_device() != index or not t.is_contiguous()


def _raw_stream(stream, index: int) -> int:
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _empty(cache: Cache, shape, dtype, stream, kept=True):
    """A new tensor that a call on `stream` (None: the current one) writes: memory of that stream, which nothing
    enqueued elsewhere still uses; where it is kept, the current stream's as well."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=cache.device)
    here = torch.cuda.current_stream(cache.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=cache.device)
    if kept:
        t.record_stream(here)
    return t


def _scratch(cache: Cache, workspace, need, stream):
    """(address, bytes) of the caller's workspace, or of one of need() bytes, and the tensor itself."""
    if workspace is None:
        workspace = _empty(cache, max(need(), 1), torch.uint8, stream, kept=False)
    elif workspace.get_device() != cache.index or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be contiguous, on {cache.device}")
    return workspace.data_ptr(), workspace.nbytes, workspace


def fib_attn_cache_commit(plan: Plan, cache: Cache, k_new, v_new, n_new, path=None, workspace=None, stream=None):
    """Sequence b gains n_new[b] rows, in every layer: k_new, v_new [n_layers, B, heads, T, 64] raw
    rows; n_new int32 [B]; path int32 [B, T], the nodes taken (None: the first ones)."""
    index, shape = cache.index, k_new.shape
    if len(shape) != 5 or v_new.shape != shape or shape[0] != cache.n_layers or shape[2] != cache.heads or \
            shape[4] != FIB_HEAD_DIM:
        raise ValueError("k_new and v_new must be [n_layers, B, heads, T, 64]")
    B, T = shape[1], shape[3]
    if _bad(k_new, cache.dtype, index) or _bad(v_new, cache.dtype, index):
        raise ValueError(f"k_new and v_new must be contiguous {cache.dtype} on {cache.device}")
    if n_new.shape != (B,) or _bad(n_new, torch.int32, index):
        raise ValueError(f"n_new must be int32 [B] on {cache.device}")
    if path is not None and (path.shape != (B, T) or _bad(path, torch.int32, index)):
        raise ValueError(f"path must be int32 [B, T] on {cache.device}")
    at, size, workspace = _scratch(cache, workspace, lambda: fib_attn_cache_workspace_size(cache), stream)
    code = lib().fib_attn_cache_commit(plan.handle, cache.pointer, B, T, n_new.data_ptr(), None if path is None else path.data_ptr(),
                                       k_new.data_ptr(), v_new.data_ptr(), at, size, _raw_stream(stream, index))
    if code:
        raise FibAttnError("fib_attn_cache_commit", code)


def fib_attn_cache_fork(cache: Cache, src, workspace=None, stream=None):
    """Sequence b becomes what sequence src[b] is now (int32 [max_seqs]; -1 ends it)."""
    if src.shape != (cache.max_seqs,) or _bad(src, torch.int32, cache.index):
        raise ValueError(f"src must be int32 [max_seqs] on {cache.device}")
    at, size, workspace = _scratch(cache, workspace, lambda: fib_attn_cache_workspace_size(cache), stream)
    code = lib().fib_attn_cache_fork(cache.pointer, src.data_ptr(), at, size, _raw_stream(stream, cache.index))
    if code:
        raise FibAttnError("fib_attn_cache_fork", code)


def fib_attn_cache_compact(cache: Cache, remap=None, workspace=None, stream=None):
    """Moves the pages in use to the lowest ids (their number: cache.state[2]); returns remap int32
    [n_pages], the new id of each page, -1 for a free one."""
    if remap is None:
        remap = _empty(cache, cache.n_pages, torch.int32, stream)
    elif remap.shape != (cache.n_pages,) or _bad(remap, torch.int32, cache.index):
        raise ValueError(f"remap must be int32 [n_pages] on {cache.device}")
    at, size, workspace = _scratch(cache, workspace, lambda: fib_attn_cache_workspace_size(cache), stream)
    code = lib().fib_attn_cache_compact(cache.pointer, remap.data_ptr(), at, size, _raw_stream(stream, cache.index))
    if code:
        raise FibAttnError("fib_attn_cache_compact", code)
    return remap


def _tree_tensors(cache: Cache, q, k_new, v_new, parent, n_nodes, o, lse, want_lse, stream):
    """Checks a tree decode's tensors; returns (B, Hq, T, o, lse) with the outputs allocated.  (Written out: each call of a
    helper costs as much as what it would check.)"""
    index, dtype = cache.index, cache.dtype
    shape = q.shape
    if len(shape) != 4 or shape[3] != FIB_HEAD_DIM:
        raise ValueError("q must be [B, Hq, T, 64]")
    B, Hq, T, _ = shape
    drafts = (B, cache.heads, T, FIB_HEAD_DIM)
    if k_new.shape != drafts or v_new.shape != drafts:
        raise ValueError("k_new and v_new must be [B, heads, T, 64]")
    if q.dtype is not dtype or k_new.dtype is not dtype or v_new.dtype is not dtype or q.get_device() != index or \
            k_new.get_device() != index or v_new.get_device() != index or \
            not (q.is_contiguous() and k_new.is_contiguous() and v_new.is_contiguous()):
        raise ValueError(f"q, k_new and v_new must be contiguous {dtype} on {cache.device}")
    if parent is not None and (parent.shape != (B, T) or parent.dtype is not torch.int32 or parent.get_device() != index or
                               not parent.is_contiguous()):
        raise ValueError(f"parent must be int32 [B, T] on {cache.device}")
    if n_nodes is not None and (n_nodes.shape != (B,) or n_nodes.dtype is not torch.int32 or n_nodes.get_device() != index or
                                not n_nodes.is_contiguous()):
        raise ValueError(f"n_nodes must be int32 [B] on {cache.device}")
    if o is None:
        o = _empty(cache, shape, dtype, stream)
    elif o.shape != shape or o.dtype is not dtype or o.get_device() != index or not o.is_contiguous():
        raise ValueError(f"o must be like q, on {cache.device}")
    if lse is not None:
        if lse.shape != (B, Hq, T) or lse.dtype is not torch.float32 or lse.get_device() != index or not lse.is_contiguous():
            raise ValueError(f"lse must be float32 [B, Hq, T] on {cache.device}")
    elif want_lse:
        lse = _empty(cache, (B, Hq, T), torch.float32, stream)
    return B, Hq, T, o, lse


def fib_attn_tree_decode(plan: Plan, layer: int, cache: Cache, q, k_new, v_new, parent=None, n_nodes=None, o=None,
                         lse=None, N=None, alpha_dev=None, want_lse: bool = True, stream=None):
    """A tree of drafted tokens over the cache, the layer's window and rungs: q [B, Hq, T, 64], k_new
    and v_new [B, heads, T, 64]; parent int32 [B, T] (None: a chain), n_nodes int32 [B] (None: T);
    N: as in fib_attn_fwd (None: the plan's N_max).  Returns (o, lse)."""
    B, Hq, T, o, lse = _tree_tensors(cache, q, k_new, v_new, parent, n_nodes, o, lse, want_lse, stream)
    if alpha_dev is not None and (alpha_dev.numel() < plan.n_layers or _bad(alpha_dev, torch.float32, cache.index)):
        raise ValueError(f"alpha_dev must be float32 [n_layers] on {cache.device}")
    code = lib().fib_attn_tree_decode(
        plan.handle, layer, cache.pointer, B, Hq, T, plan.N_max if N is None else N, q.data_ptr(), k_new.data_ptr(),
        v_new.data_ptr(), None if parent is None else parent.data_ptr(), None if n_nodes is None else n_nodes.data_ptr(),
        o.data_ptr(), None if lse is None else lse.data_ptr(), None if alpha_dev is None else alpha_dev.data_ptr(),
        _raw_stream(stream, cache.index))
    if code:
        raise FibAttnError("fib_attn_tree_decode", code)
    return o, lse


def fib_attn_dense_tree_workspace_size(plan: Plan, cache: Cache, B: int, Hq: int, T: int) -> int:
    return int(lib().fib_attn_dense_tree_workspace_size(plan.handle, cache.pointer, B, Hq, T))


def fib_attn_dense_tree_decode(plan: Plan, layer: int, cache: Cache, q, k_new, v_new, parent=None, n_nodes=None,
                               o=None, lse=None, want_lse: bool = True, workspace=None, stream=None):
    """fib_attn_tree_decode for the dense control: every cached row, the ancestors, the node itself."""
    B, Hq, T, o, lse = _tree_tensors(cache, q, k_new, v_new, parent, n_nodes, o, lse, want_lse, stream)
    at, size, workspace = _scratch(cache, workspace,
                                   lambda: fib_attn_dense_tree_workspace_size(plan, cache, B, Hq, T), stream)
    code = lib().fib_attn_dense_tree_decode(
        plan.handle, layer, cache.pointer, B, Hq, T, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
        None if parent is None else parent.data_ptr(), None if n_nodes is None else n_nodes.data_ptr(), o.data_ptr(),
        None if lse is None else lse.data_ptr(), at, size, _raw_stream(stream, cache.index))
    if code:
        raise FibAttnError("fib_attn_dense_tree_decode", code)
    return o, lse


def fib_attn_bwd_workspace_size(plan: Plan, B: int, H: int, N: int) -> int:
    return int(lib().fib_attn_bwd_workspace_size(plan.handle, B, H, N))


def fib_attn_bwd(plan: Plan, layer: int, q, k, v, o, lse, dO, dq=None, dk=None, dv=None,
                 dalpha=None, alpha_dev=None, workspace=None, stream=None):
    """Returns (dq, dk, dv, dalpha[1])."""
    B, H, N = _shape(q)
    _same(q, k, v, o, dO, dq, dk, dv)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    if dalpha is None:
        dalpha = torch.empty(1, dtype=torch.float32, device=q.device)
    need = fib_attn_bwd_workspace_size(plan, B, H, N)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check("fib_attn_bwd", lib().fib_attn_bwd(
        plan.handle, layer, B, H, N, _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
        _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dalpha), _ptr(alpha_dev), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return dq, dk, dv, dalpha


def fib_attn_bwd_prepared(plan: Plan, layer: int, q, kv_prepared, o, lse, dO, dq=None, dk=None, dv=None,
                          dalpha=None, alpha_dev=None, workspace=None, stream=None):
    """Backward from the forward's prepared K'/V' rows (the uint8 workspace that
    fib_attn_fwd or fib_attn_fwd_prepare_kv filled for this layer's k and v): returns
    (dq, dk, dv, dalpha[1]), those of fib_attn_bwd up to the float16 rounding of K'."""
    B, H, N = _shape(q)
    _same(q, o, dO, dq, dk, dv)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    if dalpha is None:
        dalpha = torch.empty(1, dtype=torch.float32, device=q.device)
    need = fib_attn_bwd_workspace_size(plan, B, H, N)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check("fib_attn_bwd_prepared", lib().fib_attn_bwd_prepared(
        plan.handle, layer, B, H, N, _DT[q.dtype], _ptr(q), _ptr(kv_prepared),
        kv_prepared.numel() * kv_prepared.element_size(), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk),
        _ptr(dv), _ptr(dalpha), _ptr(alpha_dev), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return dq, dk, dv, dalpha


def fib_attn_bwd_noalloc(plan: Plan, layer: int, q, k, v, o, lse, dO, dq, dk, dv, dalpha,
                         alpha_dev=None, stream=None):
    """Backward into caller-provided dq, dk, dv, dalpha[1] with the library's fixed scratch
    array: no workspace argument and nothing allocated (for callers that may not allocate)."""
    B, H, N = _shape(q)
    _same(q, k, v, o, dO, dq, dk, dv)
    _check("fib_attn_bwd_noalloc", lib().fib_attn_bwd_noalloc(
        plan.handle, layer, B, H, N, _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
        _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dalpha), _ptr(alpha_dev), _stream(stream)))
    return dq, dk, dv, dalpha


def fib_attn_debug_indices(plan: Plan, layer: int, N: int, i_begin: int, i_end: int,
                           alpha_dev=None, stream=None):
    """Returns (rows int32 [(i_end-i_begin), W + 32] with -1 padding, w float32 [32])."""
    out = torch.empty((i_end - i_begin, plan.W + FIB_MAX_RUNGS), dtype=torch.int32, device="cuda")
    w = torch.empty(FIB_MAX_RUNGS, dtype=torch.float32, device="cuda")
    _check("fib_attn_debug_indices", lib().fib_attn_debug_indices(
        plan.handle, layer, N, i_begin, i_end, _ptr(out), _ptr(w), _ptr(alpha_dev), _stream(stream)))
    return out, w


def fib_attn_plan_set_debug(plan: Plan, skip_first_rung_copy: bool, wait_ns: int,
                            corrupt_table: bool = False):
    flags = (FIB_DEBUG_SKIP_COPY if skip_first_rung_copy else 0) | \
        (FIB_DEBUG_CORRUPT_TABLE if corrupt_table else 0)
    _check("fib_attn_plan_set_debug", lib().fib_attn_plan_set_debug(plan.handle, flags, int(wait_ns)))


def fib_attn_debug_fill_shared(pattern: int, stream=None):
    """Test hook: fill every SM's shared memory with a 32-bit pattern (stale contents for the
    kernels launched next)."""
    _check("fib_attn_debug_fill_shared", lib().fib_attn_debug_fill_shared(int(pattern) & 0xffffffff, _stream(stream)))


def fib_attn_last_device_status(plan: Plan) -> int:
    return int(lib().fib_attn_last_device_status(plan.handle))
