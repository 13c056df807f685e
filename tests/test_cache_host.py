"""The paged cache's argument checks that need no GPU: a struct that breaks the rules, null and
misaligned pointers and short workspaces are refused before any device call."""
import ctypes

import pytest

from fibonacci_offset_sparse_gb300 import fib_attn as fa


@pytest.fixture(scope="module")
def lib():
    import os
    from fibonacci_offset_sparse_gb300 import build as b
    srcs = [os.path.join(b.CSRC, s) for s in os.listdir(b.CSRC)]
    if not os.path.exists(b.LIB) or os.path.getmtime(b.LIB) < max(os.path.getmtime(s) for s in srcs):
        b.build()
    return fa.lib()


def struct(**kw):
    """A valid description of memory that no call here reaches."""
    x = dict(dtype=fa.FIB_DTYPE_BF16, n_layers=2, heads=4, page_rows=64, n_pages=10, max_seqs=3, max_pages=5, device=0,
             k=1 << 20, v=2 << 20, table=3 << 20, lens=4 << 20, refs=5 << 20, state=6 << 20)
    x.update(kw)
    return fa.CacheStruct(*[x[f] for f, _ in fa.CacheStruct._fields_])


BAD = [dict(dtype=2), dict(n_layers=0), dict(n_layers=257), dict(heads=0), dict(heads=1025), dict(page_rows=8),
       dict(page_rows=48), dict(page_rows=512), dict(page_rows=0), dict(n_pages=0), dict(max_seqs=0),
       dict(max_seqs=1025), dict(max_pages=0), dict(max_pages=(1 << 24) + 1), dict(n_pages=(1 << 23)), dict(k=None), dict(v=None),
       dict(k=(1 << 20) + 8), dict(v=1 << 20), dict(table=None), dict(table=(3 << 20) + 2), dict(lens=None),
       dict(refs=None), dict(refs=(5 << 20) + 4), dict(state=None), dict(state=(6 << 20) + 4)]


@pytest.mark.parametrize("kw", BAD, ids=[str(x) for x in BAD])
def test_struct_rules(lib, kw):
    s = struct(**kw)
    p = ctypes.byref(s)
    assert lib.fib_attn_cache_workspace_size(p) == 0
    assert lib.fib_attn_cache_fork(p, 7 << 20, 8 << 20, 1 << 30, None) == fa.FIB_ERR_INVALID_ARG
    assert lib.fib_attn_cache_compact(p, 7 << 20, 8 << 20, 1 << 30, None) == fa.FIB_ERR_INVALID_ARG


def test_null_struct_and_plan(lib):
    s = struct()
    assert lib.fib_attn_cache_workspace_size(None) == 0
    assert lib.fib_attn_cache_workspace_size(ctypes.byref(s)) > 0
    assert lib.fib_attn_cache_fork(None, 7 << 20, 8 << 20, 1 << 30, None) == fa.FIB_ERR_INVALID_ARG
    p = ctypes.byref(s)
    assert lib.fib_attn_cache_commit(None, p, 1, 1, 16, None, 16, 16, 256, 1 << 30, None) == fa.FIB_ERR_INVALID_ARG
    assert lib.fib_attn_tree_decode(None, 0, p, 1, 4, 1, 10, 16, 16, 16, None, None, 32, None, None,
                                    None) == fa.FIB_ERR_INVALID_ARG
    assert lib.fib_attn_dense_tree_decode(None, 0, p, 1, 4, 1, 16, 16, 16, None, None, 32, None, 256, 1 << 30,
                                          None) == fa.FIB_ERR_INVALID_ARG
    assert lib.fib_attn_dense_tree_workspace_size(None, p, 1, 4, 1) == 0


def test_fork_and_compact_arguments(lib):
    s = struct()
    p = ctypes.byref(s)
    need = lib.fib_attn_cache_workspace_size(p)
    for fn in (lib.fib_attn_cache_fork, lib.fib_attn_cache_compact):
        assert fn(p, None, 8 << 20, need, None) == fa.FIB_ERR_INVALID_ARG
        assert fn(p, (7 << 20) + 2, 8 << 20, need, None) == fa.FIB_ERR_INVALID_ARG
        assert fn(p, 7 << 20, None, need, None) == fa.FIB_ERR_INVALID_ARG
        assert fn(p, 7 << 20, (8 << 20) + 16, need, None) == fa.FIB_ERR_INVALID_ARG
        assert fn(p, 7 << 20, 8 << 20, need - 1, None) == fa.FIB_ERR_INVALID_ARG
        assert fn(p, s.lens, 8 << 20, need, None) == fa.FIB_ERR_INVALID_ARG
        assert fn(p, s.table, 8 << 20, need, None) == fa.FIB_ERR_INVALID_ARG
    assert lib.fib_attn_cache_compact(p, s.refs, 8 << 20, need, None) == fa.FIB_ERR_INVALID_ARG


def test_status_name(lib):
    assert fa.error_string(fa.FIB_ERR_NO_PAGES) not in ("unknown status", "")


def test_cache_needs_a_gpu_device():
    with pytest.raises(ValueError):
        import torch
        fa.fib_attn_cache_create(1, 1, 16, 4, 1, 2, torch.float32, device="cpu")
