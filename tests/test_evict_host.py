"""Eviction and weighing, what needs no GPU: argument checks, and the oracle's eviction on a case written out."""
import ctypes

import numpy as np
import pytest

from fibonacci_offset_sparse_gb300 import fib_attn as fa
from oracle import cache_oracle as co
from tests.test_cache_host import BAD, lib, struct  # noqa: F401


@pytest.mark.parametrize("kw", BAD, ids=[str(x) for x in BAD])
def test_struct_rules(lib, kw):  # noqa: F811
    p = ctypes.byref(struct(**kw))
    assert lib.fib_attn_cache_evict_workspace_size(p, 100) == 0
    assert lib.fib_attn_cache_evict(1 << 12, p, 1, 100, 16, 0, 0, 32, None, 256, 1 << 40, None) == fa.FIB_ERR_INVALID_ARG


def test_evict_arguments(lib):  # noqa: F811
    s = struct()
    p = ctypes.byref(s)
    need = lib.fib_attn_cache_evict_workspace_size(p, 100)
    assert need > 0 and lib.fib_attn_cache_evict_workspace_size(p, 0) == 0 and lib.fib_attn_cache_evict_workspace_size(None, 1) == 0
    assert lib.fib_attn_cache_evict(None, p, 1, 100, 16, 0, 0, 32, None, 256, need, None) == fa.FIB_ERR_INVALID_ARG
    plan = 1 << 12  # never looked into: each call is refused for another argument
    good = dict(B=1, rows=100, keep=16, sink=0, recent=0, weights=32, dropped=None, ws=256, size=need)
    for kw in (dict(B=0), dict(B=4), dict(rows=0), dict(rows=(1 << 30) + 1), dict(keep=None), dict(keep=18), dict(sink=-1), dict(recent=-1),
               dict(recent=(1 << 29) + 1), dict(weights=None), dict(weights=34), dict(dropped=17), dict(dropped=16), dict(dropped=s.lens),
               dict(dropped=s.refs), dict(ws=None), dict(ws=272), dict(size=need - 1), dict(weights=256)):
        x = {**good, **kw}
        assert lib.fib_attn_cache_evict(plan, p, x["B"], x["rows"], x["keep"], x["sink"], x["recent"], x["weights"], x["dropped"], x["ws"],
                                        x["size"], None) == fa.FIB_ERR_INVALID_ARG, kw


def test_oracle_evicts_as_written():
    """Two sequences of two pages of 4 rows that share the first page; one layer, one head of two dims."""
    k = np.arange(5 * 4 * 2, dtype=np.float64).reshape(1, 5, 1, 4, 2)
    c = co.PagedCache(k.copy(), k.copy() + 100, [[0, 1], [0, 2]], [7, 6], [2, 1, 1, 0, 0])
    w = np.array([[[[9, 1, 5, 5, 2, 7, 0, 3]], [[0, 0, 0, 0, 0, 0, 0, 0]]]], np.float32)
    dropped = [0, 0]
    assert c.evict(w, [4, 6], 1, 1, dropped, turns=False)
    # rows 0 (first), 6 (last), 5 (weight 7) and 2 (5, the first of two) stay, in the first free page, as the old one is shared
    assert c.table == [[3, -1], [0, 2]] and c.lens == [4, 6] and c.refs == [1, 0, 1, 1, 0] and dropped == [3, 0]
    assert np.array_equal(c.k[0, 3, 0], [k[0, 0, 0, 0], k[0, 0, 0, 2], k[0, 1, 0, 1], k[0, 1, 0, 2]])
    assert np.array_equal(c.v[0, 3, 0], c.k[0, 3, 0] + 100)
    assert w[0, 0, 0].tolist() == [9, 5, 7, 0, 2, 7, 0, 3]


def test_weigh_arguments(lib):  # noqa: F811
    s = struct()
    p = ctypes.byref(s)
    need = lib.fib_attn_cache_weigh_workspace_size(p, 2, 8, 3)
    assert need > 0 and lib.fib_attn_cache_weigh_workspace_size(None, 2, 8, 3) == 0
    assert lib.fib_attn_cache_weigh(None, p, 2, 8, 3, 100, 16, None, None, 16, 16, 32, 256, need, None) == fa.FIB_ERR_INVALID_ARG
    good = dict(B=2, Hq=8, T=3, rows=100, n=16, path=None, first=None, q=512, lse=16, w=32, ws=256, size=need)
    for kw in (dict(B=0), dict(B=4), dict(Hq=0), dict(Hq=6), dict(Hq=1028), dict(T=0), dict(T=(1 << 20) + 1), dict(rows=0), dict(n=None), dict(n=18),
               dict(path=18), dict(first=17), dict(q=None), dict(q=520), dict(lse=None), dict(lse=18), dict(w=None), dict(w=33), dict(w=16),
               dict(ws=None), dict(ws=264), dict(size=need - 1), dict(q=256), dict(lse=256), dict(w=256)):
        x = {**good, **kw}
        assert lib.fib_attn_cache_weigh(1 << 12, p, x["B"], x["Hq"], x["T"], x["rows"], x["n"], x["path"], x["first"], x["q"], x["lse"], x["w"],
                                        x["ws"], x["size"], None) == fa.FIB_ERR_INVALID_ARG, kw
    huge = ctypes.byref(struct(n_layers=256, max_seqs=1024, heads=1024, page_rows=16, n_pages=1))
    assert lib.fib_attn_cache_weigh_workspace_size(huge, 1024, 1024, 65) == 0  # 2^40 values of queries at most
    assert lib.fib_attn_cache_weigh_workspace_size(huge, 1024, 1024, 64) > 1 << 40
    with_bad = ctypes.byref(struct(heads=0))
    assert lib.fib_attn_cache_weigh_workspace_size(with_bad, 2, 8, 3) == 0
    assert lib.fib_attn_cache_weigh(1 << 12, with_bad, 2, 8, 3, 100, 16, None, None, 512, 16, 32, 256, need, None) == fa.FIB_ERR_INVALID_ARG


def test_oracle_weighs_as_written():
    """One layer, one head of two dims at rest (no rotation); three rows, of which the last two are new."""
    k = np.array([[2.0, 0.0], [0.0, 2.0], [1.0, 1.0], [9.0, 9.0]]).reshape(1, 1, 1, 4, 2)
    c = co.PagedCache(k, k, [[0]], [3], [1])
    w = np.array([[[[10.0, 20.0, 30.0, 40.0]]]])
    q = np.array([[1.0, 0.0], [0.0, 1.0]]).reshape(1, 1, 1, 2, 2)
    c.weigh(w, q, np.zeros((1, 1, 1, 2)), [2], turns=False)
    e = np.exp(np.array([2.0, 0.0, 1.0]) / np.sqrt(2)), np.exp(np.array([0.0, 2.0, 1.0]) / np.sqrt(2))
    assert np.allclose(w[0, 0, 0], [10 + e[0][0] + e[1][0], e[0][1] + e[1][1], e[1][2], 40.0], rtol=1e-14)
