"""The paged cache and the tree decodes over it against the float64 oracle (needs a GPU).

Tolerances.  Whole numbers are equal.  A stored K row is the rotation in float32 (an error of a few
2^-24 of the row's size, below 1e-5 for |x| < 8) rounded once to the cache's type, half a step: 2^-24
(float32) or 2^-8 (bf16) of the value.  V is copied.  A decode takes the cache's rows as they stand;
its scores are sums of 64 float32 products of size |q||k|/8 whose rounding and rotation errors of
2^-24 each (some 8 of them a product, of random sign) leave about sqrt(64 * 8) 2^-24 = 1.4e-6 and at most 3e-5,
which moves a softmax weight by as much relatively and an output by at most twice that times the
largest value (5): 3e-4 at worst, 1.4e-5 as a rule; ten standard errors, 1.5e-4, are allowed.  A bf16
output adds half a step, 2^-8 of it.
"""
import os

import numpy as np
import pytest
import torch

import oracle
from fibonacci_offset_sparse_gb300 import fib_attn as fa
from fibonacci_offset_sparse_gb300 import inputs
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TOL_O, TOL_LSE = 1.5e-4, 3e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fibonacci_offset_sparse_gb300 import build as b
    if not os.path.exists(b.LIB):
        b.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return fa.lib()


def rng(*seed):
    return np.random.default_rng([20261202, 60, *seed])


def draw(r, shape, dtype):
    """N(0, 1) on the GPU in `dtype`, and the same values in float64."""
    t = torch.from_numpy(r.standard_normal(shape).astype(np.float32)).to(DT[dtype])
    return t.cuda(), t.double().numpy()


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


def make_cache(r, dtype, L, H, P, lens, max_pages, spare=4, share=()):
    """A cache whose sequences hold randomly placed pages of random rows, and its oracle.  share:
    (b, a, pages): sequence b's first pages are sequence a's."""
    S = len(lens)
    used = [-(-n // P) for n in lens]
    NP = sum(used) + spare
    ids = r.permutation(NP).tolist()
    table = np.full((S, max_pages), -1)
    for b in range(S):
        for j in range(used[b]):
            table[b, j] = ids.pop()
    for b, a, pages in share:
        table[b, :pages] = table[a, :pages]
    refs = np.zeros(NP, int)
    for b in range(S):
        for j in range(used[b]):
            refs[table[b, j]] += 1
    k, kf = draw(r, (L, NP, H, P, 64), dtype)
    v, vf = draw(r, (L, NP, H, P, 64), dtype)
    c = fa.fib_attn_cache_create(L, H, P, NP, S, max_pages, DT[dtype], k=k, v=v)
    c.table.copy_(i32(table))
    c.lens.copy_(i32(lens))
    c.refs.copy_(i32(refs))
    return c, co.PagedCache(kf, vf, table, lens, refs)


def same_tables(c, ref):
    assert c.table.cpu().tolist() == ref.table
    assert c.lens.cpu().tolist() == ref.lens
    assert c.refs.cpu().tolist() == ref.refs


def close_rows(c, ref, dtype):
    k, v = c.k.double().cpu().numpy(), c.v.double().cpu().numpy()
    assert np.array_equal(v, ref.v)
    assert np.all(np.abs(k - ref.k) <= 1e-5 + HALF[dtype] * np.abs(ref.k))


def plan_for(N=4096, W=8, alpha=(1.0, 1.0, 1.0), mode=fa.FIB_MODE_MASK, base=fa.FIB_BASE_FIBONACCI):
    return fa.fib_attn_plan_create(base, list(alpha), W, N, mode)


# ------------------------------------------------------------------------------------ commit
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("P,H,T,lens,n_new,use_path", [
    (16, 1, 1, [0], [1], False),                                # the first token of an empty sequence
    (16, 3, 1, [15, 16, 17, 0], [1, 1, 1, 1], False),           # a page filled, opened, entered
    (64, 2, 70, [0, 63, 5], [70, 65, 0], False),                # prompts over several pages; one untouched
    (32, 5, 9, [31, 33, 64, 1], [9, 3, 0, 1], True),            # accepted paths
    (256, 1, 64, [200, 256], [64, 1], True),
    (16, 2, 130, [3, 0], [129, 130], False),                    # more than two chunks of tokens
])
def test_commit(dtype, P, H, T, lens, n_new, use_path):
    r = rng(1, P, T, H)
    L, B = 3, len(lens)
    most = max(n + T for n in lens)
    c, ref = make_cache(r, dtype, L, H, P, lens, -(-most // P) + 1, spare=sum(-(-n // P) + 1 for n in n_new))
    kn, kf = draw(r, (L, B, H, T, 64), dtype)
    vn, vf = draw(r, (L, B, H, T, 64), dtype)
    path = np.stack([r.permutation(T) for _ in range(B)]) if use_path else None
    plan = plan_for()
    fa.fib_attn_cache_commit(plan, c, kn, vn, i32(n_new), path=None if path is None else i32(path))
    assert ref.commit(kf, vf, n_new, path)
    same_tables(c, ref)
    close_rows(c, ref, dtype)
    assert fa.fib_attn_cache_status(c) == fa.FIB_OK
    plan.close()


@pytest.mark.parametrize("writers", [[1, 1, 1], [1, 0, 1], [0, 1, 0], [2, 3, 1], [0, 0, 0]])
@pytest.mark.parametrize("held", [0, 1])
def test_commit_copies_a_shared_last_page(writers, held):
    """Three sequences share their last, partly filled page; `held`: the caller holds it too."""
    r = rng(2, *writers, held)
    lens, P, L, H = [37, 37, 37, 20], 16, 2, 2
    c, ref = make_cache(r, "bf16", L, H, P, lens, 5, spare=9, share=[(1, 0, 3), (2, 0, 3)])
    page = ref.table[0][2]
    ref.refs[page] += held
    c.refs[page] += held
    T = 3
    kn, kf = draw(r, (L, 4, H, T, 64), "bf16")
    vn, vf = draw(r, (L, 4, H, T, 64), "bf16")
    n_new = writers + [1]
    plan = plan_for()
    fa.fib_attn_cache_commit(plan, c, kn, vn, i32(n_new))
    assert ref.commit(kf, vf, n_new)
    same_tables(c, ref)
    close_rows(c, ref, "bf16")
    assert c.refs[page].item() >= held
    plan.close()


@pytest.mark.parametrize("lens", [[18, 40, 25], [40, 18, 40], [47, 33, 34], [33, 34, 47]])
def test_commit_of_sequences_that_were_shortened(lens):
    """Holders of one page of different lengths all gain rows: the copies are of the page as it was."""
    r = rng(24, *lens)
    c, ref = make_cache(r, "f32", 2, 2, 16, [48, 48, 48], 6, share=[(1, 0, 3), (2, 0, 3)])
    for b, n in enumerate(lens):  # as a caller does that takes back rejected rows
        for j in range(ref.pages(n), ref.pages(48)):
            ref.refs[ref.table[b][j]] -= 1
            ref.table[b][j] = -1
        ref.lens[b] = n
    c.table.copy_(i32(ref.table))
    c.lens.copy_(i32(ref.lens))
    c.refs.copy_(i32(ref.refs))
    c.state[0] = 0
    kn, kf = draw(r, (2, 3, 2, 9, 64), "f32")
    vn, vf = draw(r, (2, 3, 2, 9, 64), "f32")
    fa.fib_attn_cache_commit(plan_for(), c, kn, vn, i32([9, 7, 9]))
    assert ref.commit(kf, vf, [9, 7, 9])
    same_tables(c, ref)
    close_rows(c, ref, "f32")


def test_commit_takes_the_lowest_free_pages_and_moves_its_bound():
    r = rng(3)
    P = 16
    c, ref = make_cache(r, "f32", 1, 1, P, [5, 0], 40, spare=6000)  # more counts than one step of the search
    kn, kf = draw(r, (1, 2, 1, 600, 64), "f32")
    vn, vf = draw(r, (1, 2, 1, 600, 64), "f32")
    c.refs[:5000] += 1  # pages that the caller holds
    ref.refs[:5000] = [x + 1 for x in ref.refs[:5000]]
    plan = plan_for()
    fa.fib_attn_cache_commit(plan, c, kn, vn, i32([600, 33]))
    assert ref.commit(kf, vf, [600, 33])
    same_tables(c, ref)
    close_rows(c, ref, "f32")
    cursor = c.state[0].item()
    assert 0 < cursor and (c.refs[:cursor] > 0).all()
    fa.fib_attn_cache_fork(c, i32([-1, 1]))  # freed pages lower it again
    ref.fork([-1, 1])
    same_tables(c, ref)
    cursor = c.state[0].item()
    assert (c.refs[:cursor] > 0).all()
    fa.fib_attn_cache_commit(plan, c, kn, vn, i32([17, 0]))
    assert ref.commit(kf, vf, [17, 0])
    same_tables(c, ref)
    plan.close()


def snapshot(c):
    return c.meta.clone(), c.k.clone(), c.v.clone()


def unchanged(c, before, status):
    assert fa.fib_attn_cache_status(c) == status
    meta, k, v = before
    c_meta = c.meta.clone()
    c_meta[1] = meta[1]
    assert torch.equal(c_meta, meta) and torch.equal(c.k, k) and torch.equal(c.v, v)


@pytest.mark.parametrize("what", ["pages", "n_new", "negative", "path", "table", "rope", "page id"])
def test_a_refused_commit_changes_nothing(what):
    r = rng(4)
    lens, P, L, H, T = [30, 16, 9], 16, 2, 1, 40
    c, ref = make_cache(r, "f32", L, H, P, lens, 4, spare=3)
    kn, _ = draw(r, (L, 3, H, T, 64), "f32")
    vn, _ = draw(r, (L, 3, H, T, 64), "f32")
    n_new, path, N, status = [2, 1, 1], None, 4096, fa.FIB_ERR_DEVICE_ASSERT
    if what == "pages":
        n_new, status = [30, 20, 2], fa.FIB_ERR_NO_PAGES  # 2 + 2 + 0 pages of 3
    elif what == "n_new":
        n_new = [2, 41, 1]
    elif what == "negative":
        n_new = [2, 1, -1]
    elif what == "path":
        path = np.zeros((3, T), int)
        path[1, 0] = T
    elif what == "table":
        n_new = [35, 1, 1]  # 65 rows in four pages of 16
    elif what == "rope":
        N = 31
    elif what == "page id":
        c.table[2, 0] = c.n_pages
    before = snapshot(c)
    plan = plan_for(N)
    fa.fib_attn_cache_commit(plan, c, kn, vn, i32(n_new), path=None if path is None else i32(path))
    torch.cuda.synchronize()
    unchanged(c, before, status)
    plan.close()


# ------------------------------------------------------------------------------- fork, compact
@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("S,P,most", [(1, 16, 5), (4, 16, 70), (33, 32, 1000), (300, 16, 40)])
def test_fork(seed, S, P, most):
    r = rng(5, seed, S)
    lens = r.integers(0, most, S).tolist()
    lens[0] = most
    c, ref = make_cache(r, "f32", 1, 1, P, lens, -(-most // P), spare=5)
    c.state[0] = 0
    for step in range(3):  # forks of forks: shared pages are freed by their last holder only
        src = r.integers(-1, S, S)
        src = np.where(r.random(S) < 0.3, np.arange(S), src).tolist()
        fa.fib_attn_cache_fork(c, i32(src))
        ref.fork(src)
        same_tables(c, ref)
        assert (c.refs[:c.state[0].item()] > 0).all()
    assert fa.fib_attn_cache_status(c) == fa.FIB_OK
    fa.fib_attn_cache_fork(c, i32([-1] * S))
    assert not c.refs.any() and not c.lens.any()


def test_a_refused_fork_changes_nothing():
    r = rng(6)
    for src, lens in (([0, 3, 1], [20, 5, 0]), ([0, -2, 1], [20, 5, 0]), ([0, 1, 1], [20, 5, 33]), ([1, 1, 1], [20, -1, 0])):
        c, ref = make_cache(r, "f32", 1, 1, 16, [20, 5, 0], 2)
        c.lens.copy_(i32(lens))
        before = snapshot(c)
        fa.fib_attn_cache_fork(c, i32(src))
        torch.cuda.synchronize()
        unchanged(c, before, fa.FIB_ERR_DEVICE_ASSERT)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,P,H,L,spare", [(1, 16, 1, 1, 0), (3, 16, 2, 2, 7), (9, 64, 3, 2, 40), (40, 16, 1, 1, 3000)])
def test_compact(dtype, S, P, H, L, spare):
    r = rng(7, S, P)
    lens = r.integers(0, 5 * P, S).tolist()
    c, ref = make_cache(r, dtype, L, H, P, lens, 5, spare=spare)
    src = [-1 if r.random() < 0.4 else b for b in range(S)]  # some end, one forks
    src[-1] = 0
    fa.fib_attn_cache_fork(c, i32(src))
    ref.fork(src)
    remap = fa.fib_attn_cache_compact(c)
    want, n = ref.compact()
    assert remap.cpu().tolist() == want
    same_tables(c, ref)
    k, v = c.k.double().cpu().numpy(), c.v.double().cpu().numpy()
    assert np.array_equal(k[:, :n], ref.k[:, :n]) and np.array_equal(v[:, :n], ref.v[:, :n])
    assert c.state[:3].tolist() == [n, fa.FIB_OK, n]
    assert (c.refs[:n] > 0).all() and not c.refs[n:].any()
    again = fa.fib_attn_cache_compact(c)  # nothing left to move
    assert again[:n].tolist() == list(range(n))
    same_tables(c, ref)


# ------------------------------------------------------------------------------- tree decodes
def keys_of(W, mode, base, alpha, N):
    b = oracle.fibonacci_base() if base == "fib" else oracle.pow2_base(N)
    if mode == "mask":
        return [(x, 0.0) for x in range(W)] + [(d, 0.0) for d in oracle.mask_distances(b, alpha, W, N)]
    return [(x, 0.0) for x in range(W)] + [(lo, float(w)) for _, lo, w in oracle.interp_rungs(b, alpha, W, N)]


def trees(r, kind, B, T):
    """parent [B, T]: chains, all roots, random."""
    if kind == "chain":
        return np.tile(np.arange(T) - 1, (B, 1))
    if kind == "roots":
        return np.full((B, T), -1)
    return np.stack([[int(r.integers(max(-1, s - 6), s)) if s else -1 for s in range(T)] for _ in range(B)])


CASES = [  # B's lengths, H, G, T, P, tree, live nodes
    ([0], 1, 1, 1, 16, None, None),
    ([1], 2, 1, 1, 16, None, None),
    ([1500], 2, 1, 1, 64, None, None),
    ([0, 1, 15, 16, 17, 333], 2, 1, 5, 16, "random", [5, 1, 5, 3, 0, 4]),
    ([100, 64, 1], 1, 3, 13, 64, "random", None),
    ([700, 3], 3, 2, 33, 32, "chain", [33, 17]),
    ([129, 300], 1, 1, 64, 128, "random", None),
    ([40, 1000], 2, 4, 64, 256, "roots", [64, 1]),
    ([2048, 63, 65], 1, 5, 7, 16, None, None),
    ([300, 17, 64], 20, 1, 64, 32, "random", [64, 50, 64]),     # enough rows for the sparse decode's tensor-core kernel
    ([90, 0, 1033, 5], 32, 3, 9, 16, "random", [9, 9, 8, 0]),
    ([5, 0, 77, 200, 16, 31, 64, 9], 32, 1, 12, 16, None, None),
    ([700, 129, 0], 2, 1, 24, 64, "random", [24, 17, 24]),      # each number of row tiles of the dense decode's
    ([128, 257], 1, 3, 16, 128, "random", [16, 11]),
]


def tree_case(r, dtype, lens, H, G, T, P, kind, nodes, poison=True):
    B = len(lens)
    c, ref = make_cache(r, dtype, 2, H, P, lens, max(1, -(-max(lens) // P)))
    q, qf = draw(r, (B, H * G, T, 64), dtype)
    kn, kf = draw(r, (B, H, T, 64), dtype)
    vn, vf = draw(r, (B, H, T, 64), dtype)
    parent = trees(r, kind or "chain", B, T)
    live = nodes or [T] * B
    if poison:  # what nobody attends: rows behind a sequence, free pages, padding
        bad = [float("nan"), float("inf"), -float("inf")]
        used = {}
        for b in range(B):
            for j in range(-(-lens[b] // P)):
                used[ref.table[b][j]] = min(P, lens[b] - j * P)
        for p in range(c.n_pages):
            c.k[:, p, :, used.get(p, 0):] = bad[p % 3]
            c.v[:, p, :, used.get(p, 0):] = bad[(p + 1) % 3]
        for b in range(B):
            kn[b, :, live[b]:] = bad[b % 3]
            vn[b, :, live[b]:] = bad[(b + 1) % 3]
            q[b, :, live[b]:] = float("nan")
    return c, ref, (q, kn, vn), (qf, kf, vf), parent, live


def check(o, lse, ref_o, ref_l, live, dtype):
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, n in enumerate(live):
        assert np.all(np.abs(o[b, :, :n] - ref_o[b, :, :n]) <= TOL_O + (HALF[dtype] * np.abs(ref_o[b, :, :n]) if dtype == "bf16" else 0))
        assert np.all(np.abs(lse[b, :, :n] - ref_l[b, :, :n]) <= TOL_LSE)
        assert np.all(o[b, :, n:] == 7) and np.all(lse[b, :, n:] == 7)  # left as they were


def sevens(q):
    return torch.full_like(q, 7), torch.full(q.shape[:3], 7.0, device=q.device)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mode,base,alpha,W", [("mask", "fib", 1.5, 12), ("interp", "fib", 0.9731, 10), ("interp", "pow2", 0.6, 1),
                                               ("mask", "pow2", 1.0, 64), ("interp", "fib", 1.0, 3)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_tree_decode(dtype, mode, base, alpha, W, case):
    r = rng(8, case, W)
    lens, H, G, T, P, kind, nodes = CASES[case]
    c, ref, dev, host, parent, live = tree_case(r, dtype, *CASES[case])
    N = max(lens) + T + 5
    m = fa.FIB_MODE_MASK if mode == "mask" else fa.FIB_MODE_INTERP
    plan = fa.fib_attn_plan_create(fa.FIB_BASE_FIBONACCI if base == "fib" else fa.FIB_BASE_POW2, [1.0, alpha], W, N + 100, m)
    o, lse = sevens(dev[0])
    fa.fib_attn_tree_decode(plan, 1, c, *dev, parent=None if kind is None else i32(parent),
                            n_nodes=None if nodes is None else i32(nodes), o=o, lse=lse, N=N)
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    check(o, lse, *co.tree_attend(ref, 1, *host, parent, live, keys_of(W, mode, base, alpha, N)), live, dtype)
    plan.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_dense_tree_decode(dtype, case):
    r = rng(9, case)
    lens, H, G, T, P, kind, nodes = CASES[case]
    c, ref, dev, host, parent, live = tree_case(r, dtype, *CASES[case])
    plan = plan_for(max(lens) + T)
    o, lse = sevens(dev[0])
    fa.fib_attn_dense_tree_decode(plan, 1, c, *dev, parent=None if kind is None else i32(parent),
                                  n_nodes=None if nodes is None else i32(nodes), o=o, lse=lse)
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    check(o, lse, *co.tree_attend(ref, 1, *host, parent, live), live, dtype)
    plan.close()


def both(plan, c, dev, **kw):
    """(name, o, lse) of the two decodes."""
    yield ("sparse", *fa.fib_attn_tree_decode(plan, 0, c, *dev, **kw))
    kw.pop("N", None)
    yield ("dense", *fa.fib_attn_dense_tree_decode(plan, 0, c, *dev, **kw))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_another_branch_never_reaches_a_node(dtype):
    """Two branches; one's rows are NaN and infinite, the other's nodes are as without them."""
    r = rng(10)
    c, ref, dev, host, _, _ = tree_case(r, dtype, [50], 2, 1, 8, 16, "chain", None)
    parent = np.asarray([[-1, 0, 0, 1, 2, 3, 4, 5]])  # 0, then 1-3-5-7 and 2-4-6
    plan = plan_for(64, W=4)
    clean = {name: (o.clone(), l.clone()) for name, o, l in both(plan, c, dev, parent=i32(parent))}
    q, kn, vn = (x.clone() for x in dev)
    for u, bad in ((2, float("nan")), (4, float("inf")), (6, -float("inf"))):
        kn[:, :, u] = bad
        vn[:, :, u] = bad
    for name, o, l in both(plan, c, (q, kn, vn), parent=i32(parent)):
        for s in (0, 1, 3, 5, 7):
            assert torch.equal(o[:, :, s], clean[name][0][:, :, s]), (name, s)
            assert torch.equal(l[:, :, s], clean[name][1][:, :, s]), (name, s)
        assert not torch.isfinite(o[:, :, 2]).any()
    plan.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G", [1, 3])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_another_branch_never_reaches_a_node_of_a_large_tree(dtype, G, bad):
    """As above, for as many query rows as the tensor-core kernels take; only v, only k, then both."""
    r = rng(20)
    T = 21
    c, ref, dev, host, _, _ = tree_case(r, dtype, [150, 0], 64, G, T, 32, "chain", None)
    parent = np.tile([-1] + [max(0, s - 2) for s in range(1, T)], (2, 1))  # 0, then the odd and the even nodes
    even = list(range(2, T, 2))
    odd = [0] + list(range(1, T, 2))
    plan = plan_for(200, W=4)
    clean = {name: (o.clone(), l.clone()) for name, o, l in both(plan, c, dev, parent=i32(parent))}
    for what in ("v", "k", "kv"):
        q, kn, vn = (x.clone() for x in dev)
        for u in (2, 10, 20):
            if "k" in what:
                kn[:, :, u, 3:9] = bad
            if "v" in what:
                vn[:, :, u, 7] = bad
        for name, o, l in both(plan, c, (q, kn, vn), parent=i32(parent)):
            assert torch.isfinite(o[:, :, odd]).all()
            # the path may be another one (the error then as against the oracle), the values are not
            assert (o[:, :, odd].float() - clean[name][0][:, :, odd].float()).abs().max().item() <= 2 * TOL_O + (2 * HALF[dtype] * 4 if dtype == "bf16" else 0)
            assert (l[:, :, odd] - clean[name][1][:, :, odd]).abs().max().item() <= 2 * TOL_LSE
            if bad != bad or "v" in what:
                assert not torch.isfinite(o[:, :, 20]).all()
    plan.close()


@pytest.mark.parametrize("mode,W,alpha", [("mask", 12, 1.1), ("interp", 30, 0.53), ("interp", 2, 0.5)])
@pytest.mark.parametrize("kind", ["chain", "random", "roots", "last first"])
@pytest.mark.parametrize("T,G", [(64, 1), (37, 2), (16, 5)])
def test_unions_of_keys_that_do_and_do_not_fit(mode, W, alpha, kind, T, G):
    """Trees of every depth over a base of close distances (several rungs read one row), bf16."""
    r = rng(21, T, W)
    lens = [500, 0, 30]
    c, ref, dev, host, parent, live = tree_case(r, "bf16", lens, 16, G, T, 16, "chain" if kind == "last first" else kind, [T, T - 1, T // 2])
    if kind == "last first":  # depths 0 .. T/2, then all at once back to the roots
        parent = np.tile([s - 1 if s <= T // 2 else -1 for s in range(T)], (3, 1))
    base = [1, 2, 3, 5, 20, 21, 22, 23, 24, 25, 40, 60, 61, 100, 150, 151, 152, 153, 300, 301, 400, 477, 499, 500]
    N = 700
    m = fa.FIB_MODE_MASK if mode == "mask" else fa.FIB_MODE_INTERP
    plan = fa.fib_attn_plan_create(fa.FIB_BASE_CUSTOM, [alpha], W, N, m, custom_base=base)
    o, lse = sevens(dev[0])
    fa.fib_attn_tree_decode(plan, 0, c, *dev, parent=i32(parent), n_nodes=i32(live), o=o, lse=lse)
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    if mode == "mask":
        keys = [(x, 0.0) for x in range(W)] + [(d, 0.0) for d in oracle.mask_distances(base, alpha, W, N)]
    else:
        keys = [(x, 0.0) for x in range(W)] + [(lo, float(w)) for _, lo, w in oracle.interp_rungs(base, alpha, W, N)]
    check(o, lse, *co.tree_attend(ref, 0, *host, parent, live, keys), live, "bf16")
    # a learned alpha on the device gives the same keys (exact in float32 where alpha is)
    if alpha == 0.5:
        o2, l2 = sevens(dev[0])
        fa.fib_attn_tree_decode(plan, 0, c, *dev, parent=i32(parent), n_nodes=i32(live), o=o2, lse=l2,
                                alpha_dev=torch.tensor([alpha], device="cuda"))
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    plan.close()


def test_an_infinite_key_that_is_attended():
    """A cached key whose scores are -inf weighs nothing; the other keys count as without it."""
    r = rng(11)
    c, ref, dev, host, parent, live = tree_case(r, "f32", [5], 1, 1, 1, 16, None, None)
    q, kn, vn = dev
    row = c.table[0, 0].item()
    for at in (0, 4):  # the first key a thread meets, and the last
        c.k[0, row, 0, at] = 0
        c.k[0, row, 0, at, 0] = float("inf")
    # position 5 turns dimension 0 of q into q0 cos 5 - q32 sin 5: make it negative
    a = 5.0
    if q[0, 0, 0, 0].item() * np.cos(a) - q[0, 0, 0, 32].item() * np.sin(a) > 0:
        q.neg_()
    ref.k[0, row, 0, [0, 4]] = 0
    plan = plan_for(64, W=6)
    keep = [1, 2, 3]
    qr = co.turn(q[0, 0, 0].double().cpu().numpy(), 5)
    ks = np.concatenate([ref.k[0, row, 0, keep], co.turn(kn[0, 0].double().cpu().numpy(), 5)])
    vs = np.concatenate([ref.v[0, row, 0, keep], vn[0, 0].double().cpu().numpy()])
    p = np.exp(ks @ qr / 8)
    for name, o, l in both(plan, c, dev):
        assert np.abs(o[0, 0, 0].double().cpu().numpy() - p @ vs / p.sum()).max() <= TOL_O, name
        assert abs(l.item() - np.log(p.sum())) <= TOL_LSE, name
    plan.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("T,H", [(1, 1), (8, 2), (9, 1), (24, 2), (40, 1), (64, 2), (64, 32)])
def test_infinite_cached_keys(dtype, sign, T, H):
    """A cached key whose dimension 0 is infinite scores +inf or -inf by the sign of the rotated query's dimension 0.
    A node all of whose such scores are -inf is as without these keys; one that meets +inf has no softmax."""
    r = rng(20, T, H)
    lens, W = [300, 150], 12
    c, ref, dev, host, parent, live = tree_case(r, dtype, lens, H, 1, T, 32, "roots", None, poison=False)
    bad = [[0, 140, 299, 297], [149, 31]]  # the last ones lie in the window of a tree of roots
    for b, rows in enumerate(bad):
        for x in rows:
            page = ref.table[b][x // 32]
            c.k[:, page, :, x % 32] = 0
            c.k[:, page, :, x % 32, 0] = sign * float("inf")
    N = 400
    plan = plan_for(N, W=W)
    qf = host[0].copy()
    up = np.stack([[[qf[b, h, s, 0] * np.cos(lens[b]) - qf[b, h, s, 32] * np.sin(lens[b]) for s in range(T)] for h in range(H)]
                   for b in range(2)]) * sign > 0  # scores +inf
    keys = {"sparse": keys_of(W, "mask", "fib", 1.0, N), "dense": None}
    for name, o, l in both(plan, c, dev, parent=i32(parent), N=N):
        meets = np.ones((2, H, T), bool)
        want_o, want_l = np.zeros((2, H, T, 64)), np.zeros((2, H, T))
        for b in range(2):
            seen = range(lens[b]) if keys[name] is None else sorted({lens[b] - d for d, _ in keys[name] if 0 < d <= lens[b]})
            meets[b] = any(x in bad[b] for x in seen)
            seen = [x for x in seen if x not in bad[b]]
            kr, vr = ref.rows(0, b)
            for h in range(H):
                for s in range(T):
                    qr = co.turn(qf[b, h, s], lens[b])
                    ks = np.concatenate([kr[seen, h], co.turn(host[1][b, h, s], lens[b])[None]])
                    vs = np.concatenate([vr[seen, h], host[2][b, h, s][None]])
                    x = ks @ qr / 8
                    p = np.exp(x - x.max())
                    want_o[b, h, s], want_l[b, h, s] = p @ vs / p.sum(), x.max() + np.log(p.sum())
        none = up & meets
        o, l = o.double().cpu().numpy(), l.double().cpu().numpy()
        assert np.isnan(o[none]).all(), name
        assert not np.isfinite(l[none]).any(), name
        tol = TOL_O + (HALF[dtype] * np.abs(want_o) if dtype == "bf16" else 0)
        assert np.all((np.abs(o - want_o) <= tol)[~none]), name
        assert np.all((np.abs(l - want_l) <= TOL_LSE)[~none]), name
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    plan.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(1, 2), (8, 1), (16, 2), (24, 1), (40, 2), (64, 1)])
def test_the_most_sequences(dtype, T, H):
    """As many sequences as a cache may have, most of them short or empty."""
    r = rng(21, T)
    B = 1024
    lens = [int(x) for x in r.integers(0, 20, B)]
    for b in r.integers(0, B, 5):
        lens[b] = 200
    nodes = [int(x) for x in r.integers(0, T + 1, B)]
    c, ref, dev, host, parent, live = tree_case(r, dtype, lens, H, 1, T, 16, "random", nodes, poison=False)
    plan = plan_for(300, W=8)
    some = sorted({int(x) for x in r.integers(0, B, 40)} | {0, B - 1} | {b for b in range(B) if lens[b] == 200})
    few = [n if b in some else 0 for b, n in enumerate(live)]
    o, lse = sevens(dev[0])
    o2, lse2 = sevens(dev[0])
    fa.fib_attn_tree_decode(plan, 1, c, *dev, parent=i32(parent), n_nodes=i32(live), o=o, lse=lse)
    fa.fib_attn_dense_tree_decode(plan, 1, c, *dev, parent=i32(parent), n_nodes=i32(live), o=o2, lse=lse2)
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    for x, l, keys in ((o, lse, keys_of(8, "mask", "fib", 1.0, 300)), (o2, lse2, None)):
        ro, rl = co.tree_attend(ref, 1, *host, parent, few, keys)
        check(x[some], l[some], ro[some], rl[some], [live[b] for b in some], dtype)
        assert all(bool((x[b, :, n:] == 7).all()) and not bool((l[b, :, :n] == 7).any()) for b, n in enumerate(live))
    plan.close()


@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("bf16", 16), ("bf16", 32), ("bf16", 64), ("f32", 5), ("f32", 30)])
def test_a_wait_that_gives_up_is_reported(dtype, T):
    """The shortest wait a plan takes, 1 us, is about as long as a read of the cache: the call ends, its result is right
    or said not to be, and that of the next call with the usual wait is right."""
    r = rng(22, T)
    c, ref, dev, host, parent, live = tree_case(r, dtype, [60000], 4, 1, T, 64, "random", None, poison=False)
    plan = plan_for(60100)
    fa.fib_attn_plan_set_debug(plan, False, 1000)
    want = co.tree_attend(ref, 0, *host, parent, live)
    for usual in (False, True):
        if usual:
            fa.fib_attn_plan_set_debug(plan, False, 10 ** 9)
        o, lse = fa.fib_attn_dense_tree_decode(plan, 0, c, *dev, parent=i32(parent))
        status = fa.fib_attn_last_device_status(plan)
        assert status == fa.FIB_OK or (status == fa.FIB_ERR_TIMEOUT and not usual)
        if status == fa.FIB_OK:
            check(o, lse, *want, live, dtype)
    plan.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [2, 6, 7, 9, 12])
def test_without_lse_and_with_outputs_allocated(dtype, case):
    """want_lse=False gives the same o; so do outputs and workspace that the call allocates."""
    c, ref, dev, host, parent, live = tree_case(rng(25, case), dtype, *CASES[case])
    plan = plan_for(2300, W=8)
    kw = dict(parent=i32(parent), n_nodes=i32(live))
    for fn in (fa.fib_attn_tree_decode, fa.fib_attn_dense_tree_decode):
        o, lse = sevens(dev[0])
        fn(plan, 1, c, *dev, o=o, lse=lse, **kw)
        o2, none = fn(plan, 1, c, *dev, want_lse=False, **kw)
        o3, l3 = fn(plan, 1, c, *dev, **kw)
        assert none is None
        for b, n in enumerate(live):
            assert torch.equal(o[b, :, :n], o2[b, :, :n]) and torch.equal(o[b, :, :n], o3[b, :, :n])
            assert torch.equal(lse[b, :, :n], l3[b, :, :n])
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    plan.close()


def test_outputs_and_workspaces_of_a_call_on_another_stream():
    """What a call allocates for a stream that it is given is that stream's memory: work that the current stream
    still has to do on freed memory of its own does not meet it."""
    r = rng(23)
    c, ref, dev, host, parent, live = tree_case(r, "bf16", [3000, 2000], 4, 1, 16, 64, "random", None, poison=False)
    plan, side = plan_for(3100), torch.cuda.Stream()
    par = i32(parent)
    want = [x.clone() for x in fa.fib_attn_dense_tree_decode(plan, 0, c, *dev, parent=par)]
    big = torch.zeros(1 << 28, device="cuda")
    torch.cuda.synchronize()
    size = fa.fib_attn_dense_tree_workspace_size(plan, c, 2, 4, 16)
    for _ in range(5):
        big.add_(1)  # the current stream is busy for a while
        for shape, dt in ((size, torch.uint8), (dev[0].shape, torch.bfloat16), (dev[0].shape[:3], torch.float32)):
            torch.empty(shape, dtype=dt, device="cuda").fill_(99)  # still to be written when it is freed
        got = fa.fib_attn_dense_tree_decode(plan, 0, c, *dev, parent=par, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    plan.close()


@pytest.mark.parametrize("what", ["nodes", "negative", "parent", "self", "len", "position", "page id"])
def test_a_bad_sequence_is_reported_and_the_others_are_right(what):
    r = rng(12)
    c, ref, dev, host, parent, live = tree_case(r, "bf16", [20, 40], 2, 2, 6, 16, "random", None)
    W, N = 8, 64
    plan = plan_for(N, W=W)
    nodes, par = [6, 6], parent.copy()
    if what == "nodes":
        nodes[0] = 7
    elif what == "negative":
        nodes[0] = -1
    elif what == "parent":
        par[0, 3] = -2
    elif what == "self":
        par[0, 3] = 3
    elif what == "len":
        c.lens[0] = 16 * c.max_pages + 1
    elif what == "position":
        c.lens[0] = 48  # 48 + a chain of 6 fits, N = 50 does not hold it
        c.table[0, 2] = c.table[0, 1]
        par[0] = np.arange(6) - 1
        N = 50
    elif what == "page id":
        c.table[0, 1] = c.n_pages
    ref_o, ref_l = co.tree_attend(ref, 0, *host, parent, [0, 6], keys_of(W, "mask", "fib", 1.0, N))
    o, lse = fa.fib_attn_tree_decode(plan, 0, c, *dev, parent=i32(par), n_nodes=i32(nodes), N=N)
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_ERR_DEVICE_ASSERT
    assert np.all(np.abs(lse[1].double().cpu().numpy() - ref_l[1]) <= TOL_LSE)
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK  # cleared
    plan.close()
    plan = plan_for(N)
    ref_o, ref_l = co.tree_attend(ref, 0, *host, parent, [0, 6])
    o, lse = fa.fib_attn_dense_tree_decode(plan, 0, c, *dev, parent=i32(par), n_nodes=i32(nodes))
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_ERR_DEVICE_ASSERT
    assert np.all(np.abs(lse[1].double().cpu().numpy() - ref_l[1]) <= TOL_LSE)
    plan.close()


def test_refusals_of_the_binding_and_the_library():
    r = rng(13)
    c, ref, (q, kn, vn), host, parent, live = tree_case(r, "f32", [20, 40], 2, 2, 6, 16, "random", None)
    plan = plan_for(64)
    for fn in (fa.fib_attn_tree_decode, fa.fib_attn_dense_tree_decode):
        for bad in (dict(q=q[..., :32]), dict(q=q.transpose(0, 1)), dict(q=q.bfloat16()), dict(q=q.cpu()), dict(k_new=kn[:, :1].contiguous()),
                    dict(v_new=vn[:, :, :3].contiguous()), dict(parent=i32(parent[:1])), dict(parent=i32(parent).long()),
                    dict(n_nodes=i32([1])), dict(o=torch.empty_like(q[:1])), dict(lse=torch.empty(3, device="cuda"))):
            args = dict(q=q, k_new=kn, v_new=vn)
            args.update(bad)
            with pytest.raises(ValueError):
                fn(plan, 0, c, **args)
        three = torch.zeros((2, 3, 6, 64), device="cuda")  # three query heads, two key heads
        for layer, x in ((2, q), (-1, q), (0, three)):
            with pytest.raises(fa.FibAttnError):
                fn(plan, layer, c, x, kn, vn)
        with pytest.raises(fa.FibAttnError):
            fn(plan, 0, c, q, kn, vn, o=q)
        big = torch.zeros((2, 2, 65, 64), device="cuda")
        with pytest.raises(fa.FibAttnError):
            fn(plan, 0, c, torch.zeros((2, 4, 65, 64), device="cuda"), big, big)
        many = torch.zeros((3, 2, 1, 64), device="cuda")
        with pytest.raises(fa.FibAttnError):
            fn(plan, 0, c, many, many, many)
    with pytest.raises(fa.FibAttnError):
        fa.fib_attn_tree_decode(plan, 0, c, q, kn, vn, N=65)
    with pytest.raises(fa.FibAttnError):
        fa.fib_attn_dense_tree_decode(plan, 0, c, q, kn, vn, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fa.fib_attn_cache_commit(plan, c, kn, vn, i32([1, 1]))
    with pytest.raises(ValueError):
        fa.fib_attn_cache_fork(c, i32([0]))
    with pytest.raises(ValueError):
        fa.fib_attn_cache_compact(c, remap=i32([0]))
    with pytest.raises(fa.FibAttnError):
        fa.fib_attn_cache_create(1, 1, 24, 4, 1, 1, torch.float32)
    with pytest.raises(ValueError):
        fa.fib_attn_cache_create(1, 1, 16, 4, 1, 1, torch.float16)
    plan.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_beyond_two_to_the_31st_element(dtype):
    """Pages at the far end of a pool of more than 2^32 bytes (and 2^31 elements)."""
    r = rng(14)
    H, P = 8, 256
    NP = (1 << 31) // (H * P * 64) + 40
    k = torch.zeros((1, NP, H, P, 64), dtype=DT[dtype], device="cuda")
    v = torch.zeros((1, NP, H, P, 64), dtype=DT[dtype], device="cuda")
    c = fa.fib_attn_cache_create(1, H, P, NP, 1, 3, DT[dtype], k=k, v=v)
    c.refs[:NP - 2] = 1
    plan = plan_for(600, W=8, alpha=(1.3,))
    T = 300
    kn, kf = draw(r, (1, 1, H, T, 64), dtype)
    vn, vf = draw(r, (1, 1, H, T, 64), dtype)
    fa.fib_attn_cache_commit(plan, c, kn, vn, i32([T]))
    assert c.table[0, :2].tolist() == [NP - 2, NP - 1]
    ref = co.PagedCache(k[:, NP - 2:].double().cpu().numpy(), v[:, NP - 2:].double().cpu().numpy(), [[0, 1, -1]], [T], [1, 1])
    want = co.turn(kf[0, 0].transpose(1, 0, 2), np.arange(T)[:, None])
    got = ref.rows(0, 0)
    assert np.all(np.abs(got[0] - want) <= 1e-5 + HALF[dtype] * np.abs(want))
    assert np.array_equal(got[1], vf[0, 0].transpose(1, 0, 2))
    q, qf = draw(r, (1, H, 2, 64), dtype)
    kd, kdf = draw(r, (1, H, 2, 64), dtype)
    vd, vdf = draw(r, (1, H, 2, 64), dtype)
    parent = np.asarray([[-1, 0]])
    for name, o, l in both(plan, c, (q, kd, vd)):
        keys = keys_of(8, "mask", "fib", 1.3, 600) if name == "sparse" else None
        ro, rl = co.tree_attend(ref, 0, qf, kdf, vdf, parent, [2], keys)
        assert np.all(np.abs(o.double().cpu().numpy() - ro) <= TOL_O + (HALF[dtype] * np.abs(ro) if dtype == "bf16" else 0)), name
        assert np.abs(l.double().cpu().numpy() - rl).max() <= TOL_LSE, name
    # and moved down by a compaction once the rest is free
    c.refs[:NP - 2] = 0
    c.state[0] = 0
    fa.fib_attn_cache_compact(c)
    assert c.table[0, :2].tolist() == [0, 1] and c.state[2].item() == 2
    assert np.array_equal(c.k[0, :2].double().cpu().numpy(), ref.k[0])
    plan.close()


# ------------------------------------------------------------------------------- as they are used
def test_decode_by_trees_equals_the_forward():
    """Prompts, then steps of: tree decode, accept a path, commit.  In float32 every accepted node's output
    is the forward's row of the finished sequence (tolerances as above; the cached rows' rounding to
    float32 is among the counted errors)."""
    r = rng(15)
    B, H, P, W, alpha, N = 3, 2, 16, 6, 1.21, 160
    plan = fa.fib_attn_plan_create(fa.FIB_BASE_FIBONACCI, [1.0, alpha], W, N, fa.FIB_MODE_INTERP)
    c = fa.fib_attn_cache_create(2, H, P, 40, B, N // P, torch.float32)
    seqs = [[], [], []]  # (q, k, v, o or None) of layer 1 a token
    n0 = [40, 1, 17]
    T = 40
    kn, vn, qn = (draw(r, (2, B, H, T, 64), "f32")[0] for _ in range(3))
    fa.fib_attn_cache_commit(plan, c, kn, vn, i32(n0))
    for b in range(B):
        seqs[b] = [(qn[1, b, :, i], kn[1, b, :, i], vn[1, b, :, i], None, None) for i in range(n0[b])]
    for step in range(5):
        T = int(r.integers(1, 12))
        parent = trees(r, "random", B, T)
        q, kn, vn = (draw(r, (2, B, H, T, 64), "f32")[0] for _ in range(3))
        outs = [fa.fib_attn_tree_decode(plan, layer, c, q[layer], kn[layer], vn[layer], parent=i32(parent))
                for layer in range(2)]
        dense = fa.fib_attn_dense_tree_decode(plan, 1, c, q[1], kn[1], vn[1], parent=i32(parent))
        path, n_new = np.zeros((B, T), int), []
        for b in range(B):
            line = [int(r.integers(0, T))]
            while parent[b, line[-1]] >= 0:
                line.append(parent[b, line[-1]])
            line = line[::-1]
            if step == 2 and b == 1:
                line = []  # nothing accepted
            path[b, :len(line)] = line
            n_new.append(len(line))
            seqs[b] += [(q[1, b, :, s], kn[1, b, :, s], vn[1, b, :, s], outs[1][0][b, :, s], dense[0][b, :, s]) for s in line]
        fa.fib_attn_cache_commit(plan, c, kn, vn, i32(n_new), path=i32(path))
    assert fa.fib_attn_cache_status(c) == fa.FIB_OK and fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    for b in range(B):
        n = len(seqs[b])
        assert c.lens[b].item() == n
        x = [torch.stack([row[i] for row in seqs[b]], 1)[None].contiguous() for i in range(3)]
        o, _ = fa.fib_attn_fwd(plan, 1, *x)
        xf = [inputs.as_f64(t.cpu()) for t in x]
        want, _ = oracle.attend(*xf, alpha, oracle.fibonacci_base(), W, "interp")
        full, _ = oracle.attend(*xf, 1.0, [], n, "mask")
        for i, row in enumerate(seqs[b]):
            if row[3] is not None:
                assert np.abs(row[3].double().cpu().numpy() - want[0, :, i]).max() <= TOL_O
                assert (row[3] - o[0, :, i]).abs().max().item() <= 2 * TOL_O
                assert np.abs(row[4].double().cpu().numpy() - full[0, :, i]).max() <= TOL_O
    plan.close()


def test_single_token_equals_the_contiguous_decode():
    r = rng(16)
    B, H, N, W = 2, 3, 400, 12
    q, k, v = (draw(r, (B, H, N, 64), "f32")[0] for _ in range(3))
    plan = plan_for(N, W=W, alpha=(1.37,), mode=fa.FIB_MODE_INTERP)
    c = fa.fib_attn_cache_create(1, H, 32, 40, B, 13, torch.float32)
    pos = N - 1
    fa.fib_attn_cache_commit(plan, c, k[None, :, :, :pos].contiguous(), v[None, :, :, :pos].contiguous(), i32([pos, pos]))
    tok = [x[:, :, pos:].contiguous() for x in (q, k, v)]
    o, lse = fa.fib_attn_tree_decode(plan, 0, c, *tok)
    want, want_l = fa.fib_attn_decode(plan, 0, pos, q[:, :, pos].contiguous(), k, v)
    assert (o[:, :, 0] - want).abs().max().item() <= 2 * TOL_O
    assert (lse[:, :, 0] - want_l).abs().max().item() <= 2 * TOL_LSE
    plan.close()


def test_on_a_stream_of_its_own_and_in_a_graph():
    """Captured once, replayed on new inputs and a longer cache; the eager call between is undisturbed."""
    r = rng(17)
    B, H, T, P = 2, 2, 4, 16
    c, ref, dev, host, parent, live = tree_case(r, "bf16", [70, 33], H, 1, T, P, "random", None, poison=False)
    c2, ref2 = make_cache(r, "bf16", 2, H, P, [70, 33], 12, spare=20)
    plan = plan_for(300, W=8)
    par, n_new = i32(parent), i32([2, 1])
    path = i32([[0, 1, 0, 0], [0, 0, 0, 0]])
    k2, k2f = draw(r, (2, B, H, T, 64), "bf16")
    v2, v2f = draw(r, (2, B, H, T, 64), "bf16")
    ws = torch.empty(max(fa.fib_attn_cache_workspace_size(c2), 1), dtype=torch.uint8, device="cuda")
    wd = torch.empty(max(fa.fib_attn_dense_tree_workspace_size(plan, c2, B, H, T), 1), dtype=torch.uint8, device="cuda")
    q = dev[0]
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
    od, lsed = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
    side = torch.cuda.Stream()

    def step(stream=None):
        fa.fib_attn_tree_decode(plan, 0, c2, q, k2[0], v2[0], parent=par, o=o, lse=lse, stream=stream)
        fa.fib_attn_dense_tree_decode(plan, 0, c2, q, k2[0], v2[0], parent=par, o=od, lse=lsed, workspace=wd, stream=stream)
        fa.fib_attn_cache_commit(plan, c2, k2, v2, n_new, path=path, workspace=ws, stream=stream)

    keys = keys_of(8, "mask", "fib", 1.0, 300)

    def verify():
        for (x, l), kk in (((o, lse), keys), ((od, lsed), None)):
            ro, rl = co.tree_attend(ref2, 0, inputs.as_f64(q.cpu()), k2f[0], v2f[0], parent, [T] * B, kk)
            check(x, l, ro, rl, [T] * B, "bf16")
        bf = lambda x: torch.from_numpy(x).to(torch.bfloat16).double().numpy()  # noqa: E731
        assert ref2.commit(k2f, v2f, [2, 1], path.cpu().tolist(), rnd=bf)
        same_tables(c2, ref2)

    side.wait_stream(torch.cuda.current_stream())
    step(stream=side)
    side.synchronize()
    verify()
    ref2.k = c2.k.double().cpu().numpy()  # rows as stored (a half step of bf16 may fall either way)
    g = torch.cuda.CUDAGraph()
    before = c2.meta.clone(), c2.k.clone(), c2.v.clone()
    with torch.cuda.graph(g):
        step()
    assert all(torch.equal(x, y) for x, y in zip(before, (c2.meta, c2.k, c2.v)))  # capture runs nothing
    for i in range(3):
        q.copy_(draw(r, q.shape, "bf16")[0])
        for x, f in ((k2, k2f), (v2, v2f)):
            t, tf = draw(r, x.shape, "bf16")
            x.copy_(t)
            f[...] = tf
        g.replay()
        torch.cuda.synchronize()
        verify()
        ref2.k = c2.k.double().cpu().numpy()
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    plan.close()


def test_two_plans_on_two_streams_at_once():
    r = rng(18)
    jobs = []
    for i in range(2):
        c, ref, dev, host, parent, live = tree_case(r, "bf16", [900, 411, 0], 4, 2, 9, 32, "random", None)
        plan = plan_for(1000, W=8)
        alone = [(o.clone(), l.clone()) for _, o, l in both(plan, c, dev, parent=i32(parent))]
        jobs.append((plan, c, dev, i32(parent), alone, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for rep in range(10):
        for i, (plan, c, dev, parent, alone, st) in enumerate(jobs):
            with torch.cuda.stream(st):
                got[i] += [(n, o, l) for n, o, l in both(plan, c, dev, parent=parent)]
    torch.cuda.synchronize()
    for i, job in enumerate(jobs):
        for j, (name, o, l) in enumerate(got[i]):
            assert torch.equal(o, job[4][j % 2][0]) and torch.equal(l, job[4][j % 2][1]), name
        job[0].close()


@pytest.mark.parametrize("pattern", [0x7fc00000, 0x7c007c00, 0xffffffff])
def test_stale_shared_memory_does_not_reach_the_outputs(pattern):
    r = rng(19)
    for case in (3, 5, 6, 9):
        c, ref, dev, host, parent, live = tree_case(r, "bf16", *CASES[case])
        plan = plan_for(2300, W=8)
        nodes = i32(live)
        clean = [(o.clone(), l.clone()) for _, o, l in both(plan, c, dev, parent=i32(parent), n_nodes=nodes)]
        outs = []
        fa.fib_attn_debug_fill_shared(pattern)
        outs.append(fa.fib_attn_tree_decode(plan, 0, c, *dev, parent=i32(parent), n_nodes=nodes))
        fa.fib_attn_debug_fill_shared(pattern)
        outs.append(fa.fib_attn_dense_tree_decode(plan, 0, c, *dev, parent=i32(parent), n_nodes=nodes))
        torch.cuda.synchronize()
        for (o, l), (co_, cl) in zip(outs, clean):
            for b, n in enumerate(live):
                assert torch.equal(o[b, :, :n], co_[b, :, :n]) and torch.equal(l[b, :, :n], cl[b, :, :n])
        plan.close()
