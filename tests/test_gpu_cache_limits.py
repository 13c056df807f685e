"""The paged cache and the tree decodes at their limits: waits that run out, several host threads, one workspace for every
size, long contexts, large tables (needs a GPU).  Tolerances as in test_gpu_cache.py, unless a test derives its own."""
import os
import threading

import numpy as np
import pytest
import torch

from fibonacci_offset_sparse_gb300 import fib_attn as fa
from oracle import cache_oracle as co

from .test_gpu_cache import (HALF, TOL_LSE, TOL_O, check, close_rows, draw, i32, keys_of, make_cache, plan_for, rng, same_tables,
                             sevens, snapshot, tree_case, unchanged)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fibonacci_offset_sparse_gb300 import build as b
    if not os.path.exists(b.LIB):
        b.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return fa.lib()


# ------------------------------------------------------------------------- waits that run out
@pytest.mark.parametrize("lens", [[20000], [0, 700, 1, 3000, 40]])
@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("bf16", 16), ("bf16", 32), ("bf16", 48), ("bf16", 64), ("f32", 5), ("f32", 30)])
def test_a_copy_that_never_comes_is_reported(dtype, T, lens):
    """The first rows of every task are never copied: each wait for them runs out after 2 ms, the call ends and says
    so, and the next ordinary call is right."""
    r = rng(30, T, len(lens))
    c, ref, dev, host, parent, live = tree_case(r, dtype, lens, 2, 1, T, 64, "random", None, poison=False)
    plan, par = plan_for(20100), i32(parent)
    want = co.tree_attend(ref, 0, *host, parent, live)
    for _ in range(2):
        fa.fib_attn_plan_set_debug(plan, True, 2_000_000)
        for _ in range(2):
            fa.fib_attn_dense_tree_decode(plan, 0, c, *dev, parent=par)
            assert fa.fib_attn_last_device_status(plan) == fa.FIB_ERR_TIMEOUT
        fa.fib_attn_plan_set_debug(plan, False, 10 ** 9)
        o, lse = fa.fib_attn_dense_tree_decode(plan, 0, c, *dev, parent=par)
        assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
        check(o, lse, *want, live, dtype)
    plan.close()


# ----------------------------------------------------------------------------- long contexts
def long_case(dtype, B, H, T, n, fill, seed):
    """B sequences of n rows in pages of 64, one after the other in the pools, and T drafts each that follow the cached
    rows alone.  fill(shape, generator): the values."""
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = -(-n // 64)
    k = torch.empty((1, B * pages, H, 64, 64), device="cuda", dtype=dt).normal_(generator=g)
    v = fill((B, pages, H, 64, 64), g).to(dt).view(1, B * pages, H, 64, 64)
    c = fa.fib_attn_cache_create(1, H, 64, B * pages, B, pages, dt, k=k, v=v)
    c.table.copy_(torch.arange(B * pages, dtype=torch.int32).view(B, pages))
    c.lens.fill_(n)
    c.refs.fill_(1)
    q, kn = (torch.empty((B, H, T, 64), device="cuda").normal_(generator=g).to(dt) for _ in range(2))
    vn = fill((B, T, H, 1, 64), g).to(dt).view(B, T, H, 64).transpose(1, 2).contiguous()
    return c, q, kn, vn, i32(np.full((B, T), -1))


def exact_long(c, q, kn, vn, n, rows, lse=False):
    """The outputs (and lse) of the drafts `rows` (a slice) in 64 bits, on the GPU."""
    B, H, T, _ = q.shape
    turned = [torch.from_numpy(co.turn(x.double().cpu().numpy(), np.full((B, H, T), n))).cuda()[:, :, rows] for x in (q, kn)]
    out = torch.empty_like(turned[0])
    log = torch.empty_like(out[..., 0])
    k, v = (x.view(B, -1, H, 64, 64) for x in (c.k, c.v))
    for b in range(B):
        for h in range(H):
            x, own = turned[0][b, h], turned[1][b, h]
            s = torch.cat([x @ k[b, :, h].reshape(-1, 64)[:n].double().T, (x * own).sum(1, keepdim=True)], 1) / 8
            p, log[b, h] = torch.softmax(s, 1), torch.logsumexp(s, 1)
            out[b, h] = p[:, :-1] @ v[b, :, h].reshape(-1, 64)[:n].double() + p[:, -1:] * vn[b, h, rows].double()
    return (out, log) if lse else out


@pytest.mark.parametrize("T", [1, 16, 17, 64])
def test_equal_values_over_a_long_context(T):
    """Every value is 1, so every output is: what is left is how the sums are held.  A block's warps add one unit of 16 rows
    after the other to O and to the sum of the weights, some 900 at most here, each rounded to nearest: an error of at most 2^-24
    of a sum that grows to its end, 2^-24 / 3 in the mean square, sqrt(900) of them 6e-7 for each of the two sums; ten of
    the two, 8.5e-6, are allowed.  Sums that round toward zero at every product err by some 2^-25 a product, all to one side."""
    c, q, kn, vn, par = long_case("f32", 8, 8, T, 65536, lambda s, g: torch.ones(s, device="cuda"), 31)
    plan = plan_for(65600)
    o, _ = fa.fib_attn_dense_tree_decode(plan, 0, c, q, kn, vn, parent=par)
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    off = (o.double() - 1).abs().max().item()
    assert off <= 8.5e-6
    plan.close()


@pytest.mark.parametrize("T", [8, 16, 32, 64])
def test_mean_error_over_a_long_context(T):
    """bf16, values around a mean of their own for each sequence, head and dimension in [1, 2).  An output is rounded to a
    multiple of 2^-7, 2^-7 / sqrt(12) / 1.4 = 1.6e-3 of it in the mean square and as often up as down: over the 16 * 8 * 64
    means 1.8e-5, of which six are allowed.  The tensor pipes' own sums, which round toward zero, may add 256 products of at
    most 2^-24 each on average, 1.5e-5."""
    B, H, n = 16, 8, 131072

    def fill(shape, g):
        mean = 1 + torch.rand((B, 1, H, 1, 64), generator=torch.Generator(device="cuda").manual_seed(7), device="cuda")
        return torch.empty(shape, device="cuda").normal_(generator=g).mul_(0.1).add_(mean)

    c, q, kn, vn, par = long_case("bf16", B, H, T, n, fill, 32)
    plan = plan_for(n + 100)
    o, _ = fa.fib_attn_dense_tree_decode(plan, 0, c, q, kn, vn, parent=par)
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    rows = slice(0, T, T // 8)
    want = exact_long(c, q, kn, vn, n, rows)
    off = ((o[:, :, rows].double() - want) / want).mean().item()
    assert abs(off) <= 1.1e-4 + 1.5e-5
    plan.close()


@pytest.mark.parametrize("T", [1, 20])
def test_mean_error_in_float32(T):
    """float32, values around 1.  What errs to one side: the two last products of a unit's sum, cut off half a step of the
    sum on average, 2^-24 each at most, and the lower part of a value, cut off half of its last step, 2^-24; 1.8e-7 in all.  The
    rest (the weights' parts, sums rounded to nearest) errs to either side and leaves nothing in the mean over the outputs."""
    B, H, n = 4, 8, 8000
    c, q, kn, vn, par = long_case("f32", B, H, T, n, lambda s, g: torch.empty(s, device="cuda").normal_(generator=g).add_(1), 33)
    plan = plan_for(n + 100)
    o, _ = fa.fib_attn_dense_tree_decode(plan, 0, c, q, kn, vn, parent=par)
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    want = exact_long(c, q, kn, vn, n, slice(0, T))
    off = ((o.double() - want) / want).mean().item()
    assert abs(off) <= 1.8e-7
    plan.close()


# ------------------------------------------------------------------------------- host threads
def in_thread(fn):
    """fn() in a host thread that has made no CUDA call yet."""
    got = []

    def run():
        try:
            got.append(fn())
        except Exception as e:
            got.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert not isinstance(got[0], Exception), got[0]
    return got[0]


@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("bf16", 16), ("bf16", 32), ("bf16", 48), ("bf16", 64), ("f32", 5), ("f32", 30)])
@pytest.mark.parametrize("op", ["dense", "sparse", "commit", "fork", "compact"])
def test_a_first_call_of_a_host_thread(op, dtype, T):
    """Everything that the call needs is there beforehand, so that it is the thread's first use of CUDA."""
    r = rng(35, T)
    c, ref, dev, host, parent, live = tree_case(r, dtype, [70, 3], 1, 1, T, 16, "random", None, poison=False)
    plan, par, side = plan_for(200), i32(parent), torch.cuda.Stream()
    o, lse = torch.empty_like(dev[0]), torch.empty(dev[0].shape[:3], device="cuda")
    kn, vn = (x[None].expand(2, -1, -1, -1, -1).contiguous() for x in dev[1:])
    n_new, src, remap = i32([1, 0]), i32([1, 0]), i32(np.zeros(c.n_pages))
    need = max(fa.fib_attn_cache_workspace_size(c), fa.fib_attn_dense_tree_workspace_size(plan, c, 2, 1, T))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    call = {
        "dense": lambda: fa.fib_attn_dense_tree_decode(plan, 0, c, *dev, parent=par, o=o, lse=lse, workspace=ws, stream=side),
        "sparse": lambda: fa.fib_attn_tree_decode(plan, 0, c, *dev, parent=par, o=o, lse=lse, stream=side),
        "commit": lambda: fa.fib_attn_cache_commit(plan, c, kn, vn, n_new, workspace=ws, stream=side),
        "fork": lambda: fa.fib_attn_cache_fork(c, src, workspace=ws, stream=side),
        "compact": lambda: fa.fib_attn_cache_compact(c, remap=remap, workspace=ws, stream=side)}[op]
    torch.cuda.synchronize()
    in_thread(call)
    torch.cuda.synchronize()
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK and fa.fib_attn_cache_status(c) == fa.FIB_OK
    if op == "dense":
        want = fa.fib_attn_dense_tree_decode(plan, 0, c, *dev, parent=par)
    if op == "sparse":
        want = fa.fib_attn_tree_decode(plan, 0, c, *dev, parent=par)
    if op in ("dense", "sparse"):
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert c.lens.tolist() == {"commit": [71, 3], "fork": [3, 70]}.get(op, [70, 3])
    plan.close()


@pytest.mark.parametrize("dtype,T,most", [("bf16", 1, 8), ("bf16", 16, 16), ("bf16", 33, 48), ("f32", 1, 16), ("f32", 17, 64)])
def test_calls_of_different_sizes_from_several_host_threads(dtype, T, most):
    """One sequence with few drafts in some threads, a thousand with many in others; the same kernel, nothing else shared.  The
    library is called directly, so that the calls lie close together."""
    jobs = []
    for i, (B, t) in enumerate(((1, T), (1000, most)) * 3):
        r = rng(34, i, t)
        c, ref, dev, host, parent, live = tree_case(r, dtype, [30] + [0] * (B - 1), 1, 1, t, 16, "random", None, poison=False)
        plan, par = plan_for(200), i32(parent)
        ws = torch.empty(fa.fib_attn_dense_tree_workspace_size(plan, c, B, 1, t), dtype=torch.uint8, device="cuda")
        want = fa.fib_attn_dense_tree_decode(plan, 0, c, *dev, parent=par)
        got = tuple(torch.empty_like(x) for x in want)
        side = torch.cuda.Stream()
        args = (plan.handle, 0, c.pointer, B, 1, t, *(x.data_ptr() for x in dev), par.data_ptr(), None, got[0].data_ptr(),
                got[1].data_ptr(), ws.data_ptr(), ws.nbytes, side.cuda_stream)
        jobs.append(dict(args=args, got=got, want=want, side=side, plan=plan, codes=set(), keep=(c, dev, par, ws)))
    torch.cuda.synchronize()
    ready, fn = threading.Barrier(len(jobs)), fa.lib().fib_attn_dense_tree_decode

    def calls(j):
        j["side"].synchronize()  # (the thread's first call)
        ready.wait()
        for _ in range(3000):
            j["codes"].add(fn(*j["args"]))

    threads = [threading.Thread(target=calls, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for j in jobs:
        assert j["codes"] == {fa.FIB_OK}
        assert all(torch.equal(x, y) for x, y in zip(j["got"], j["want"]))
        j["plan"].close()


# ------------------------------------------------------------------------------- workspaces
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G", [1, 2])
def test_one_workspace_for_every_number_of_drafts(dtype, G):
    """Sized for the largest tree, it serves every smaller one."""
    r = rng(36, G)
    c, ref, dev, host, parent, live = tree_case(r, dtype, [2000, 0, 333], 2, G, 64, 32, "random", None, poison=False)
    plan = plan_for(2100)
    sizes = [fa.fib_attn_dense_tree_workspace_size(plan, c, 3, 2 * G, T) for T in range(1, 65)]
    assert sizes == sorted(sizes)
    assert sizes[-1] == fa.fib_attn_dense_tree_workspace_size(plan, c, 1, 2 * G, 64)
    assert sizes[-1] <= fa.fib_attn_dense_tree_workspace_size(plan, c, 3, 8 * G, 64)
    ws = torch.empty(sizes[-1], dtype=torch.uint8, device="cuda")
    for T in (1, 8, 9, 16, 17, 24, 32, 33, 48, 49, 64):
        q, kn, vn = (x[:, :, :T].contiguous() for x in dev)
        o, lse = fa.fib_attn_dense_tree_decode(plan, 0, c, q, kn, vn, parent=i32(parent[:, :T]), workspace=ws)
        want = co.tree_attend(ref, 0, *(x[:, :, :T] for x in host), parent[:, :T], [T] * 3)
        check(o, lse, *want, [T] * 3, dtype)
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    plan.close()


# --------------------------------------------------------------------------- far below zero
@pytest.mark.parametrize("nearest", ["cached", "drafted"])
@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("bf16", 16), ("bf16", 32), ("bf16", 48), ("bf16", 64), ("f32", 5), ("f32", 30)])
def test_scores_far_below_zero(dtype, T, nearest):
    """Every score is below -1e30, as of keys that a caller has put out of the way.  Those of one size differ by nothing and
    those of different ones by 1e30 and more, so that the nearest share the weight, whatever a score's rounding is."""
    r = rng(37, T)
    c, ref, dev, host, parent, live = tree_case(r, dtype, [500, 40, 300], 1, 1, T, 32, "roots", None, poison=False)
    for x in (c.k, dev[0], dev[1]):
        x.zero_()
    for x in (ref.k, host[0], host[1]):
        x[...] = 0
    size = 2.0 ** (53 + r.integers(1, 4, ref.k.shape[:4]))
    ref.k[..., 31] = size
    c.k[..., 31] = torch.from_numpy(size).to(c.k)
    host[0][..., 31], host[1][..., 31] = -2.0 ** 53, 2.0 ** (53 if nearest == "drafted" else 57)  # (dimension 31 turns by 1.3e-4 a row)
    for t, h in zip(dev[:2], host[:2]):
        t.copy_(torch.from_numpy(h))
    plan = plan_for(600)
    o, lse = fa.fib_attn_dense_tree_decode(plan, 0, c, *dev, parent=i32(parent))
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    ro, rl = co.tree_attend(ref, 0, *host, parent, live)
    assert rl.max() < -1e30
    assert np.all(np.abs(o.double().cpu().numpy() - ro) <= TOL_O + (HALF[dtype] * np.abs(ro) if dtype == "bf16" else 0))
    assert np.all(np.abs(lse.double().cpu().numpy() / rl - 1) <= 2.0 ** -15)  # (a bf16 query is held in 16 bits)
    plan.close()


@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("bf16", 8), ("bf16", 16), ("bf16", 32), ("bf16", 48), ("bf16", 64), ("f32", 3), ("f32", 40)])
def test_dense_decode_of_a_long_context(dtype, T):
    """Every output and lse over 300000 rows; the same rows in pages in another order give the same bits."""
    B, H, n = 2, 1, 300000
    c, q, kn, vn, par = long_case(dtype, B, H, T, n, lambda s, g: torch.empty(s, device="cuda").normal_(generator=g), 38)
    plan = plan_for(n + 100)
    o, lse = fa.fib_attn_dense_tree_decode(plan, 0, c, q, kn, vn, parent=par)
    want, want_l = exact_long(c, q, kn, vn, n, slice(0, T), lse=True)
    order = torch.from_numpy(rng(38).permutation(c.n_pages)).cuda()  # the same rows in other pages
    moved = torch.empty_like(order)
    moved[order] = torch.arange(c.n_pages, device="cuda")
    for x in (c.k, c.v):
        x.copy_(x[:, order])
    c.table.copy_(moved[c.table.long()].int())
    o2, lse2 = fa.fib_attn_dense_tree_decode(plan, 0, c, q, kn, vn, parent=par)
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert ((o.double() - want).abs() <= TOL_O + (HALF[dtype] * want.abs() if dtype == "bf16" else 0)).all()
    assert ((lse.double() - want_l).abs() <= TOL_LSE).all()
    plan.close()


# ------------------------------------------------------------------------------ large tables
@pytest.mark.parametrize("S,P,most", [(300, 16, 1000), (1024, 16, 200), (9, 16, 20000)])
def test_fork_of_a_large_table(S, P, most):
    """More than 8192 table entries: the two launches."""
    r = rng(39, S)
    lens = [int(x) for x in r.integers(0, most, S)]
    max_pages = -(-most // P)
    assert S * max_pages > 8192
    c, ref = make_cache(r, "f32", 1, 1, P, lens, max_pages, spare=300)
    for _ in range(3):
        src = [int(x) for x in np.where(r.random(S) < 0.3, np.arange(S), r.integers(-1, S, S))]
        fa.fib_attn_cache_fork(c, i32(src))
        ref.fork(src)
        same_tables(c, ref)
        cursor = c.state[0].item()
        assert (c.refs[:cursor] > 0).all()
    assert fa.fib_attn_cache_status(c) == fa.FIB_OK
    for bad in ([S] + [-1] * (S - 1), [-1] * (S - 1) + [-2]):
        before = snapshot(c)
        fa.fib_attn_cache_fork(c, i32(bad))
        unchanged(c, before, fa.FIB_ERR_DEVICE_ASSERT)
    fa.fib_attn_cache_fork(c, i32([-1] * S))
    assert not c.refs.any() and not c.lens.any() and (c.table == -1).all()


def test_fork_of_a_large_table_in_a_graph():
    r = rng(40)
    S, P, most = 200, 16, 1000
    lens = [int(x) for x in r.integers(0, most, S)]
    c, ref = make_cache(r, "f32", 1, 1, P, lens, -(-most // P))
    src = i32(np.arange(S))
    ws = torch.empty(fa.fib_attn_cache_workspace_size(c), dtype=torch.uint8, device="cuda")
    fa.fib_attn_cache_fork(c, src, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.fib_attn_cache_fork(c, src, workspace=ws)
    for _ in range(3):
        new = r.integers(-1, S, S)
        src.copy_(i32(new))
        g.replay()
        torch.cuda.synchronize()
        ref.fork([int(x) for x in new])
        same_tables(c, ref)


def test_a_commit_that_takes_thousands_of_pages():
    """More pages than the plan keeps in shared memory, from between pages that are in use."""
    r = rng(41)
    P, T, lens, n_new = 16, 34000, [5, 0, 33], [33000, 34000, 1]
    c, ref = make_cache(r, "f32", 1, 1, P, lens, 2200, spare=9000)
    held = r.random(c.n_pages) < 0.4  # by the caller
    c.refs += i32(held)
    ref.refs = [a + int(b) for a, b in zip(ref.refs, held)]
    (kn, kf), (vn, vf) = draw(r, (1, 3, 1, T, 64), "f32"), draw(r, (1, 3, 1, T, 64), "f32")
    plan = plan_for(40000)
    fa.fib_attn_cache_commit(plan, c, kn, vn, i32(n_new))
    assert ref.commit(kf, vf, n_new)
    same_tables(c, ref)
    close_rows(c, ref, "f32")
    assert fa.fib_attn_cache_status(c) == fa.FIB_OK
    # and one page too many
    free = int((c.refs == 0).sum())
    c.refs[torch.nonzero(c.refs == 0)[:free - 4300].flatten()] = 1
    c.state[0] = 0
    before = snapshot(c)
    fa.fib_attn_cache_commit(plan, c, kn, vn, i32([34000, 0, 34000]))
    unchanged(c, before, fa.FIB_ERR_DEVICE_ASSERT)  # (33005 + 34000 rows pass the table)
    c.lens[0] = c.lens[1] = 0
    before = snapshot(c)
    fa.fib_attn_cache_commit(plan, c, kn, vn, i32([34000, 34000, 34000]))
    unchanged(c, before, fa.FIB_ERR_NO_PAGES)
    plan.close()


@pytest.mark.parametrize("where", [None, 1023, 1024, 1030, 2047, 2399])
def test_paths_of_more_than_a_thousand_entries(where):
    r = rng(42)
    B, T, P = 12, 200, 16
    c, ref = make_cache(r, "bf16", 1, 2, P, [7] * B, 20, spare=200)
    (kn, kf), (vn, vf) = draw(r, (1, B, 2, T, 64), "bf16"), draw(r, (1, B, 2, T, 64), "bf16")
    path = np.stack([r.permutation(T) for _ in range(B)])
    n_new = [T, 3, T, 0, T, T, 150, T, T, T, 199, T]
    path[3], path[1, 3:], path[10, 199:] = -5, T, 1 << 30  # not taken, so of no matter
    plan = plan_for()
    if where is not None:
        b, i = divmod(where, T)
        assert i < n_new[b]
        path[b, i] = T if where % 2 else -1
        before = snapshot(c)
        fa.fib_attn_cache_commit(plan, c, kn, vn, i32(n_new), path=i32(path))
        unchanged(c, before, fa.FIB_ERR_DEVICE_ASSERT)
    else:
        fa.fib_attn_cache_commit(plan, c, kn, vn, i32(n_new), path=i32(path))
        assert ref.commit(kf, vf, n_new, path)
        same_tables(c, ref)
        close_rows(c, ref, "bf16")
    plan.close()


# --------------------------------------------------------------- a learned alpha on the device
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("base,alpha,W,N", [("fib", 1.2713, 12, None), ("fib", 0.53, 1, 2000), ("pow2", 0.8125, 9, None)])
@pytest.mark.parametrize("lens,H,G,T", [([1500, 0, 3], 2, 1, 1), ([700, 129], 3, 2, 9), ([33, 1900, 0, 64], 8, 2, 20)])
def test_sparse_decode_row_by_row_with_a_device_alpha(dtype, base, alpha, W, N, lens, H, G, T):
    """Learned alpha: the key table is built on the device, of one row's four warps and of a warp a row."""
    r = rng(43, T)
    c, ref, dev, host, parent, live = tree_case(r, dtype, lens, H, G, T, 16, "random", None)
    plan = fa.fib_attn_plan_create(fa.FIB_BASE_FIBONACCI if base == "fib" else fa.FIB_BASE_POW2, [1.0, 0.7], W, 2048, fa.FIB_MODE_INTERP)
    learned = torch.tensor([9.0, alpha], device="cuda", dtype=torch.float32)
    o, lse = sevens(dev[0])
    fa.fib_attn_tree_decode(plan, 1, c, *dev, parent=i32(parent), o=o, lse=lse, N=N, alpha_dev=learned)
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    keys = keys_of(W, "interp", base, float(learned[1]), N or 2048)
    check(o, lse, *co.tree_attend(ref, 1, *host, parent, live, keys), live, dtype)
    plan.close()


# ------------------------------------------------------------------------------ bad sequences
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,G", [(6, 2, 2), (24, 1, 1), (64, 20, 1)])
@pytest.mark.parametrize("what", ["nodes", "parent", "len", "page id"])
def test_outputs_beside_a_bad_sequence(dtype, T, H, G, what):
    """The sequence after a refused one, its outputs and all, in each kernel."""
    r = rng(44, T)
    c, ref, dev, host, parent, live = tree_case(r, dtype, [20, 700, 45], H, G, T, 16, "random", None)
    plan = plan_for(900)
    nodes, par = [T] * 3, parent.copy()
    if what == "nodes":
        nodes[0] = T + 1
    elif what == "parent":
        par[0, 3] = 3
    elif what == "len":
        c.lens[0] = 16 * c.max_pages + 1
    else:
        c.table[0, 0] = c.n_pages
    for fn, keys in ((fa.fib_attn_tree_decode, keys_of(8, "mask", "fib", 1.0, 900)), (fa.fib_attn_dense_tree_decode, None)):
        o, lse = fn(plan, 0, c, *dev, parent=i32(par), n_nodes=i32(nodes))
        assert fa.fib_attn_last_device_status(plan) == fa.FIB_ERR_DEVICE_ASSERT
        ro, rl = co.tree_attend(ref, 0, *host, parent, [0, T, T], keys)
        check(o[1:], lse[1:], ro[1:], rl[1:], [T, T], dtype)
    plan.close()


# ---------------------------------------------------------------------------- lse in 32 bits
@pytest.mark.parametrize("op", ["dense", "sparse"])
@pytest.mark.parametrize("T,H,G", [(1, 24, 1), (5, 8, 1), (16, 4, 1), (11, 3, 2), (47, 2, 1), (64, 2, 1), (64, 8, 1), (24, 32, 2)])
def test_lse_of_bf16_is_that_of_float32(op, T, H, G):
    """Short contexts, whose lse is little more than a score.  bf16 inputs, everything between them and lse in float32: of a score of
    size 1 the sums of the tensor pipes, cut off at four products or so of up to 2^-23 each, leave some 2.5e-7 in the mean square, 2^x
    and log2 2e-7, rotation and the rest 1e-7: 3.4e-7.  A query that is held in 16 bits leaves 1.3e-6."""
    r = rng(45, T, H)
    lens = [0, 1, 2, 3, 5, 9, 17, 40]
    c, ref, dev, host, parent, live = tree_case(r, "bf16", lens, H, G, T, 16, "random", None, poison=False)
    plan = plan_for(200)
    fn, keys = (fa.fib_attn_dense_tree_decode, None) if op == "dense" else (fa.fib_attn_tree_decode, keys_of(8, "mask", "fib", 1.0, 200))
    _, lse = fn(plan, 0, c, *dev, parent=i32(parent))
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    _, want = co.tree_attend(ref, 0, *host, parent, live, keys)
    off = np.sqrt(np.mean((lse.double().cpu().numpy() - want) ** 2))
    assert off <= 5e-7
    plan.close()


def test_lse_of_bf16_where_the_union_takes_two_steps():
    """The same for the sparse decode of a tree so deep that its rows are served in two steps: queries four times as large, cached
    keys of 0, so that the drafted keys make lse; four times the errors above."""
    r = rng(46)
    c, ref, dev, host, parent, live = tree_case(r, "bf16", [1500], 40, 1, 64, 64, "random", None, poison=False)
    parent = np.arange(64)[None] - 4
    parent[parent < 0] = -1
    c.k.zero_()
    ref.k[...] = 0
    dev[0].mul_(4)
    host[0][...] *= 4
    plan = plan_for(2000)
    _, lse = fa.fib_attn_tree_decode(plan, 0, c, *dev, parent=i32(parent))
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    _, want = co.tree_attend(ref, 0, *host, parent, live, keys_of(8, "mask", "fib", 1.0, 2000))
    off = np.sqrt(np.mean((lse.double().cpu().numpy() - want) ** 2, axis=(0, 1)))
    assert off[:32].max() <= 2e-6 and off[32:].max() <= 2e-6
    plan.close()


# ------------------------------------------------------------------- traffic of other blocks
@pytest.mark.parametrize("dtype,T,H", [("f32", 64, 20), ("f32", 16, 30), ("f32", 1, 64), ("bf16", 1, 64), ("bf16", 8, 64), ("bf16", 16, 40),
                                       ("bf16", 64, 20)])
def test_the_same_bits_beside_blocks_that_report_at_once(dtype, T, H):
    """The blocks of a refused tree all write the status word, which holds up the loads of the blocks beside them: the other
    sequences' outputs are the same bits as without, every time."""
    r = rng(47, T)
    c, ref, dev, host, parent, live = tree_case(r, dtype, [20, 700, 45, 900], H, 1, T, 16, "random", None)
    plan, good, bad = plan_for(1000), i32(parent), i32(parent)
    bad[0, T // 2] = T // 2
    for fn in (fa.fib_attn_dense_tree_decode, fa.fib_attn_tree_decode):
        want = [x.clone() for x in fn(plan, 0, c, *dev, parent=good)]
        assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
        for _ in range(100):
            got = fn(plan, 0, c, *dev, parent=bad)
            assert all(torch.equal(x[1:], y[1:]) for x, y in zip(got, want))
        assert fa.fib_attn_last_device_status(plan) == fa.FIB_ERR_DEVICE_ASSERT
    plan.close()
