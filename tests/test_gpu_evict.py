"""Eviction from the paged cache by accumulated attention weight against the oracle (needs a GPU).

Which rows stay, and so every table, count, weight and value, is equal.  A K row that moves is rotated in float32 (a few 2^-24 of
its size, below 1e-5 for |x| < 8) and rounded once to the cache's type: half a step, 2^-24 or 2^-8 of the value."""
import math

import numpy as np
import pytest
import torch

from fibonacci_offset_sparse_gb300 import fib_attn as fa
from tests.test_gpu_cache import close_rows, draw, i32, make_cache, plan_for, rng, same_tables

pytestmark = pytest.mark.gpu


def weights_of(r, c, rows, ties=True):
    w = r.standard_normal((c.n_layers, c.max_seqs, c.heads, rows)).astype(np.float32) ** 2
    return np.floor(w * 8) / 8 if ties else w


def run(c, ref, plan, w, keep, sink, recent, dtype, turns=True):
    """The call and the oracle's, compared in all they leave."""
    wd, dropped, d_ref = torch.from_numpy(w.copy()).cuda(), i32([7] * len(keep)), [7] * len(keep)
    fa.fib_attn_cache_evict(plan, c, wd, i32(keep), sink, recent, dropped=dropped)
    assert ref.evict(w, keep, sink, recent, d_ref, turns)
    assert fa.fib_attn_cache_status(c) == fa.FIB_OK
    same_tables(c, ref)
    close_rows(c, ref, dtype)
    assert np.array_equal(wd.cpu().numpy(), w, equal_nan=True) and dropped.cpu().tolist() == d_ref
    cursor = int(c.state[0])
    assert all(ref.refs[:cursor])  # no free page lies below it


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("P,H,lens,keep,sink,recent", [
    (16, 1, [2], [1], 0, 0),                                   # one row of two
    (16, 3, [1, 0, 5], [0, 0, 5], 0, 0),                       # nothing left; an empty one; one that fits
    (16, 2, [100, 40, 17, 16], [33, 33, 16, 16], 4, 8),        # pages that end inside
    (64, 2, [300, 129], [128, 128], 64, 64),                   # whole pages at both ends, nothing between to keep
    (32, 5, [257, 256, 255], [255, 200, 254], 0, 31),
    (16, 2, [90, 90], [60, 45], 33, 0),                        # a sink over two pages and a row
    (256, 1, [700, 3], [699, 2], 1, 1),
    (128, 2, [5000, 2049, 2048], [2500, 2048, 1024], 5, 100),  # more than a step of 2048 rows
])
@pytest.mark.parametrize("turns", [True, False])
def test_rows_that_stay(dtype, P, H, lens, keep, sink, recent, turns):
    r = rng(100, P, H, *lens)
    c, ref = make_cache(r, dtype, 2, H, P, lens, -(-max(lens) // P) + 1)
    plan = plan_for(8192)
    fa.fib_attn_plan_set_rotation(plan, turns)
    run(c, ref, plan, weights_of(r, c, max(lens) + 3), keep, sink, recent, dtype, turns)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,keep,sink,recent", [
    ([5200, 300, 0], [2600, 299, 0], 4, 100),         # room for more than a block of 256 threads holds
    ([16384, 6000, 20], [16383, 10, 19], 0, 3),       # all that a block of 1024 holds
    ([16385, 20001], [8000, 20000], 5, 0),            # more: the weights are read anew in each pass
    ([33000, 16500], [1, 16000], 1, 0),
])
def test_long_sequences(dtype, lens, keep, sink, recent):
    r = rng(111, *lens)
    c, ref = make_cache(r, dtype, 1, 2, 64, lens, -(-max(lens) // 64) + 1)
    w = weights_of(r, c, max(lens) + 1)
    w[:, 0, 0, 5:max(lens):7], w[:, 0, 0, 3::1000], w[:, 0, 0, 4::2000], w[:, 0, 0, 11::900] = 0.0, np.nan, np.inf, -1.5
    run(c, ref, plan_for(1 << 16), w, keep, sink, recent, dtype)


def test_weights_of_every_kind():
    """Equal ones, zeros of both signs, negative, infinite and NaN ones."""
    r = rng(101)
    lens, keep = [400, 400, 400, 90], [100, 399, 20, 88]
    c, ref = make_cache(r, "f32", 2, 2, 16, lens, 26)
    w = weights_of(r, c, 400)
    w[0] = 0.25
    w[1, 0] = np.where(r.random((2, 400)) < 0.5, 0.0, -0.0)
    w[1, 1] = -w[1, 1]
    w[1, 2, 0, ::3], w[1, 2, 0, 1::3] = np.nan, -np.inf
    w[1, 2, 1, 5:300:40], w[1, 2, 1, 7] = np.inf, np.nan
    w[1, 3, :, 40:60] = 1e-42  # below the normal numbers
    run(c, ref, plan_for(), w, keep, 2, 3, "f32")


@pytest.mark.parametrize("held", [0, 1])
def test_shared_pages_are_left_to_the_others(held):
    """Three sequences share four pages; one of them stays whole, the sink's page stays shared.  `held`: the caller holds a page too."""
    r = rng(102, held)
    lens, P = [75, 70, 66, 30], 16
    c, ref = make_cache(r, "bf16", 2, 3, P, lens, 6, spare=12, share=[(1, 0, 4), (2, 0, 4)])
    page = ref.table[3][1]
    ref.refs[page] += held
    c.refs[page] += held
    w = weights_of(r, c, 80)
    refused(c, plan_for(), torch.from_numpy(w).cuda(), [50, 40, 66, 20], 17, 9, fa.FIB_ERR_DEVICE_ASSERT)  # 17 + 9 rows are sure to stay
    run(c, ref, plan_for(), w, [50, 40, 66, 26], 17, 9, "bf16")


def test_the_whole_group_shrinks():
    """No sequence keeps the pages that all shared: they are free at the end, and the next call takes them."""
    r = rng(103)
    c, ref = make_cache(r, "bf16", 1, 2, 16, [64, 64, 64], 5, spare=6, share=[(1, 0, 4), (2, 0, 4)])
    plan = plan_for()
    run(c, ref, plan, weights_of(r, c, 64), [32, 32, 20], 0, 4, "bf16")
    assert sum(x == 0 for x in ref.refs) == len(ref.refs) - 6
    kn, kf = draw(r, (1, 3, 2, 20, 64), "bf16")
    vn, vf = draw(r, (1, 3, 2, 20, 64), "bf16")
    fa.fib_attn_cache_commit(plan, c, kn, vn, i32([20, 1, 12]))
    assert ref.commit(kf, vf, [20, 1, 12])
    same_tables(c, ref)


def refused(c, plan, w, keep, sink, recent, code):
    before = [t.clone() for t in (c.meta, c.k, c.v, w)]
    dropped = i32([3] * len(keep))
    fa.fib_attn_cache_evict(plan, c, w, i32(keep), sink, recent, dropped=dropped)
    assert fa.fib_attn_cache_status(c) == code
    assert all(torch.equal(a, b) for a, b in zip(before, (c.meta, c.k, c.v, w))) and (dropped == 3).all()


def test_all_or_nothing():
    r = rng(104)
    c, ref = make_cache(r, "f32", 2, 2, 16, [64, 64, 50], 5, spare=2, share=[(1, 0, 4)])
    plan, w = plan_for(4096), torch.rand(2, 3, 2, 70, device="cuda")
    # 3 + 1 shared pages are to be replaced; of the 6 free ones (2, and the 4 that the second sequence does not need) the caller takes 3
    taken = [p for p, x in enumerate(ref.refs) if x == 0][:3]
    for p in taken:
        ref.refs[p] = 1
        c.refs[p] = 1
    refused(c, plan, w, [48, 10, 5], 0, 0, fa.FIB_ERR_NO_PAGES)
    refused(c, plan, w, [64, 64, -1], 0, 0, fa.FIB_ERR_DEVICE_ASSERT)
    refused(c, plan, w, [64, 64, 9], 5, 5, fa.FIB_ERR_DEVICE_ASSERT)  # sink and recent alone are more
    refused(c, plan, w[..., :60].contiguous(), [32, 32, 32], 0, 0, fa.FIB_ERR_DEVICE_ASSERT)
    refused(c, plan_for(63), w, [32, 64, 50], 0, 0, fa.FIB_ERR_DEVICE_ASSERT)
    for at, bad in ((1, -1), (3, c.n_pages)):
        was = int(c.table[2, at])
        c.table[2, at] = bad
        refused(c, plan, w, [64, 64, 40], 0, 0, fa.FIB_ERR_DEVICE_ASSERT)
        c.table[2, at] = was
    for bad in (-1, 81):
        c.lens[2] = bad
        refused(c, plan, w, [64, 64, 100], 0, 0, fa.FIB_ERR_DEVICE_ASSERT)
    c.lens[2] = 50
    # a sequence that fits is bound by nothing but its length
    fa.fib_attn_cache_evict(plan_for(1), c, w[..., :1].contiguous(), i32([64, 64, 50]), 400, 400)
    assert fa.fib_attn_cache_status(c) == fa.FIB_OK
    run(c, ref, plan, w.cpu().numpy(), [64, 64, 40], 0, 0, "f32")


def test_sequences_behind_the_batch_are_left():
    r = rng(105)
    c, ref = make_cache(r, "f32", 1, 1, 16, [60, 60, 60], 5)
    run(c, ref, plan_for(), weights_of(r, c, 60), [30, 60], 0, 0, "f32")


def test_refusals():
    r = rng(106)
    c, _ = make_cache(r, "f32", 2, 2, 16, [64, 64], 5)
    plan, w, keep = plan_for(), torch.zeros(2, 2, 2, 70, device="cuda"), i32([32, 32])
    for kw in (dict(weights=w.double()), dict(weights=w[:1]), dict(weights=w[..., ::2]), dict(weights=w.cpu()), dict(keep=keep.long()), dict(keep=keep[None]),
               dict(dropped=keep[:1]), dict(workspace=torch.zeros(8, device="cuda")[::2])):
        with pytest.raises(ValueError):
            fa.fib_attn_cache_evict(plan, c, **{**dict(weights=w, keep=keep, sink=0, recent=0), **kw})
    for kw in (dict(sink=-1), dict(recent=-1), dict(sink=1 << 30), dict(keep=i32([1, 2, 3])), dict(weights=w[..., :0]),
               dict(workspace=torch.zeros(16, device="cuda", dtype=torch.uint8)), dict(dropped=keep), dict(dropped=c.lens)):
        with pytest.raises(fa.FibAttnError) as e:
            fa.fib_attn_cache_evict(plan, c, **{**dict(weights=w, keep=keep, sink=0, recent=0), **kw})
        assert e.value.code == fa.FIB_ERR_INVALID_ARG
    assert fa.fib_attn_cache_evict_workspace_size(c, 0) == 0


def test_captured_and_replayed():
    """Lengths, weights and what to keep are read at the replay; a workspace full of anything serves."""
    r = rng(107)
    lens = [120, 64]
    c, ref = make_cache(r, "bf16", 2, 2, 16, lens, 9)
    plan, w = plan_for(), weights_of(r, c, 130)
    wd, keep = torch.from_numpy(w.copy()).cuda(), i32([200, 200])
    ws = torch.full((fa.fib_attn_cache_evict_workspace_size(c, 130),), 255, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fib_attn_cache_evict(plan, c, wd, keep, 3, 5, workspace=ws)
    for now in ([200, 200], [100, 64], [100, 40], [31, 31]):
        keep.copy_(i32(now))
        graph.replay()
        assert ref.evict(w, now, 3, 5, [0, 0])
        same_tables(c, ref)
        # up to four turns, each rounded: half a step of bf16 a turn, of a value at most as large as its pair
        k = c.k.double().cpu().numpy()
        assert np.array_equal(c.v.double().cpu().numpy(), ref.v)
        pair = np.hypot(ref.k[..., :32], ref.k[..., 32:])
        assert np.all(np.abs(k - ref.k) <= 4 * 2 * 2.0 ** -8 * np.concatenate([pair, pair], -1) + 1e-5)
        assert np.array_equal(wd.cpu().numpy(), w)


def test_on_a_stream_of_its_own():
    r = rng(108)
    c, ref = make_cache(r, "f32", 1, 2, 16, [50], 4)
    w = weights_of(r, c, 50)
    wd, keep, side = torch.from_numpy(w.copy()).cuda(), i32([20]), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fa.fib_attn_cache_evict(plan_for(), c, wd, keep, 1, 1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert ref.evict(w, [20], 1, 1, [0])
    same_tables(c, ref)
    close_rows(c, ref, "f32")


def test_many_sequences():
    r = rng(109)
    lens = [int(x) for x in r.integers(0, 60, 1024)]
    c, ref = make_cache(r, "f32", 1, 1, 16, lens, 4)
    run(c, ref, plan_for(), weights_of(r, c, 60), [int(x) for x in r.integers(2, 50, 1024)], 1, 1, "f32")


def test_decode_after_eviction_sees_what_is_left():
    """The dense decode over the evicted cache against the same rows in a cache of their own."""
    from oracle import cache_oracle as co
    r = rng(110)
    c, ref = make_cache(r, "f32", 1, 2, 16, [90, 40], 7)
    plan = plan_for(200)
    run(c, ref, plan, weights_of(r, c, 90), [37, 30], 2, 4, "f32")
    x = [draw(r, (2, 2, 1, 64), "f32") for _ in range(3)]
    o, lse = fa.fib_attn_dense_tree_decode(plan, 0, c, *(t[0] for t in x))
    O_ref, lse_ref = co.tree_attend(ref, 0, *(t[1] for t in x), [[-1], [-1]], [1, 1])
    # the cached keys are within 1e-5 of the oracle's: 64 products of them move a score by 64 * 5 * 1e-5 / 8 at most, 1e-4 as a rule
    assert np.abs(lse.double().cpu().numpy() - lse_ref).max() <= 1e-4
    assert np.abs(o.double().cpu().numpy() - O_ref).max() <= 1e-3
    assert math.isfinite(float(o.sum()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L,H,P,lens,keep,sink,recent", [
    (16, 5, 64, [5500], [2200], 70, 300),                           # 80 long ones: a block each
    (7, 7, 32, [6000, 17], [5990, 12], 3, 9),                       # 98, with one that is short
    (2, 3, 16, [700, 2100, 64, 5000], [699, 1000, 64, 33], 5, 20),  # 24: clusters, some with nothing to do
    (1, 2, 128, [300, 513], [257, 300], 130, 1),                    # 4 of few rows
    (5, 8, 16, [900, 800, 700, 640, 100], [400, 400, 699, 1, 0], 0, 0),  # 200
])
def test_blocks_that_share_rows(dtype, L, H, P, lens, keep, sink, recent):
    r = rng(112, L, H)
    c, ref = make_cache(r, dtype, L, H, P, lens, -(-max(lens) // P) + 1)
    run(c, ref, plan_for(1 << 13), weights_of(r, c, max(lens) + 1), keep, sink, recent, dtype)


def test_blocks_that_share_rows_of_shared_pages():
    """Replaced pages, a sink that stays shared, and one sequence that is left whole."""
    r = rng(113)
    lens = [2000, 1900, 1800, 1500]
    c, ref = make_cache(r, "bf16", 2, 2, 32, lens, 64, spare=200, share=[(1, 0, 50), (2, 0, 50)])
    run(c, ref, plan_for(1 << 12), weights_of(r, c, 2000), [1000, 1899, 300, 1500], 70, 100, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("captured", [True, False])
@pytest.mark.parametrize("lens,keeps", [([120, 64], ([100, 64], [40, 31])), ([6000], ([2500], [1999]))])
def test_a_replay_turns_as_the_plan_does_then(dtype, captured, lens, keeps):
    """The setting of the plan when the graph is replayed, not when the call was captured, says whether K is turned."""
    r = rng(114, *lens)
    c, ref = make_cache(r, dtype, 2, 2, 16, lens, -(-max(lens) // 16) + 1)
    plan, w = plan_for(8192), weights_of(r, c, max(lens))
    wd, keep = torch.from_numpy(w.copy()).cuda(), i32(lens)
    ws = torch.empty(fa.fib_attn_cache_evict_workspace_size(c, max(lens)), dtype=torch.uint8, device="cuda")
    fa.fib_attn_plan_set_rotation(plan, captured)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fib_attn_cache_evict(plan, c, wd, keep, 3, 5, workspace=ws)
    for turns, now in zip((not captured, captured), keeps):
        fa.fib_attn_plan_set_rotation(plan, turns)
        keep.copy_(i32(now))
        graph.replay()
        before = ref.k.copy()
        assert ref.evict(w, now, 3, 5, [0] * len(lens), turns)
        assert fa.fib_attn_cache_status(c) == fa.FIB_OK
        same_tables(c, ref)
        assert not np.array_equal(before, ref.k)
        if turns:
            close_rows(c, ref, dtype)
        else:
            assert np.array_equal(c.k.double().cpu().numpy(), ref.k) and np.array_equal(c.v.double().cpu().numpy(), ref.v)
        ref.k = c.k.double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("turns", [True, False])
def test_a_row_at_a_time(dtype, turns):
    """64 calls, each of which lets go of the first row, so that all others move by one place and, where the plan rotates, are turned and rounded
    64 times.  A rounding moves a pair by half a step of its size at most, and the factors (12 * 2^-24 for each of its two values) by less than
    2^-19: that, added up, is the bound of one pair.  Of all together it is what rounding 64 times gives, computed here in 64 bits between the roundings: a value
    that the kernel rounds to the other side, of its factors' error of a thousandth of a step, is one in a thousand."""
    from oracle.cache_oracle import turn
    from tests.test_gpu_cache import DT, HALF
    r = rng(115)
    n, length = 64, 200
    c, ref = make_cache(r, dtype, 1, 2, 16, [length], 13)
    plan = plan_for()
    fa.fib_attn_plan_set_rotation(plan, turns)
    rows = lambda pool: torch.as_tensor(pool)[0, ref.table[0]].transpose(0, 1).reshape(2, -1, 64)  # noqa: E731
    first, values = (rows(x)[:, n:length].clone() for x in (ref.k, ref.v))
    w = torch.arange(1.0, length + 1, device="cuda").expand(1, 1, 2, length).contiguous()
    for i in range(1, n + 1):
        fa.fib_attn_cache_evict(plan, c, w, i32([length - i]), 0, 0)
    assert fa.fib_attn_cache_status(c) == fa.FIB_OK and c.lens.tolist() == [length - n]
    got, got_v = (rows(x.double().cpu())[:, :length - n] for x in (c.k, c.v))
    assert torch.equal(got_v, values) and w[0, 0, 0, :length - n].tolist() == [float(x) for x in range(n + 1, length + 1)]
    if not turns:
        assert torch.equal(got, first)  # moved, whatever the number of calls
        return
    steps = first.numpy()
    for _ in range(n):
        steps = torch.from_numpy(turn(steps, -1)).to(DT[dtype]).double().numpy()
    want = turn(first.numpy(), -n)
    size = np.hypot(want[..., :32], want[..., 32:])
    error = got.numpy() - want
    assert (np.hypot(error[..., :32], error[..., 32:]) <= ((1 + HALF[dtype] + 2.0 ** -19) ** n - 1) * size).all()
    drift = np.linalg.norm(steps - want)
    if dtype == "bf16":
        assert 0.9 * drift <= np.linalg.norm(error) <= 1.1 * drift and 0.03 <= drift / np.linalg.norm(want) <= 0.05
    else:
        assert np.linalg.norm(error) <= n * 2.0 ** -22 * np.linalg.norm(want)
