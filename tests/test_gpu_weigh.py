"""The attention weight that new tokens give to cached rows against the oracle (needs a GPU).

Tolerance.  A term is exp(s - lse).  Errors of s: the rotation's (a pair's factors within 8 * 2^-24, of sum |q||k|/8 <= 10 here: 5e-6 at
worst), the operands' (bf16: none, float32: three of 2^-22 of the same sum, 7e-6) and the sum's (2^-24 of it a product of 16
dims: 3e-6); of the exponent, which is at most 25 in base 2: 2^-24 of that a rounding, twice: 3e-6; of exp2, 2^-22.  2e-5 in all at worst of
each term, and so of a sum of positive terms; a sum of N terms and the old weight adds N 2^-24 of itself."""
import math

import numpy as np
import pytest
import torch

from fibonacci_offset_sparse_gb300 import fib_attn as fa
from tests.test_gpu_cache import draw, i32, make_cache, plan_for, rng

pytestmark = pytest.mark.gpu
LEAVE = 7.0


def tolerance(new, old, terms):
    return 2e-5 * np.abs(new) + (terms + 1) * 2.0 ** -24 * (np.abs(new) + np.abs(old))


def setup(r, dtype, L, H, G, T, P, lens, n_new, rows=None, use_path=False):
    B = len(lens)
    c, ref = make_cache(r, dtype, L, H, P, lens, -(-max(lens + [1]) // P) + 1)
    q, qf = draw(r, (L, B, H * G, T, 64), dtype)
    lse = (r.standard_normal((L, B, H * G, T)) + 3.0).astype(np.float32)
    w = r.standard_normal((L, B, H, rows or max(lens) + 3)).astype(np.float32) ** 2
    path = [sorted(r.permutation(T)[:n].tolist()) + [0] * (T - n) for n in n_new] if use_path else None
    return c, ref, q, qf, lse, w, path


def run(c, ref, plan, q, qf, lse, w, n_new, path=None, first=None, turns=True):
    wd = torch.from_numpy(w.copy()).cuda()
    fa.fib_attn_cache_weigh(plan, c, q, torch.from_numpy(lse).cuda(), i32(n_new), wd, path=None if path is None else i32(path),
                            first=None if first is None else i32(first))
    want = w.astype(np.float64)
    ref.weigh(want, qf, lse.astype(np.float64), n_new, path, first, turns)
    got = wd.double().cpu().numpy()
    terms = q.shape[3] * (q.shape[2] // c.heads)
    # what the call adds: the oracle's from empty weights
    new = np.zeros_like(want)
    ref.weigh(new, qf, lse.astype(np.float64), n_new, path, [0] * len(n_new), turns)
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= tolerance(new, want - new, terms)) & ~((got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])
    for b, n in enumerate(n_new):  # what is not a row of the sequence, or of one that gained nothing, is as it was
        at = 0 if n == 0 else ref.lens[b]
        assert np.array_equal(got[:, b, :, at:], w[:, b, :, at:].astype(np.float64), equal_nan=True)
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("P,H,G,T,lens,n_new,use_path", [
    (16, 1, 1, 1, [1], [1], False),                                    # one token, the only one
    (16, 2, 1, 1, [33, 0, 64, 65], [1, 0, 1, 0], False),               # an empty sequence, some that take no part
    (64, 3, 2, 4, [200, 4, 129], [3, 4, 1], True),                     # 8 query rows, accepted paths
    (32, 2, 3, 3, [100, 7], [3, 2], True),                             # 9
    (16, 1, 1, 16, [127, 128, 129, 16], [16, 15, 1, 16], False),
    (128, 2, 1, 33, [300, 33, 40], [33, 33, 5], False),
    (16, 2, 4, 16, [600, 17], [16, 16], True),                         # 64
    (64, 1, 5, 13, [513, 511], [13, 2], False),                        # 65
    (256, 1, 1, 200, [1025, 200, 512], [200, 200, 150], False),        # several groups of 64 queries, prompts of their own
    (16, 1, 2, 520, [520, 1100], [520, 300], False),
    (64, 1, 16, 8, [260], [8], False),                                 # 16 query heads to a key head
    (64, 1, 1, 2, [1900, 1], [2, 1], False),                           # two columns of parts, runs over many blocks
    (16, 2, 2, 1, [1030, 15, 16], [1, 1, 1], False),
])
@pytest.mark.parametrize("kind", ["add", "set", "some"])
def test_weights(dtype, P, H, G, T, lens, n_new, use_path, kind):
    r = rng(200, P, H, G, T, len(lens))
    x = setup(r, dtype, 2, H, G, T, P, lens, n_new, use_path=use_path)
    first = {"add": None, "set": [0] * len(lens), "some": [max(0, n - 20) for n in lens]}[kind]
    run(x[0], x[1], plan_for(2048), x[2], x[3], x[4], x[5], n_new, path=x[6], first=first)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [2, 24])
def test_a_plan_that_does_not_rotate(dtype, T):
    r = rng(201, T)
    x = setup(r, dtype, 2, 2, 1, T, 16, [70, 30], [T, T])
    plan = plan_for(100)
    fa.fib_attn_plan_set_rotation(plan, False)
    run(x[0], x[1], plan, x[2], x[3], x[4], x[5], [T, T], turns=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G,T", [(1, 1), (2, 12), (1, 100)])
def test_what_is_not_seen_is_not_used(dtype, G, T):
    """NaN in rows behind the last one, in pages of others, in queries of nodes that were not taken, and in weights that begin anew."""
    r = rng(202, G, T)
    lens, n = [150, 131], [T, max(1, T - 1)]
    c, ref, q, qf, lse, w, path = setup(r, dtype, 1, 2, G, T, 64, lens, n, use_path=True)
    for b in range(2):
        page, row = ref.table[b][lens[b] // 64], lens[b] % 64
        c.k[:, page, :, row:] = math.nan
    held = {p for t, m in zip(ref.table, lens) for p in t[:-(-m // 64)]}
    for p in range(c.n_pages):
        if p not in held:
            c.k[:, p] = math.inf
    if T > 1:
        dead = [x for x in range(T) if x not in path[1][:n[1]]]
        q[:, 1, :, dead] = math.nan
        lse[:, 1, :, dead] = math.nan
    w[:, :, :, 140:] = math.nan
    got = run(c, ref, plan_for(), q, np.nan_to_num(qf), lse, w, n, path=path, first=[100, 131])
    assert np.isfinite(got[0, 0, :, :150]).all() and np.isfinite(got[0, 1, :, :131]).all() and np.isnan(got[0, 0, :, 150:]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G,T", [(1, 3), (1, 20), (2, 70)])
def test_infinite_and_nan_keys(dtype, G, T):
    """A score of an infinite key is what the formula says, and no other row's weight changes."""
    r = rng(203, G, T)
    c, ref, q, qf, lse, w, _ = setup(r, dtype, 1, 1, G, T, 16, [140], [T])
    plan = plan_for()
    fa.fib_attn_plan_set_rotation(plan, False)
    for row, dim, v in ((5, 3, math.inf), (50, 60, -math.inf), (9, 1, math.inf), (9, 2, -math.inf), (139, 7, math.inf), (100, 0, math.nan)):
        page = ref.table[0][row // 16]
        c.k[0, page, 0, row % 16, dim] = ref.k[0, page, 0, row % 16, dim] = v
    with np.errstate(invalid="ignore", over="ignore"):
        run(c, ref, plan, q, qf, lse, w, [T], turns=False)


def test_bad_sequences_are_reported_and_left():
    r = rng(204)
    lens, T = [50, 50, 50, 50, 50, 50], 4
    c, ref, q, qf, lse, w, _ = setup(r, "bf16", 2, 2, 3, T, 16, lens, [4] * 6, rows=50)
    plan = plan_for(60)

    def call(n_new, touched, rows=50, path=None, plan=plan):
        wd = torch.from_numpy(w[..., :rows].copy()).cuda()
        fa.fib_attn_cache_weigh(plan, c, q, torch.from_numpy(lse).cuda(), i32(n_new), wd, path=None if path is None else i32(path))
        assert fa.fib_attn_last_device_status(plan) == fa.FIB_ERR_DEVICE_ASSERT
        got = wd.cpu().numpy()
        for b in range(6):
            assert np.array_equal(got[:, b], w[:, b, :, :rows]) != (b in touched)

    call([5, -1, 4, 0, 4, 1], {2, 4, 5})
    c.lens[2], c.lens[4] = -3, 97  # the table holds 5 pages
    call([4, 4, 4, 4, 4, 4], {0, 1, 3, 5})
    c.lens[2], c.lens[4] = 3, 61   # fewer rows than new ones; more than the plan holds
    call([4, 4, 4, 4, 4, 4], {0, 1, 3, 5})
    c.lens.fill_(50)
    call([4] * 6, set(), rows=49)
    call([4] * 6, set(), plan=plan_for(49))
    # a page outside the pool: its rows alone are left
    for bad in (-1, c.n_pages, 2 ** 31 - 1):
        was = int(c.table[1, 2])
        c.table[1, 2] = bad
        wd = torch.from_numpy(w.copy()).cuda()
        fa.fib_attn_cache_weigh(plan, c, q, torch.from_numpy(lse).cuda(), i32([4] * 6), wd)
        assert fa.fib_attn_last_device_status(plan) == fa.FIB_ERR_DEVICE_ASSERT
        got = wd.cpu().numpy()
        assert np.array_equal(got[:, 1, :, 32:48], w[:, 1, :, 32:48])
        assert (got[:, 1, :, :32] != w[:, 1, :, :32]).any() and (got[:, 1, :, 48:50] != w[:, 1, :, 48:50]).any()
        c.table[1, 2] = was
    for bad in (-1, 4):
        fa.fib_attn_cache_weigh(plan, c, q, torch.from_numpy(lse).cuda(), i32([4] * 6), torch.zeros(2, 6, 2, 50, device="cuda"),
                                path=i32([[0, 1, bad, 3]] * 6))
        assert fa.fib_attn_last_device_status(plan) == fa.FIB_ERR_DEVICE_ASSERT
    run(c, ref, plan, q, qf, lse, w, [4] * 6)


def test_refusals():
    r = rng(205)
    c, ref, q, qf, lse, w, _ = setup(r, "bf16", 2, 2, 2, 4, 16, [20, 20], [4, 4])
    plan, good = plan_for(), dict(q=q, lse=torch.from_numpy(lse).cuda(), n_new=i32([4, 4]), weights=torch.from_numpy(w).cuda())
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(q=q[:1]), dict(q=q.transpose(3, 4)), dict(q=q[..., ::2]), dict(q=q.cpu()), dict(lse=good["lse"].double()),
               dict(lse=good["lse"][:, :, :1]), dict(n_new=i32([4])), dict(n_new=i32([4, 4]).long()), dict(weights=good["weights"][:, :1]),
               dict(path=i32([[0, 1, 2, 3]])), dict(first=i32([0])), dict(workspace=torch.zeros(8, device="cuda")[::2])):
        with pytest.raises(ValueError):
            fa.fib_attn_cache_weigh(plan, c, **{**good, **kw})
    for kw in (dict(q=q[:, :, :3].contiguous(), lse=good["lse"][:, :, :3].contiguous()), dict(weights=good["weights"][..., :0]),
               dict(workspace=torch.zeros(16, device="cuda", dtype=torch.uint8)),
               dict(q=q.repeat(1, 2, 1, 1, 1), lse=good["lse"].repeat(1, 2, 1, 1), n_new=i32([4] * 4))):
        with pytest.raises(fa.FibAttnError) as e:
            fa.fib_attn_cache_weigh(plan, c, **{**good, **kw})
        assert e.value.code == fa.FIB_ERR_INVALID_ARG
    for x in ((3, 4, 1), (0, 4, 1), (2, 3, 1), (2, 0, 1), (2, 4, 0), (2, 4, (1 << 20) + 1), (2, 1026, 1)):
        assert fa.fib_attn_cache_weigh_workspace_size(c, *x) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G,T", [(2, 3), (1, 40)])
def test_captured_and_replayed_and_the_same_every_time(dtype, G, T):
    r = rng(206, G, T)
    lens = [200, 77, 160]
    c, ref, q, qf, lse, w, _ = setup(r, dtype, 2, 2, G, T, 16, lens, [T] * 3)
    plan, n, ld = plan_for(), i32([T] * 3), torch.from_numpy(lse).cuda()
    wd = torch.from_numpy(w.copy()).cuda()
    size = fa.fib_attn_cache_weigh_workspace_size(c, 3, 2 * G, T)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fib_attn_cache_weigh(plan, c, q, ld, n, wd, workspace=ws)
    for now in ([T, T, T], [0, 1, T - 1], [T, 0, 2]):
        before = wd.cpu().numpy()
        n.copy_(i32(now))
        graph.replay()
        first = wd.clone()
        run(c, ref, plan, q, qf, lse, before, now)
        again = torch.from_numpy(before).cuda()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        fa.fib_attn_cache_weigh(plan, c, q, ld, n, again, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(first, again)  # bit for bit, whatever the workspace held


def test_many_sequences():
    r = rng(207)
    lens = [int(x) for x in r.integers(1, 40, 1024)]
    n = [int(x) for x in r.integers(0, 2, 1024)]
    x = setup(r, "bf16", 1, 1, 1, 1, 16, lens, n)
    run(x[0], x[1], plan_for(), *x[2:6], n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 12, 100])
def test_commit_decode_weigh_evict_as_they_are_used(dtype, T):
    """Prompts and steps of T tokens: the weight that a step adds up is one for each token and query head, as softmax's is; then the
    cache is cut and goes on."""
    r = rng(208, T)
    L, H, G, B, P = 2, 2, 2, 2, 16
    plan = plan_for(1024)
    c = fa.fib_attn_cache_create(L, H, P, 64, B, 20, torch.float32 if dtype == "f32" else torch.bfloat16)
    w = torch.full((L, B, H, 300), math.nan, device="cuda")
    dropped, keep = i32([0, 0]), i32([60 + T, 60 + T])
    for step in range(4):
        n = [T, T - 1 if T > 1 else 1]
        kn, vn, q = (draw(r, s, dtype)[0] for s in ((L, B, H, T, 64), (L, B, H, T, 64), (L, B, H * G, T, 64)))
        lse = torch.empty((L, B, H * G, T), device="cuda")
        if T <= fa.FIB_MAX_DRAFTS:
            for layer in range(L):
                fa.fib_attn_dense_tree_decode(plan, layer, c, q[layer], kn[layer], vn[layer], lse=lse[layer])
            before = c.lens.tolist()
            fa.fib_attn_cache_commit(plan, c, kn, vn, i32(n))
        else:
            fa.fib_attn_cache_commit(plan, c, kn, vn, i32(n))
            before = [x - m for x, m in zip(c.lens.tolist(), n)]
            for layer in range(L):  # scores in torch: what a prompt's attention gives
                for b in range(B):
                    pages = c.table[b, :-(-int(c.lens[b]) // P)].long()
                    K = c.k[layer, pages].transpose(0, 1).reshape(H, -1, 64)[:, :int(c.lens[b])].double()
                    at = torch.arange(before[b], before[b] + T, device="cuda")
                    m = torch.arange(32, device="cuda", dtype=torch.float64)
                    a = at.double()[:, None] * 10000.0 ** (-m / 32)
                    x = q[layer, b].double()
                    x = torch.cat([x[..., :32] * a.cos() - x[..., 32:] * a.sin(), x[..., :32] * a.sin() + x[..., 32:] * a.cos()], -1)
                    s = (x.view(H, G, T, 64) @ K[:, None].transpose(-1, -2) / 8).masked_fill(torch.arange(K.shape[1], device="cuda") > at[:, None], -math.inf)
                    lse[layer, b] = torch.logsumexp(s, -1).view(H * G, T)
        was = w.nan_to_num().double()
        fa.fib_attn_cache_weigh(plan, c, q, lse, i32(n), w)
        assert c.lens.tolist() == [x + m for x, m in zip(before, n)]
        for b in range(B):
            live = w[:, b, :, :int(c.lens[b])].double()
            assert torch.isfinite(live).all()
            gain = live.sum(-1) - was[:, b, :, :before[b]].sum(-1)
            # Each row of a softmax adds to one; lse is float32, within 3e-5.  In bf16 the decode's lse has the new keys as they were
            # given, turned in float32, and the cache has them rounded, each element by 2^-8 of it at most: a new row's score is off by
            # 2^-8 sum |q_d k_d| / 8 <= 2^-8 |q| |k| / 8, with |q| |k| below 100 for these a twentieth, and the token's sum by no more.
            new = 0.05 if dtype == "bf16" and T <= fa.FIB_MAX_DRAFTS else 0.0
            assert (gain - n[b] * G).abs().max() <= n[b] * G * (1e-4 + new) + 1e-4
        fa.fib_attn_cache_evict(plan, c, w, keep, 4, T, dropped=dropped)
    assert fa.fib_attn_cache_status(c) == fa.FIB_OK and fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    assert (c.lens <= keep).all() and [int(x) + int(y) for x, y in zip(c.lens, dropped)] == [4 * T, 4 * (T - 1 if T > 1 else 1)]


def test_a_wait_that_runs_out():
    """A copy that never comes: the call ends, reports, and the next one is right."""
    r = rng(209)
    c, ref, q, qf, lse, w, _ = setup(r, "bf16", 2, 2, 1, 20, 16, [600, 100], [20, 20])
    plan = plan_for(1000)
    fa.fib_attn_plan_set_debug(plan, True, 2_000_000)
    fa.fib_attn_cache_weigh(plan, c, q, torch.from_numpy(lse).cuda(), i32([20, 20]), torch.from_numpy(w).cuda())
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_ERR_TIMEOUT
    fa.fib_attn_plan_set_debug(plan, False, 1_000_000_000)
    run(c, ref, plan, q, qf, lse, w, [20, 20])


@pytest.mark.parametrize("dtype,G,T", [("f32", 1, 1), ("f32", 2, 10), ("f32", 2, 200), ("bf16", 1, 2), ("bf16", 1, 30), ("bf16", 2, 30), ("bf16", 1, 200)])
def test_a_limit_too_short_for_a_copy(dtype, G, T):
    """The call ends and says so, or was quick enough; the next one is right."""
    r = rng(215, G, T)
    lens, n = [900, 300], [T, T]
    c, ref, q, qf, lse, w, _ = setup(r, dtype, 1, 2, G, T, 16, lens, n)
    plan = plan_for(1000)
    fa.fib_attn_plan_set_debug(plan, False, 1000)
    for _ in range(3):
        fa.fib_attn_cache_weigh(plan, c, q, torch.from_numpy(lse).cuda(), i32(n), torch.from_numpy(w).cuda())
        assert fa.fib_attn_last_device_status(plan) in (fa.FIB_OK, fa.FIB_ERR_TIMEOUT)
    fa.fib_attn_plan_set_debug(plan, False, 1_000_000_000)
    run(c, ref, plan, q, qf, lse, w, n)


@pytest.mark.parametrize("P,H,G,T,lens,n_new", [
    (16, 1, 1, 65, [65], [65]),                     # 5 units, eight warps each
    (32, 1, 2, 40, [500, 70], [40, 33]),            # 37: eight
    (16, 2, 1, 130, [1500, 300], [130, 1]),         # 226: four
    (64, 3, 1, 90, [1500, 1200], [90, 0]),          # 282: four
    (16, 2, 3, 30, [3000, 1700], [30, 30]),         # 588: two
    (128, 4, 1, 70, [2500, 2300], [70, 70]),        # 1204: one
])
@pytest.mark.parametrize("first", [False, True])
def test_warps_that_share_rows(P, H, G, T, lens, n_new, first):
    r = rng(216, H, G, T)
    x = setup(r, "f32", 1, H, G, T, P, lens, n_new)
    run(x[0], x[1], plan_for(4000), *x[2:6], n_new, first=[0, 3] if first and len(lens) == 2 else None)


def test_a_long_call_is_no_wait_that_runs_out():
    """A limit that every step keeps to, and that a block's whole work, 1024 chunks of queries, does not."""
    r = rng(213)
    c = fa.fib_attn_cache_create(1, 1, 64, 150, 1, 150, torch.bfloat16)
    plan = plan_for(1 << 14)
    kn, q = (draw(r, s, "bf16")[0] for s in ((1, 1, 1, 9000, 64), (1, 1, 16, 8192, 64)))
    fa.fib_attn_cache_commit(plan, c, kn, kn, i32([9000]))
    lse = torch.full((1, 1, 16, 8192), 5.0, device="cuda")
    ws = []
    for ns in (1_000_000_000, 400_000):
        fa.fib_attn_plan_set_debug(plan, False, ns)
        ws.append(torch.zeros((1, 1, 1, 9000), device="cuda"))
        fa.fib_attn_cache_weigh(plan, c, q, lse, i32([8192]), ws[-1], first=i32([0]))
        assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    assert torch.equal(*ws) and (ws[0] > 0).all()


@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("bf16", 3), ("bf16", 20), ("bf16", 100), ("f32", 20)])
def test_pages_beyond_32_bits(dtype, T):
    """Pages at the end of a pool whose K and V have more than 2^31 values a layer: weights and eviction as in a small pool of the same rows."""
    r = rng(210, T)
    P, H, n = 64, 8, 150
    small = fa.fib_attn_cache_create(2, H, P, 8, 1, 4, torch.float32 if dtype == "f32" else torch.bfloat16)
    pages = (1 << 32) // (H * P * 64) // (2 if dtype == "f32" else 1) + 8
    big = fa.fib_attn_cache_create(2, H, P, pages, 1, 4, small.dtype, k=torch.empty((2, pages, H, P, 64), dtype=small.dtype, device="cuda"),
                                   v=torch.empty((2, pages, H, P, 64), dtype=small.dtype, device="cuda"))
    big.refs[:pages - 8] = 1  # the free ones are the last
    plan = plan_for(400)
    kn, vn, q = (draw(r, s, dtype)[0] for s in ((2, 1, H, n, 64), (2, 1, H, n, 64), (2, 1, H, T, 64)))
    lse = torch.full((2, 1, H, T), 4.0, device="cuda")
    ws = []
    for c in (small, big):
        w = torch.zeros((2, 1, H, n), device="cuda")
        fa.fib_attn_cache_commit(plan, c, kn, vn, i32([n]))
        fa.fib_attn_cache_weigh(plan, c, q, lse, i32([T]), w, first=i32([0]))
        ws.append(w.clone())
        fa.fib_attn_cache_evict(plan, c, w, i32([90]), 3, 20)
        ws.append(w)
    assert fa.fib_attn_cache_status(big) == fa.FIB_OK and fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    assert torch.equal(ws[0], ws[2]) and torch.equal(ws[1], ws[3])
    rows = [[x[:, c.table[0, :2].long()] for x in (c.k, c.v)] for c in (small, big)]
    assert int(big.table[0, 0]) == pages - 8
    for a, b in zip(*rows):
        live = torch.arange(2 * P, device="cuda").view(2, P) < 90
        assert torch.equal(a.transpose(2, 3)[:, live], b.transpose(2, 3)[:, live])


def test_one_plan_on_two_streams():
    """Calls with workspaces of their own side by side."""
    r = rng(211)
    x = [setup(r, "bf16", 2, 4, 1, T, 16, [900, 300], [T, T]) for T in (1, 40, 150)]
    plan = plan_for(1000)
    streams = [torch.cuda.Stream() for _ in x]
    done = []
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (c, ref, q, qf, lse, w, _p) in zip(streams, x):
            with torch.cuda.stream(s):
                wd = torch.from_numpy(w).cuda()
                fa.fib_attn_cache_weigh(plan, c, q, torch.from_numpy(lse).cuda(), i32([q.shape[3]] * 2), wd)
                done.append(wd)
    torch.cuda.synchronize()
    for (c, ref, q, qf, lse, w, _p), *got in zip(x, done[:3], done[3:6], done[6:]):
        assert all(torch.equal(got[0], g) for g in got)
        want = w.astype(np.float64)
        ref.weigh(want, qf, lse.astype(np.float64), [q.shape[3]] * 2)
        assert np.allclose(got[0].double().cpu().numpy(), want, rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G,T", [(1, 1), (2, 4), (1, 40), (3, 90)])
def test_long_sequences(dtype, G, T):
    r = rng(212, G, T)
    lens, n = [9001, 4000], [T, max(1, T // 2)]
    x = setup(r, dtype, 1, 2, G, T, 32, lens, n)
    run(x[0], x[1], plan_for(1 << 14), *x[2:6], n, first=[0, 5])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_query_rows_of_an_odd_number_of_heads(dtype):
    """More rows to rotate than the device holds at once, whose threads take several heads each."""
    r = rng(214)
    lens, n = [700, 600], [600, 333]
    x = setup(r, dtype, 16, 5, 1, 600, 64, lens, n)
    run(x[0], x[1], plan_for(1000), *x[2:6], n, first=[0, 267])


def test_a_tile_that_few_queries_see_is_no_wait_that_runs_out():
    """Rows from 384 on are seen by the last of 1600 chunks of queries alone: their sums begin after a time that no single step takes."""
    L, G, T = 77, 512, 400  # (as many layers as leave every block a task of four tiles)
    c = fa.fib_attn_cache_create(L, 1, 16, 25, 1, 25, torch.bfloat16)
    plan = plan_for(512, alpha=[1.0] * L)
    g = torch.Generator(device="cuda").manual_seed(217)
    kn = torch.empty((L, 1, 1, T, 64), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    q = torch.empty((L, 1, G, T, 64), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    fa.fib_attn_cache_commit(plan, c, kn, kn, i32([T]))
    lse = torch.full((L, 1, G, T), 5.0, device="cuda")
    workspace = torch.empty(fa.fib_attn_cache_weigh_workspace_size(c, 1, G, T), dtype=torch.uint8, device="cuda")
    ws = []
    for ns in (1_000_000_000, 200_000):
        fa.fib_attn_plan_set_debug(plan, False, ns)
        ws.append(torch.zeros((L, 1, 1, T), device="cuda"))
        fa.fib_attn_cache_weigh(plan, c, q, lse, i32([T]), ws[-1], first=i32([0]), workspace=workspace)
        assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    assert torch.equal(*ws) and (ws[0] > 0).all()


@pytest.mark.parametrize("dtype,G,T", [("f32", 1, 1), ("f32", 2, 10), ("f32", 2, 200), ("bf16", 1, 2), ("bf16", 1, 30), ("bf16", 2, 30), ("bf16", 1, 200)])
def test_a_short_limit_is_kept_or_reported(dtype, G, T):
    """Limits from too short for any copy to long enough: a call that reports nothing has given every weight."""
    r = rng(218, G, T)
    lens, n = [900, 300], [T, T]
    c, ref, q, qf, lse, w, _ = setup(r, dtype, 1, 2, G, T, 16, lens, n)
    plan, want, new = plan_for(1000), w.astype(np.float64), np.zeros(w.shape)
    ref.weigh(want, qf, lse.astype(np.float64), n)
    ref.weigh(new, qf, lse.astype(np.float64), n, None, [0, 0])
    ld, nd, kept = torch.from_numpy(lse).cuda(), i32(n), []
    for ns in (1000, 1500, 2500, 5000, 10_000, 100_000, 1_000_000_000):
        fa.fib_attn_plan_set_debug(plan, False, ns)
        for _ in range(8):
            wd = torch.from_numpy(w).cuda()
            fa.fib_attn_cache_weigh(plan, c, q, ld, nd, wd)
            status = fa.fib_attn_last_device_status(plan)
            assert status in (fa.FIB_OK, fa.FIB_ERR_TIMEOUT)
            if status == fa.FIB_OK:
                got = wd.double().cpu().numpy()
                assert (np.abs(got - want) <= tolerance(new, want - new, T * G)).all(), ns
                kept.append(ns)
    assert kept.count(1_000_000_000) == 8


@pytest.mark.parametrize("dtypes,Ts", [(("bf16", "bf16", "bf16"), (1, 40, 150)), (("f32", "f32", "bf16"), (3, 20, 60)), (("bf16", "bf16", "bf16"), (200, 200, 200))])
def test_calls_that_are_released_together(dtypes, Ts):
    """One plan; streams whose calls all stand in line behind one event, with workspaces of their own: bit for bit what the calls give alone."""
    r = rng(219, *Ts)
    lens = [1500, 300, 700]
    plan, calls = plan_for(2000), []
    for dtype, T in zip(dtypes, Ts):
        c, _, q, _, lse, w, _ = setup(r, dtype, 8, 4, 1, T, 16, lens, [T] * 3)
        n, lse, w = i32([T] * 3), torch.from_numpy(lse).cuda(), torch.from_numpy(w).cuda()
        size = fa.fib_attn_cache_weigh_workspace_size(c, 3, 4, T)
        alone = w.clone()
        fa.fib_attn_cache_weigh(plan, c, q, lse, n, alone)
        assert not torch.equal(alone, w)
        outs = [w.clone() for _ in range(6)]
        calls.append((torch.cuda.Stream(), c, q, lse, n, torch.empty(size, dtype=torch.uint8, device="cuda"), outs, alone))
    torch.cuda.synchronize()
    gate = torch.cuda.Event()
    torch.cuda._sleep(60_000_000)  # some 30 ms, in which all calls are put in line
    gate.record()
    for s, *_ in calls:
        s.wait_event(gate)
    for i in range(6):
        for s, c, q, lse, n, workspace, outs, _ in calls:
            fa.fib_attn_cache_weigh(plan, c, q, lse, n, outs[i], workspace=workspace, stream=s)
    in_line = not gate.query()
    torch.cuda.synchronize()
    assert in_line and fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    for *_, outs, alone in calls:
        assert all(torch.equal(x, alone) for x in outs)
