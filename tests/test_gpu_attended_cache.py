"""Calls of the paged cache in any order with weighing and eviction among them, batches smaller than the cache, and the other calls of a
plan that does not rotate (needs a GPU).  Tolerances are those of the calls' own tests."""
import numpy as np
import pytest
import torch

import oracle
from fibonacci_offset_sparse_gb300 import fib_attn as fa
from fibonacci_offset_sparse_gb300.autograd import fib_attention
from oracle.cache_oracle import turn
from tests.test_gpu_cache import DT, HALF, close_rows, draw, i32, make_cache, plan_for, rng, same_tables
from tests.test_gpu_weigh import run as weigh_and_compare, setup, tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seed", [1, 2, 3, 4])
def test_a_walk(dtype, seed):
    """Commits, forks, compactions, weighings and evictions as they come; whatever fails for want of pages changes nothing."""
    r = rng(400, seed)
    L, H, G, P, S, room = 2, 2, int(r.integers(1, 4)), int(r.choice([16, 32])), 5, 150
    c, ref = make_cache(r, dtype, L, H, P, [0] * S, -(-room // P), spare=int(r.integers(14, 30)))
    plan = plan_for(room)
    w = np.zeros((L, S, H, room), np.float32)
    wd = torch.from_numpy(w.copy()).cuda()
    dropped, d_ref = i32([0] * S), [0] * S
    done = {"commit": 0, "fork": 0, "compact": 0, "evict": 0}
    for step in range(40):
        op = r.choice(["commit", "commit", "commit", "fork", "compact", "evict", "evict"])
        before = [t.clone() for t in (c.meta, c.k, c.v)]
        if op == "commit":
            T = int(r.choice([1, 3, 20, 40]))
            n = [int(min(r.integers(0, T + 1), room - x)) for x in ref.lens]
            path = [sorted(r.permutation(T)[:m].tolist()) + [0] * (T - m) for m in n] if r.random() < 0.5 else None
            kn, kf = draw(r, (L, S, H, T, 64), dtype)
            vn, vf = draw(r, (L, S, H, T, 64), dtype)
            fa.fib_attn_cache_commit(plan, c, kn, vn, i32(n), path=None if path is None else i32(path))
            if not ref.commit(kf, vf, n, path):
                assert fa.fib_attn_cache_status(c) == fa.FIB_ERR_NO_PAGES and all(torch.equal(a, b) for a, b in zip(before, (c.meta, c.k, c.v)))
                continue
            same_tables(c, ref)
            close_rows(c, ref, dtype)
            ref.k = c.k.double().cpu().numpy()
            q, qf = draw(r, (L, S, H * G, T, 64), dtype)
            lse = (r.standard_normal((L, S, H * G, T)) + 3.0).astype(np.float32)
            first = [int(r.integers(0, x + 1)) for x in ref.lens] if r.random() < 0.5 else None
            fa.fib_attn_cache_weigh(plan, c, q, torch.from_numpy(lse).cuda(), i32(n), wd, path=None if path is None else i32(path),
                                    first=None if first is None else i32(first))
            want, new = w.astype(np.float64), np.zeros(w.shape)
            ref.weigh(want, qf, lse.astype(np.float64), n, path, first)
            ref.weigh(new, qf, lse.astype(np.float64), n, path, [0] * S)
            got = wd.double().cpu().numpy()
            assert (np.abs(got - want) <= tolerance(new, want - new, T * G)).all()
            w = wd.cpu().numpy()
        elif op == "fork":
            src = [int(r.integers(-1, S)) if r.random() < 0.4 else b for b in range(S)]
            fa.fib_attn_cache_fork(c, i32(src))
            ref.fork(src)
            w = w[:, [max(x, 0) for x in src]].copy()  # weights go with their sequences
            wd = torch.from_numpy(w.copy()).cuda()
        elif op == "compact":
            remap = fa.fib_attn_cache_compact(c)
            assert remap.cpu().tolist() == ref.compact()[0]
        else:
            sink, recent = int(r.choice([0, 1, 5, 20])), int(r.choice([0, 2, 10]))
            keep = [int(x if r.random() < 0.3 else max(sink + recent, r.integers(0, x + 1))) for x in ref.lens]
            fa.fib_attn_cache_evict(plan, c, wd, i32(keep), sink, recent, dropped=dropped)
            if not ref.evict(w, keep, sink, recent, d_ref):
                assert fa.fib_attn_cache_status(c) == fa.FIB_ERR_NO_PAGES and all(torch.equal(a, b) for a, b in zip(before, (c.meta, c.k, c.v)))
                continue
            assert np.array_equal(wd.cpu().numpy(), w) and dropped.cpu().tolist() == d_ref
        assert fa.fib_attn_cache_status(c) == fa.FIB_OK and fa.fib_attn_last_device_status(plan) == fa.FIB_OK
        done[op] += 1
        same_tables(c, ref)
        close_rows(c, ref, dtype)
        assert all(ref.refs[:int(c.state[0])])  # no free page lies below the bound
        ref.k = c.k.double().cpu().numpy()
    assert all(done.values())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G,T", [(1, 1), (2, 3), (1, 30), (1, 60), (2, 90)])
def test_a_batch_smaller_than_the_cache(dtype, G, T):
    r = rng(401, G, T)
    lens, B = [140, 95, 130, 100], 2
    c, ref, q, qf, lse, w, _ = setup(r, dtype, 3, 2, G, T, 16, lens, [T] * 4)
    weigh_and_compare(c, ref, plan_for(200), q[:, :B].contiguous(), qf[:, :B], np.ascontiguousarray(lse[:, :B]), w, [T, max(1, T - 1)])


def attended(q, k, v, at=None):
    """Dense causal softmax attention of rows as they are, float64."""
    s = np.einsum("bhid,bhjd->bhij", q, k) / 8
    i = np.arange(q.shape[2])[:, None] if at is None else np.array([[at]])
    s = np.where(np.arange(k.shape[2]) <= i, s, -np.inf)
    m = s.max(-1, keepdims=True)
    e = np.exp(s - m)
    return np.einsum("bhij,bhjd->bhid", e / e.sum(-1, keepdims=True), v), (m + np.log(e.sum(-1, keepdims=True)))[..., 0]


def test_the_dense_forward_of_a_plan_that_does_not_rotate():
    """Weights and K' are bf16 in it: half a step of each, 2^-8, twice, of scores below 4 and of values below 5 in the mean of a few dozen."""
    r = rng(402)
    plan = plan_for(300)
    (q, qf), (k, kf), (v, vf) = (draw(r, (2, 3, 300, 64), "bf16") for _ in range(3))
    rotated = fa.fib_attn_dense_fwd(plan, q, k, v)
    fa.fib_attn_plan_set_rotation(plan, False)
    o, lse = fa.fib_attn_dense_fwd(plan, q, k, v)
    want, lse_want = attended(qf, kf, vf)
    assert np.abs(o.double().cpu().numpy() - want).max() <= 4e-2 and np.abs(lse.double().cpu().numpy() - lse_want).max() <= 2e-2
    # and far from what the plan gives that rotates
    assert float((o - rotated[0]).abs().max()) > 0.2


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mode", ["mask", "interp"])
def test_the_decode_of_a_plan_that_does_not_rotate(dtype, mode):
    """One token over a contiguous cache: the oracle, which rotates, is given the rows turned back."""
    r = rng(403)
    N, W, alpha = 150, 8, 1.2345
    plan = fa.fib_attn_plan_create(fa.FIB_BASE_FIBONACCI, [alpha], W, N, fa.FIB_MODE_MASK if mode == "mask" else fa.FIB_MODE_INTERP)
    (q, qf), (k, kf), (v, vf) = (draw(r, (2, 3, N, 64), dtype) for _ in range(3))
    fa.fib_attn_plan_set_rotation(plan, False)
    back = lambda x: turn(x, -np.arange(N))  # noqa: E731
    want, lse_want = oracle.attend(back(qf), back(kf), vf, alpha, oracle.fibonacci_base(), W, mode)
    for pos in (0, 7, 77, N - 1):
        o, lse = fa.fib_attn_decode(plan, 0, pos, q[:, :, pos].contiguous(), k, v)
        err = np.abs(o.double().cpu().numpy() - want[:, :, pos])
        assert (err - HALF[dtype] * np.abs(want[:, :, pos])).max() <= 1.5e-4 and np.abs(lse.double().cpu().numpy() - lse_want[:, :, pos]).max() <= 3e-5


@pytest.mark.parametrize("mode", ["mask", "interp"])
def test_a_training_step_in_bf16_of_a_plan_that_does_not_rotate(mode):
    """Forward and backward by the prepared rows, against the oracle given the rows turned back; its gradients are turned to the rows'."""
    r = rng(404)
    N, W, alpha = 128, 8, 1.2345
    plan = fa.fib_attn_plan_create(fa.FIB_BASE_FIBONACCI, [alpha], W, N, fa.FIB_MODE_MASK if mode == "mask" else fa.FIB_MODE_INTERP)
    fa.fib_attn_plan_set_rotation(plan, False)
    rows = [draw(r, (2, 2, N, 64), "bf16") for _ in range(4)]
    q, k, v = (x[0].requires_grad_() for x in rows[:3])
    o = fib_attention(plan, 0, q, k, v)
    (o.float() * rows[3][0].float()).sum().backward()
    back = lambda x: turn(x, -np.arange(N))  # noqa: E731
    ref = back(rows[0][1]), back(rows[1][1]), rows[2][1]
    want, _ = oracle.attend(*ref, alpha, oracle.fibonacci_base(), W, mode)
    assert (np.abs(o.detach().double().cpu().numpy() - want) - HALF["bf16"] * np.abs(want)).max() <= 1e-2
    rq, rk, rv, _ = oracle.attend_bwd(*ref, rows[3][1], alpha, oracle.fibonacci_base(), W, mode)
    for x, g in ((q, turn(rq, np.arange(N))), (k, turn(rk, np.arange(N))), (v, rv)):
        assert x.grad.dtype == DT["bf16"]
        assert np.linalg.norm(x.grad.double().cpu().numpy() - g) <= 2e-2 * np.linalg.norm(g)
