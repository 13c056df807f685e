"""Rotary positions on the GPU against binary64: layouts, parts of the head, scalings, positions, strides, the transposed map,
gradients, refusals; and attention by a plan that does not rotate.

Tolerance: e^{i p theta} is the product of two float32 table entries (each off by sqrt(2) 2^-24 at most) rounded twice more and
scaled: 8 * 2^-24 amplitude is above their sum; the two products and the sum of a pair add 3 * 2^-24.  So 12 * 2^-24 amplitude
(|a| + |b|), and half a step of bf16, 2^-8 of the value, where the output is that."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from fibonacci_offset_sparse_gb300 import fib_attn as fa
from fibonacci_offset_sparse_gb300.autograd import fib_attention, rotary
from oracle.cache_oracle import turn

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def pairs(R, layout):
    m = np.arange(R // 2)
    return (m, m + R // 2) if layout == fa.FIB_ROPE_HALF else (2 * m, 2 * m + 1)


def reference(x, pos, theta, amp, layout, transpose=False):
    """(rotated x, the tolerance's |a| + |b|), binary64; x [B, H, N, 64], pos [B, N]."""
    R = 2 * len(theta)
    i, j = pairs(R, layout)
    a = pos[:, None, :, None] * np.asarray(theta) * (-1 if transpose else 1)
    c, s = amp * np.cos(a), amp * np.sin(a)
    y, size = x.copy(), np.zeros_like(x)
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., i] * s + x[..., j] * c
    size[..., i] = size[..., j] = amp * (np.abs(x[..., i]) + np.abs(x[..., j]))
    return y, size


def check(got, x, pos, theta, amp, layout, dtype, transpose=False):
    want, size = reference(x.double().cpu().numpy(), np.asarray(pos, np.float64), theta, amp, layout, transpose)
    err = np.abs(got.double().cpu().numpy() - want)
    tol = 12 * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)
    tol[size == 0] = 0  # what is only copied is equal
    assert (err <= tol).all(), float((err - tol).max())


def rand(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", [fa.FIB_ROPE_HALF, fa.FIB_ROPE_INTERLEAVED])
@pytest.mark.parametrize("R", [64, 48, 32, 16, 2, 6, 20, 62])
@pytest.mark.parametrize("B,Hq,Hk,N", [(1, 1, 0, 1), (2, 5, 2, 33), (3, 3, 3, 130)])
def test_layouts_and_parts(dtype, layout, R, B, Hq, Hk, N):
    rope = fa.fib_attn_rope_create(N + 1, rot_dim=R, layout=layout)
    q, k = rand((B, Hq, N, 64), dtype, 1), rand((B, Hk, N, 64), dtype, 2) if Hk else None
    pos = np.tile(np.arange(N), (B, 1))
    theta = fa.fib_attn_rope_frequencies(R)
    for transpose in (False, True):
        qo, ko = fa.fib_attn_rotary(rope, q, k, transpose=transpose)
        check(qo, q, pos, theta, 1.0, layout, dtype, transpose)
        if Hk:
            check(ko, k, pos, theta, 1.0, layout, dtype, transpose)
        else:
            assert ko is None
    assert fa.fib_attn_rope_status(rope) == fa.FIB_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scaling,factor,amplitude", [(fa.FIB_ROPE_LINEAR, 8.0, None), (fa.FIB_ROPE_NTK, 4.0, 1.0), (fa.FIB_ROPE_YARN, 16.0, None),
                                                      (fa.FIB_ROPE_PLAIN, 1.0, 2.5)])
def test_scalings_far_positions(dtype, scaling, factor, amplitude):
    N = 1 << 20
    rope = fa.fib_attn_rope_create(N, scaling=scaling, factor=factor, amplitude=amplitude)
    pos = np.array([[0, 1, 63, 64, 65, 4095, 131071, N - 1], [N - 1, N - 64, N - 65, 777777, 5, 0, 2, 1]])
    q = rand((2, 3, 8, 64), dtype, 3)
    out, _ = fa.fib_attn_rotary(rope, q, pos=torch.tensor(pos, dtype=torch.int32, device="cuda"))
    amp = amplitude if amplitude is not None else 0.1 * math.log(factor) + 1 if scaling == fa.FIB_ROPE_YARN else 1.0
    check(out, q, pos, fa.fib_attn_rope_frequencies(64, scaling=scaling, factor=factor), amp, fa.FIB_ROPE_HALF, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout,R", [(fa.FIB_ROPE_HALF, 64), (fa.FIB_ROPE_INTERLEAVED, 24), (fa.FIB_ROPE_HALF, 20)])
def test_strides_in_place_and_broadcast(dtype, layout, R):
    B, Hq, Hk, N = 3, 4, 2, 37
    rope = fa.fib_attn_rope_create(2000, rot_dim=R, layout=layout)
    theta = fa.fib_attn_rope_frequencies(R)
    start = torch.tensor([1000, 0, 1900], dtype=torch.int32, device="cuda")
    pos = start.cpu().numpy()[:, None] + np.arange(N)
    base = rand((B, N, Hq + 2 * Hk, 64), dtype, 4)
    before = base.clone()
    q, k = base[:, :, :Hq].transpose(1, 2), base[:, :, Hq:Hq + Hk].transpose(1, 2)
    q0, k0 = q.clone(), k.clone()
    qo, ko = fa.fib_attn_rotary(rope, q, k, start=start)
    assert qo.is_contiguous() and ko.is_contiguous() and torch.equal(base, before)
    check(qo, q0, pos, theta, 1.0, layout, dtype)
    check(ko, k0, pos, theta, 1.0, layout, dtype)
    fa.fib_attn_rotary(rope, q, k, start=start, q_out=q, k_out=k)  # in place, the values' part stays
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(base[:, :, Hq + Hk:], before[:, :, Hq + Hk:])
    # one query for every head and sequence; rows at an odd place in memory
    one = rand((1, 1, N, 64), dtype, 5).expand(B, Hq, N, 64)
    check(fa.fib_attn_rotary(rope, one, start=start)[0], one, pos, theta, 1.0, layout, dtype)
    odd = rand((B * Hq * N * 65 + 1,), dtype, 6)[1:].view(B, Hq, N, 65)[..., :64]
    check(fa.fib_attn_rotary(rope, odd, start=start)[0], odd, pos, theta, 1.0, layout, dtype)
    assert fa.fib_attn_rope_status(rope) == fa.FIB_OK


def test_rows_beyond_32_bits():
    """The last row of a view starts behind 2^32 bytes and 2^31 elements."""
    N, stride = 3, 1 << 30
    x = torch.empty(2 * stride + 64, dtype=torch.bfloat16, device="cuda")
    v = x.as_strided((1, 1, N, 64), (0, 0, stride, 1))
    v.copy_(rand((1, 1, N, 64), "bf16", 7))
    rope = fa.fib_attn_rope_create(4)
    check(fa.fib_attn_rotary(rope, v)[0], v, np.arange(N)[None], fa.fib_attn_rope_frequencies(64), 1.0, fa.FIB_ROPE_HALF, "bf16")


def test_infinite_and_nan_values_stay_in_their_pair():
    rope = fa.fib_attn_rope_create(8, rot_dim=16, layout=fa.FIB_ROPE_INTERLEAVED)
    q = rand((1, 1, 8, 64), "f32", 8)
    q[0, 0, 3, 5], q[0, 0, 4, 40], q[0, 0, 5, 63] = math.nan, math.inf, math.nan
    got = fa.fib_attn_rotary(rope, q)[0][0, 0].cpu().numpy()
    bad = ~np.isfinite(got)
    want = np.zeros_like(bad)
    want[3, 4:6] = want[4, 40] = want[5, 63] = True
    assert (bad == want).all() and got[4, 40] == math.inf


def test_bad_positions_are_reported_and_left():
    rope = fa.fib_attn_rope_create(100)
    q = rand((2, 2, 3, 64), "f32", 9)
    out = torch.full_like(q, 7.0)
    pos = torch.tensor([[0, 100, 99], [-1, 5, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    fa.fib_attn_rotary(rope, q, pos=pos, q_out=out)
    assert fa.fib_attn_rope_status(rope) == fa.FIB_ERR_DEVICE_ASSERT and fa.fib_attn_rope_status(rope) == fa.FIB_OK
    left = torch.tensor([[False, True, False], [True, False, True]], device="cuda")[:, None, :, None].expand_as(q)
    assert (out[left] == 7.0).all() and (out[~left] != 7.0).all()
    fa.fib_attn_rotary(rope, q, start=torch.tensor([2 ** 31 - 1, 0], dtype=torch.int32, device="cuda"), q_out=out)
    assert fa.fib_attn_rope_status(rope) == fa.FIB_ERR_DEVICE_ASSERT
    fa.fib_attn_rotary(rope, q, q_out=out)
    assert fa.fib_attn_rope_status(rope) == fa.FIB_OK


def test_refusals():
    rope = fa.fib_attn_rope_create(100)
    q = rand((2, 2, 3, 64), "f32", 10)
    i32 = dict(dtype=torch.int32, device="cuda")
    for kw in (dict(q=q.half()), dict(q=q.cpu()), dict(q=q[..., :32]), dict(q=q.transpose(2, 3)), dict(q=q[0]), dict(k=q[:1]), dict(k=q[:, :, :2]),
               dict(k=q.bfloat16()), dict(pos=torch.zeros(3, **i32)), dict(pos=torch.zeros(2, 3, device="cuda")), dict(start=torch.zeros(3, **i32)),
               dict(q_out=q[:, :1]), dict(q_out=q.bfloat16()), dict(k_out=q)):
        with pytest.raises(ValueError):
            fa.fib_attn_rotary(rope, **{**dict(q=q), **kw})
    buffer = rand((2, 2, 4, 64), "f32", 11)
    for kw in (dict(pos=torch.zeros(2, 3, **i32), start=torch.zeros(2, **i32)), dict(q_out=torch.empty(1, 1, 1, 64, device="cuda").expand(2, 2, 3, 64)),
               dict(q=buffer[:, :, :3], q_out=buffer[:, :, 1:]), dict(k=q.clone(), q_out=(x := q.clone()), k_out=x), dict(q=q[:, :, :0])):
        with pytest.raises(fa.FibAttnError) as e:
            fa.fib_attn_rotary(rope, **{**dict(q=q), **kw})
        assert e.value.code == fa.FIB_ERR_INVALID_ARG


def test_streams_and_graphs():
    rope = fa.fib_attn_rope_create(5000)
    q = rand((2, 4, 50, 64), "bf16", 12)
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = fa.fib_attn_rotary(rope, q, start=start, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(on_side, fa.fib_attn_rotary(rope, q, start=start)[0])
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
    with torch.cuda.graph(graph):
        fa.fib_attn_rotary(rope, q, start=start, q_out=out)
    for at in (0, 17, 4950):
        start.fill_(at)  # read on the device, at the replay
        graph.replay()
        check(out, q, at + np.tile(np.arange(50), (2, 1)), fa.fib_attn_rope_frequencies(64), 1.0, fa.FIB_ROPE_HALF, "bf16")


@pytest.mark.parametrize("layout,R", [(fa.FIB_ROPE_HALF, 64), (fa.FIB_ROPE_INTERLEAVED, 12)])
def test_gradients(layout, R):
    """Against the formula's (the map is linear: its transpose) and against differences."""
    B, Hq, Hk, N = 2, 3, 1, 9
    rope = fa.fib_attn_rope_create(64, rot_dim=R, layout=layout, amplitude=1.25)
    start = torch.tensor([3, 40], dtype=torch.int32, device="cuda")
    x = rand((B, N, Hq + Hk, 64), "f32", 13).requires_grad_()
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:].transpose(1, 2)
    gq, gk = rand((B, Hq, N, 64), "f32", 14), rand((B, Hk, N, 64), "f32", 15)
    yq, yk = rotary(rope, q, k, start=start)
    (yq * gq).sum().add((yk * gk).sum()).backward()
    pos = start.cpu().numpy()[:, None] + np.arange(N)
    theta = fa.fib_attn_rope_frequencies(R)
    check(x.grad[:, :, :Hq].transpose(1, 2), gq, pos, theta, 1.25, layout, "f32", transpose=True)
    check(x.grad[:, :, Hq:].transpose(1, 2), gk, pos, theta, 1.25, layout, "f32", transpose=True)
    # a step of 1 in one element: the map is linear, so the difference is the derivative but for its float32 roundings
    for at in ((0, 2, 1, 5), (1, 8, 3, R - 1), (1, 0, 0, 63)):
        with torch.no_grad():
            moved = x.detach().clone()
            moved[at] += 1
            loss = [sum((y.double() * g.double()).sum() for y, g in zip(fa.fib_attn_rotary(rope, v[:, :, :Hq].transpose(1, 2), v[:, :, Hq:].transpose(1, 2),
                                                                                                 start=start), (gq, gk))) for v in (x.detach(), moved)]
        assert abs(float(loss[1] - loss[0]) - float(x.grad[at])) <= 1e-4
    # one output's gradient alone, an expanded one, and shared keys
    k1 = rand((1, 1, N, 64), "f32", 16).requires_grad_()
    _, yk = rotary(rope, q.detach(), k1.expand(B, Hk, N, 64), start=start)
    yk.sum().backward()
    want = sum(reference(np.ones((1, 1, N, 64)), pos[b:b + 1].astype(float), theta, 1.25, layout, True)[0] for b in range(B))
    assert np.abs(k1.grad.double().cpu().numpy() - want).max() <= 2 * 12 * 2.0 ** -24 * 2.5 + 2.0 ** -22  # two terms of |a| + |b| = 2.5, and their sum


def test_no_second_derivatives():
    rope = fa.fib_attn_rope_create(64)
    q = rand((1, 2, 16, 64), "f32", 18).requires_grad_()
    g, = torch.autograd.grad(rotary(rope, q)[0].square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        g.square().sum().backward()


def test_backward_under_capture_with_an_eager_graph_alive():
    """Of the same memory; the leaf is one of the capture's own, as torch ties a leaf to the stream of its living graphs."""
    rope = fa.fib_attn_rope_create(64)
    q = rand((1, 2, 16, 64), "f32", 17).requires_grad_()
    kept = rotary(rope, q)[0].sum()  # an eager graph
    x = q.detach().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(rotary(rope, x)[0].square().sum(), x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g, = torch.autograd.grad(rotary(rope, x)[0].square().sum(), x)
    graph.replay()
    torch.cuda.synchronize()
    # R is orthogonal: the gradient of |R q|^2 is 2 q
    assert (g - 2 * q).abs().max() <= 2 * 2 * 24 * 2.0 ** -24 * 2 * float(q.detach().abs().max())
    kept.backward()


@pytest.mark.parametrize("dtype,tol", [("f32", 1e-5), ("bf16", 1e-2)])
@pytest.mark.parametrize("mode", ["mask", "interp"])
def test_attention_of_a_plan_that_does_not_rotate(dtype, tol, mode):
    """Rows rotated here by another layout and a part of the head, attended by a plan that leaves them: the oracle, which rotates, is
    given the rows turned back in binary64."""
    B, H, N, W, alpha = 1, 2, 200, 8, 1.2345
    plan = fa.fib_attn_plan_create(fa.FIB_BASE_FIBONACCI, [alpha], W, N, fa.FIB_MODE_MASK if mode == "mask" else fa.FIB_MODE_INTERP)
    x = [rand((B, H, N, 64), dtype, 18 + i) for i in range(4)]
    with_own = fa.fib_attn_fwd(plan, 0, *x[:3])
    fa.fib_attn_plan_set_rotation(plan, False)
    rope = fa.fib_attn_rope_create(N, rot_dim=32, layout=fa.FIB_ROPE_INTERLEAVED)
    q, k = fa.fib_attn_rotary(rope, x[0], x[1])
    o, lse = fa.fib_attn_fwd(plan, 0, q, k, x[2])
    back = lambda t: turn(t.double().cpu().numpy(), -np.arange(N))  # noqa: E731
    ref = back(q), back(k), x[2].double().cpu().numpy()
    O_ref, lse_ref = oracle.attend(*ref, alpha, oracle.fibonacci_base(), W, mode)
    lse_tol = 1e-5 if dtype == "f32" else 5e-3
    assert (np.abs(o.double().cpu().numpy() - O_ref) - (2.0 ** -8 * np.abs(O_ref) if dtype == "bf16" else 0)).max() <= tol
    assert np.abs(lse.double().cpu().numpy() - lse_ref).max() <= lse_tol
    # gradients of the rotated rows: the oracle's, rotated to them
    dq, dk, dv, _ = fa.fib_attn_bwd(plan, 0, q, k, x[2], o, lse, x[3])
    rq, rk, rv, _ = oracle.attend_bwd(*ref, x[3].double().cpu().numpy(), alpha, oracle.fibonacci_base(), W, mode)
    for g, r in ((dq, turn(rq, np.arange(N))), (dk, turn(rk, np.arange(N))), (dv, rv)):
        assert np.linalg.norm(g.double().cpu().numpy() - r) <= (1e-5 if dtype == "f32" else 2e-2) * np.linalg.norm(r)
    # and as it was
    fa.fib_attn_plan_set_rotation(plan, True)
    again = fa.fib_attn_fwd(plan, 0, *x[:3])
    assert torch.equal(with_own[0], again[0]) and torch.equal(with_own[1], again[1])


def test_a_training_step_through_both():
    B, H, N = 2, 2, 64
    plan = fa.fib_attn_plan_create(fa.FIB_BASE_FIBONACCI, [1.1], 8, N, fa.FIB_MODE_INTERP)
    fa.fib_attn_plan_set_rotation(plan, False)
    rope = fa.fib_attn_rope_create(N)
    x = rand((B, N, 3 * H, 64), "f32", 30).requires_grad_()
    alpha = torch.tensor([1.1], device="cuda", requires_grad=True)
    q, k = rotary(rope, x[:, :, :H].transpose(1, 2), x[:, :, H:2 * H].transpose(1, 2))
    g = rand((B, H, N, 64), "f32", 31)
    (fib_attention(plan, 0, q, k, x[:, :, 2 * H:].transpose(1, 2).contiguous(), alpha) * g).sum().backward()
    # the same layer by a plan that rotates
    own = fa.fib_attn_plan_create(fa.FIB_BASE_FIBONACCI, [1.1], 8, N, fa.FIB_MODE_INTERP)
    y, a2 = x.detach().clone().requires_grad_(), alpha.detach().clone().requires_grad_()
    rows = [y[:, :, i * H:(i + 1) * H].transpose(1, 2).contiguous() for i in range(3)]
    (fib_attention(own, 0, *rows, a2) * g).sum().backward()
    # two float32 paths, each within 1e-5 (norm) of the same gradient
    assert float((x.grad - y.grad).norm()) <= 2e-5 * float(y.grad.norm())
    assert abs(float(alpha.grad - a2.grad)) <= 2e-4 * abs(float(a2.grad))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,Hq", [(1, 2), (5, 4), (12, 4)])
def test_decodes_of_a_plan_that_does_not_rotate(dtype, T, Hq):
    """Rows rotated by fib_attn_rotary at positions of their own (a cache that lost rows: 1000 behind), committed and decoded as they are, against
    the oracle, which is given rows and queries turned back to the positions that it turns them to."""
    from oracle import cache_oracle as co
    from tests.test_gpu_cache import TOL_LSE, TOL_O, HALF, draw as cache_draw, i32, rng
    r = rng(300, T, Hq)
    B, H, P, lens = 2, 2, 16, [45, 20]
    plan = fa.fib_attn_plan_create(fa.FIB_BASE_FIBONACCI, [1.0], 6, 100, fa.FIB_MODE_MASK)
    fa.fib_attn_plan_set_rotation(plan, False)
    rope = fa.fib_attn_rope_create(2000, rot_dim=32, layout=fa.FIB_ROPE_INTERLEAVED, scaling=fa.FIB_ROPE_NTK, factor=2.0)
    cache = fa.fib_attn_cache_create(1, H, P, 12, B, 6, DT[dtype])
    k, _ = cache_draw(r, (B, H, 45, 64), dtype)
    v, _ = cache_draw(r, (B, H, 45, 64), dtype)
    k = fa.fib_attn_rotary(rope, k, start=i32([1000, 1000]))[0]
    fa.fib_attn_cache_commit(plan, cache, k[None], v[None], i32(lens))
    assert torch.equal(cache.k[0, cache.table[0, 0].long()], k[0, :, :P])  # as they came
    q, _ = cache_draw(r, (B, Hq, T, 64), dtype)
    kn, _ = cache_draw(r, (B, H, T, 64), dtype)
    vn, vf = cache_draw(r, (B, H, T, 64), dtype)
    q, kn = fa.fib_attn_rotary(rope, q, kn, start=cache.lens + 1000)
    ref = co.PagedCache(cache.k.double().cpu().numpy(), cache.v.double().cpu().numpy(), cache.table.cpu().tolist(), cache.lens.cpu().tolist(),
                        cache.refs.cpu().tolist())
    pos = np.array(lens)[:, None] + np.arange(T)
    back = lambda x: turn(x.double().cpu().numpy(), -pos[:, None])  # noqa: E731
    parent = [[i - 1 for i in range(T)]] * B
    keys = [(x, 0.0) for x in range(6)] + [(x, 0.0) for x in fa.fib_attn_plan_distances(plan, 0, 100)]
    for kk, (o, lse) in ((None, fa.fib_attn_dense_tree_decode(plan, 0, cache, q, kn, vn)), (keys, fa.fib_attn_tree_decode(plan, 0, cache, q, kn, vn, N=100))):
        want, lse_want = co.tree_attend(ref, 0, back(q), back(kn), vf, parent, [T] * B, kk)
        assert np.abs(lse.double().cpu().numpy() - lse_want).max() <= TOL_LSE
        assert (np.abs(o.double().cpu().numpy() - want) - HALF[dtype] * np.abs(want)).max() <= TOL_O
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK and fa.fib_attn_rope_status(rope) == fa.FIB_OK


@pytest.mark.parametrize("B,Hq,Hk,N", [(1, 1, 1, 1), (2, 1, 3, 5), (3, 4, 1, 9), (2, 2, 2, 130), (1, 5, 2, 33)])
@pytest.mark.parametrize("order", ["qkv", "vqk", "kvq"])
@pytest.mark.parametrize("tokens_first", [True, False])
def test_parts_of_one_projection(B, Hq, Hk, N, order, tokens_first):
    """Queries and keys between one another's rows, in place and into another projection: they overlap in extent and not in memory."""
    rope = fa.fib_attn_rope_create(N)
    heads, at = {"q": Hq, "k": Hk, "v": Hk}, {}
    for x in order:
        at[x] = sum(heads[y] for y in order[:order.index(x)])
    shape = (B, N, Hq + 2 * Hk, 64) if tokens_first else (B, Hq + 2 * Hk, N, 64)
    part = lambda x, t: t.transpose(1, 2)[:, at[x]:at[x] + heads[x]] if tokens_first else t[:, at[x]:at[x] + heads[x]]  # noqa: E731
    base = rand(shape, "f32", 40)
    q, k = part("q", base), part("k", base)
    want = fa.fib_attn_rotary(rope, q, k)
    into = torch.full_like(base, 3.0)
    fa.fib_attn_rotary(rope, q, k, q_out=part("q", into), k_out=part("k", into))
    assert torch.equal(part("q", into), want[0]) and torch.equal(part("k", into), want[1]) and (part("v", into) == 3.0).all()
    values = part("v", base).clone()
    fa.fib_attn_rotary(rope, q, k, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(part("v", base), values)
    assert fa.fib_attn_rope_status(rope) == fa.FIB_OK
