"""Rotary positions, what needs no GPU: frequencies against their formulas, refusals."""
import ctypes
import math

import pytest

from fibonacci_offset_sparse_gb300 import fib_attn as fa


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    from fibonacci_offset_sparse_gb300 import build as b
    srcs = [os.path.join(b.CSRC, s) for s in os.listdir(b.CSRC)]
    if not os.path.exists(b.LIB) or os.path.getmtime(b.LIB) < max(os.path.getmtime(s) for s in srcs):
        b.build()
    return fa.lib()


def formula(R, base, scaling, factor, n_train, slow, fast):
    out = []
    for m in range(R // 2):
        t = base ** (-2 * m / R)
        if scaling == fa.FIB_ROPE_LINEAR:
            t /= factor
        if scaling == fa.FIB_ROPE_NTK and R > 2:
            t = base ** (-2 * m / R) * factor ** (-2 * m / (R - 2))
        if scaling == fa.FIB_ROPE_YARN:
            g = min(1.0, max(0.0, (n_train * t / (2 * math.pi) - slow) / (fast - slow)))
            t = g * t + (1 - g) * t / factor
        out.append(t)
    return out


@pytest.mark.parametrize("R", [2, 6, 20, 32, 64])
@pytest.mark.parametrize("scaling", [fa.FIB_ROPE_PLAIN, fa.FIB_ROPE_LINEAR, fa.FIB_ROPE_NTK, fa.FIB_ROPE_YARN])
@pytest.mark.parametrize("base,factor,n_train,slow,fast", [(10000.0, 4.0, 1024, 1.0, 32.0), (500000.0, 1.0, 1, 0.0, 0.5), (1.5, 37.5, 8192, 2.0, 2.5)])
def test_frequencies(R, scaling, base, factor, n_train, slow, fast):
    got = fa.fib_attn_rope_frequencies(R, fa.FIB_ROPE_HALF, base, scaling, factor, n_train, slow, fast)
    want = formula(R, base, scaling, factor, n_train, slow, fast)
    assert len(got) == R // 2
    for g, w in zip(got, want):
        assert abs(g - w) <= 1e-13 * w  # a few binary64 powers and products


def test_scaling_by_one_is_plain():
    plain = fa.fib_attn_rope_frequencies(64)
    for scaling in (fa.FIB_ROPE_LINEAR, fa.FIB_ROPE_NTK, fa.FIB_ROPE_YARN):
        assert fa.fib_attn_rope_frequencies(64, scaling=scaling) == pytest.approx(plain, rel=1e-14)


BAD = [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=66), dict(rot_dim=-2), dict(layout=2), dict(layout=-1), dict(scaling=4), dict(scaling=-1),
       dict(base=1.0), dict(base=math.inf), dict(base=math.nan), dict(base=-2.0), dict(scaling=fa.FIB_ROPE_LINEAR, factor=0.5),
       dict(scaling=fa.FIB_ROPE_NTK, factor=math.nan), dict(scaling=fa.FIB_ROPE_YARN, factor=math.inf), dict(scaling=fa.FIB_ROPE_YARN, n_train=0),
       dict(scaling=fa.FIB_ROPE_YARN, slow=-1.0), dict(scaling=fa.FIB_ROPE_YARN, slow=32.0), dict(scaling=fa.FIB_ROPE_YARN, fast=math.inf)]


@pytest.mark.parametrize("kw", BAD, ids=[str(x) for x in BAD])
def test_spec_rules(kw):
    with pytest.raises(fa.FibAttnError) as e:
        fa.fib_attn_rope_frequencies(**kw)
    assert e.value.code == fa.FIB_ERR_INVALID_ARG


def test_create_and_null_arguments(lib):
    spec = fa.RopeSpec(0, 64, 0, 0, 10000.0, 1.0, 0.0, 0.0, 1.0)
    h, x = ctypes.c_void_p(), (ctypes.c_double * 32)()
    assert lib.fib_attn_rope_frequencies(None, x) == fa.FIB_ERR_INVALID_ARG
    assert lib.fib_attn_rope_frequencies(ctypes.byref(spec), None) == fa.FIB_ERR_INVALID_ARG
    assert lib.fib_attn_rope_create(None, ctypes.byref(spec), 16) == fa.FIB_ERR_INVALID_ARG
    assert lib.fib_attn_rope_create(ctypes.byref(h), None, 16) == fa.FIB_ERR_INVALID_ARG
    for n in (0, -1, (1 << 20) + 1):
        assert lib.fib_attn_rope_create(ctypes.byref(h), ctypes.byref(spec), n) == fa.FIB_ERR_INVALID_ARG
    for a in (0.0, -1.0, math.nan, math.inf):
        assert lib.fib_attn_rope_create(ctypes.byref(h), ctypes.byref(fa.RopeSpec(0, 64, 0, 0, 10000.0, 1.0, 0.0, 0.0, a)), 16) == fa.FIB_ERR_INVALID_ARG
    assert not h.value
    s = (ctypes.c_int64 * 3)(64, 64, 64)
    assert lib.fib_attn_rotary(None, 0, 1, 1, 1, 0, 64, s, 1 << 20, s, None, None, None, None, None, None, 0, None) == fa.FIB_ERR_INVALID_ARG
    assert lib.fib_attn_rope_status(None) == fa.FIB_ERR_INVALID_ARG
    assert lib.fib_attn_rope_destroy(None) == fa.FIB_OK
    assert lib.fib_attn_plan_set_rotation(None, 0) == fa.FIB_ERR_INVALID_ARG


@pytest.mark.parametrize("amplitude", [1e39, 1e-60, math.inf, math.nan])
def test_an_amplitude_is_a_float32(amplitude):
    spec = fa.RopeSpec(fa.FIB_ROPE_HALF, 64, fa.FIB_ROPE_PLAIN, 1024, 10000.0, 1.0, 1.0, 32.0, amplitude)
    out = (ctypes.c_double * 32)()
    assert fa.lib().fib_attn_rope_frequencies(ctypes.byref(spec), out) == fa.FIB_ERR_INVALID_ARG


FAR = 1 << 39  # elements; times 2^25 it is 2^64


@pytest.mark.parametrize("dtype", [fa.FIB_DTYPE_F32, fa.FIB_DTYPE_BF16])
@pytest.mark.parametrize("shape,strides", [
    ((1, 1, (1 << 25) + 1), (64, 64, FAR)),              # the product alone leaves 64 bits, and the extent comes out as one row
    (((1 << 25) + 1, 1, 1), (FAR, 64, 64)),
    ((1, 1, (1 << 24) + 1), (64, 64, FAR)),              # 2^63
    ((1 << 15, 1 << 10, 1 << 10), (FAR, FAR, FAR)),      # a sum of three
    ((1, 1, (1 << 19) + 1), (64, 64, FAR)),              # 2^58: the first that is too far
])
@pytest.mark.parametrize("far", ["in", "out", "k in", "k out"])
def test_strides_that_leave_64_bits(lib, dtype, shape, strides, far):
    B, H, N = shape
    near, wide = (ctypes.c_int64 * 3)(64 * H * N, 64 * N, 64), (ctypes.c_int64 * 3)(*strides)
    rows = [1 << 20, near, 1 << 44, near, 1 << 45, near, 1 << 46, near]  # memory that no call here reaches: q, q_out, k, k_out
    rows[1 + 2 * ["in", "out", "k in", "k out"].index(far)] = wide
    rope = 1 << 12  # never looked into: the call is refused for its strides
    assert lib.fib_attn_rotary(rope, dtype, B, N, H, H, *rows, None, None, 0, None) == fa.FIB_ERR_INVALID_ARG


def _rows(B, H, N, layout):
    """Strides (b, h, n) of [B, H, N, 64], of [B, N, H, 64], or of H heads of a projection of 8."""
    return {"rows": (H * N * 64, N * 64, 64), "tokens": (N * H * 64, 64, H * 64), "part": (N * 8 * 64, 64, 8 * 64)}[layout]


MEET = [  # the second tensor begins so many elements behind the first; queries and keys with their heads
    ("rows", 3, 3, 64), ("rows", 3, 3, 1), ("rows", 3, 2, 5 * 64), ("rows", 3, 1, -63), ("rows", 2, 4, 2 * 2 * 5 * 64 - 64),
    ("tokens", 3, 3, 3 * 64), ("tokens", 4, 2, 128), ("tokens", 1, 1, 64 * 9),
    ("part", 5, 2, 4 * 64), ("part", 2, 5, -4 * 64), ("part", 3, 3, 8 * 64), ("part", 3, 3, 8 * 64 * 4 + 2 * 64), ("part", 1, 1, 63), ("part", 1, 1, 8 * 64 * 5),
]


@pytest.mark.parametrize("dtype", [fa.FIB_DTYPE_F32, fa.FIB_DTYPE_BF16])
@pytest.mark.parametrize("layout,Hq,Hk,behind", MEET)
@pytest.mark.parametrize("which", ["q_out on k", "k_out on q", "both outputs"])
def test_outputs_that_overlap_the_other_tensors(lib, dtype, layout, Hq, Hk, behind, which):
    B, N, es = 2, 5, 4 if dtype == fa.FIB_DTYPE_F32 else 2
    first, strides = 1 << 30, [(ctypes.c_int64 * 3)(*_rows(B, H, N, layout)) for H in (Hq, Hk)]
    at = {"q": 1 << 40, "q_out": 1 << 41, "k": 1 << 42, "k_out": 1 << 43}  # memory that no call here reaches
    for name, place in zip({"q_out on k": ("q_out", "k"), "k_out on q": ("q", "k_out"), "both outputs": ("q_out", "k_out")}[which], (first, first + behind * es)):
        at[name] = place
    rope = 1 << 12  # never looked into
    assert lib.fib_attn_rotary(rope, dtype, B, N, Hq, Hk, at["q"], strides[0], at["q_out"], strides[0], at["k"], strides[1], at["k_out"], strides[1],
                               None, None, 0, None) == fa.FIB_ERR_INVALID_ARG
