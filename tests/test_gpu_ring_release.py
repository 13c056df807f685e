"""The bf16 forward and the dense control while other blocks of the same call write the status word at once, which holds up
the loads of the blocks beside them (needs a GPU): the same bits as without, every time."""
import os

import pytest
import torch

from fibonacci_offset_sparse_gb300 import fib_attn as fa
from fibonacci_offset_sparse_gb300 import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from fibonacci_offset_sparse_gb300 import build as b
    if not os.path.exists(b.LIB):
        b.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return fa.lib()


@pytest.mark.parametrize("kind", ["mask", "interp", "dense"])
@pytest.mark.parametrize("N", [333, 2048])
def test_the_same_bits_beside_queries_out_of_range(kind, N):
    B, H = 2, 24
    q, k, v = (t.cuda() for t in inputs.qkv(B, H, N, 64, 940, 0, "bf16"))
    plan = fa.fib_attn_plan_create(fa.FIB_BASE_FIBONACCI, [1.17], 12, N, fa.FIB_MODE_INTERP if kind == "interp" else fa.FIB_MODE_MASK)

    def call(x):
        return fa.fib_attn_dense_fwd(plan, x, k, v) if kind == "dense" else fa.fib_attn_fwd(plan, 0, x, k, v)

    want = [x.clone() for x in call(q)]
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_OK
    far = q.clone()
    far[:, ::3] = 1e30  # a third of the heads: beyond the float16 range
    keep = [h for h in range(H) if h % 3]
    for _ in range(60):
        got = call(far)
        assert all(torch.equal(x[:, keep], y[:, keep]) for x, y in zip(got, want))
    assert fa.fib_attn_last_device_status(plan) == fa.FIB_ERR_RANGE
    plan.close()
