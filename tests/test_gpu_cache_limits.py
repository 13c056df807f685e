"""The paged cache and the tree decodes at their limits: waits that run out, several host threads, one workspace for every
size, long contexts, large tables (needs a GPU).  Tolerances as in test_gpu_cache.py, unless a test derives its own."""
import os

import numpy as np
import pytest
import torch

from fibonacci_offset_sparse_gb300 import fib_attn as fa
from oracle import cache_oracle as co

from .test_gpu_cache import check, i32, plan_for, rng, tree_case

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
