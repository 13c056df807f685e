"""torch.autograd wrapper of one layer of the sparse attention (argument marshalling only).

``fib_attention(plan, layer, q, k, v, alpha)`` returns O; its backward calls the library's
backward, which returns dQ, dK, dV and, in INTERP mode, dl/dalpha of the layer ("Depth-
Staggered Fibonacci Spacing for Sparse Attention", Methodology > "Implementation": the
interpolated rows give alpha a gradient).  ``alpha`` is the per-layer alpha vector on the
device (float32, one entry per layer of the plan); its gradient is nonzero at ``layer`` only.
Every step runs in the CUDA library; nothing here computes attention.  Where the forward
prepares K'/V' rows (bf16, W <= 16), the Function keeps that workspace for the backward in
place of k and v (the same bytes) and the backward starts from it.
"""
import torch
from torch.autograd.function import once_differentiable

from . import fib_attn as fa


class _FibAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, alpha, plan, layer):
        B, H, N = q.shape[:3]
        need = fa.fib_attn_fwd_workspace_size(plan, B, H, N, q.dtype)
        ctx.plan, ctx.layer, ctx.prepared = plan, layer, need > 0
        if ctx.prepared:
            kv = torch.empty(need, dtype=torch.uint8, device=q.device)
            o, lse = fa.fib_attn_fwd(plan, layer, q, k, v, alpha_dev=alpha, workspace=kv)
            ctx.save_for_backward(q, kv, o, lse, alpha)
        else:
            o, lse = fa.fib_attn_fwd(plan, layer, q, k, v, alpha_dev=alpha)
            ctx.save_for_backward(q, k, v, o, lse, alpha)
        return o

    @staticmethod
    def backward(ctx, dO):
        if ctx.prepared:
            q, kv, o, lse, alpha = ctx.saved_tensors
            dq, dk, dv, da = fa.fib_attn_bwd_prepared(ctx.plan, ctx.layer, q, kv, o, lse, dO.contiguous(),
                                                      alpha_dev=alpha)
        else:
            q, k, v, o, lse, alpha = ctx.saved_tensors
            dq, dk, dv, da = fa.fib_attn_bwd(ctx.plan, ctx.layer, q, k, v, o, lse, dO.contiguous(),
                                             alpha_dev=alpha)
        dalpha = None
        if alpha is not None and ctx.needs_input_grad[3]:
            dalpha = torch.zeros_like(alpha)
            dalpha[ctx.layer] = da[0]
        return dq, dk, dv, dalpha, None, None


def fib_attention(plan, layer: int, q, k, v, alpha=None):
    """O of layer ``layer`` for q, k, v [B, H, N, 64] (contiguous CUDA, float32 or bfloat16);
    ``alpha``: device float32 [n_layers] (INTERP: used and differentiated) or None."""
    return _FibAttention.apply(q, k, v, alpha, plan, layer)


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, pos, start, rope):
        ctx.rope = rope
        ctx.save_for_backward(pos, start)
        return fa.fib_attn_rotary(rope, q, k, pos=pos, start=start)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        pos, start = ctx.saved_tensors
        # the map is linear, and its transpose the same kernel; gradients come in any strides
        grads = [g if g.stride(-1) == 1 else g.contiguous() for g, need in zip((dq, dk), ctx.needs_input_grad) if need]
        out = iter(fa.fib_attn_rotary(ctx.rope, *grads, pos=pos, start=start, transpose=True) if grads else ())
        return (*(next(out) if need else None for need in ctx.needs_input_grad[:2]), None, None, None)


def rotary(rope, q, k=None, pos=None, start=None):
    """(q, k) rotated by their positions (fib_attn_rotary): q [B, Hq, N, 64], k [B, Hk, N, 64] or None, in any strides, as views
    of a projection are; pos int32 [B, N], or start int32 [B] + n, or n.  For plans that do not rotate
    (fib_attn_plan_set_rotation).  The backward reads pos or start again (so not a cache's lens that a commit changes before it) and
    is not differentiable itself.  A backward that is captured into a graph needs leaves of which no eager graph lives, as
    any of torch does: x.detach().requires_grad_() is one."""
    return _Rotary.apply(q, k, pos, start, rope)
