"""Attention and rotary positions as differentiable PyTorch ops.

attention: attn_fwd forward, attn_bwd backward.  rope: eio.rope both ways (the
gradient of a rotation is the rotation back, which keeps nothing but the positions).

The forward keeps only what "FlashAttention: memory-saving exact attention"
(section 4) says a backward needs: the output O and the row statistics (the
LSE); the backward recomputes P from Q, K and the LSE inside attn_bwd.

    o = attention(q, k, v, mask_kind=MASK_CAUSAL)       # q [B,N,Hq,d] bf16 CUDA
    o.float().sum().backward()                          # q.grad, k.grad, v.grad

The LSE is returned with return_lse=True but is not differentiable (no
gradient flows through it).  `fwd` and `bwd` replace the two library calls,
with the signatures of default_fwd / default_bwd below; tests use that to
check this wrapper's bookkeeping against the oracle on the CPU.
"""
from __future__ import annotations

import math

import numpy as np


def default_fwd(q, k, v, mask_kind, scale, block_map):
    from . import attn_fwd
    return attn_fwd(q, k, v, scale=scale, mask_kind=mask_kind, block_map=block_map)


def default_bwd(q, k, v, o, lse, dout, mask_kind, scale, block_map):
    from . import attn_bwd
    return attn_bwd(q, k, v, o, lse, dout, scale=scale, mask_kind=mask_kind, block_map=block_map)


def _function():
    import torch

    class _Attention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, mask_kind, scale, block_map, fwd, bwd):
            o, lse = fwd(q.contiguous(), k.contiguous(), v.contiguous(), mask_kind, scale, block_map)
            ctx.save_for_backward(q, k, v, o, lse)
            ctx.mask_kind, ctx.scale, ctx.block_map, ctx.bwd = mask_kind, scale, block_map, bwd
            ctx.mark_non_differentiable(lse)
            return o, lse

        @staticmethod
        def backward(ctx, dout, _dlse):
            q, k, v, o, lse = ctx.saved_tensors
            dq, dk, dv = ctx.bwd(q.contiguous(), k.contiguous(), v.contiguous(), o, lse, dout.contiguous(),
                                 ctx.mask_kind, ctx.scale, ctx.block_map)
            return dq, dk, dv, None, None, None, None, None

    return _Attention


_FN = None


def attention(q, k, v, mask_kind=0, scale=None, block_map=None, return_lse=False, fwd=None, bwd=None):
    """softmax(q k^T * scale + mask) v for q [B,Nq,Hq,d], k, v [B,Nkv,Hkv,d],
    differentiable in q, k and v.  mask_kind and block_map as for attn_fwd;
    scale defaults to 1/sqrt(d).  Returns o (and the LSE [B,Hq,Nq] if
    return_lse)."""
    global _FN
    if _FN is None:
        _FN = _function()
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    o, lse = _FN.apply(q, k, v, mask_kind, float(scale), block_map, fwd or default_fwd, bwd or default_bwd)
    return (o, lse) if return_lse else o


def default_rope(q, k, positions, axes, freq, interleaved, inverse):
    from . import rope as call
    return call(q, k, positions, axes, freq, interleaved=interleaved, inverse=inverse)


def _rows(x):
    """x, or a contiguous copy where its layout is not one that eio.rope reads (expanded
    gradients, transposed heads, strides or addresses that are not whole 16 bytes)."""
    import torch
    if x.is_contiguous():
        return x if x.data_ptr() % 16 == 0 else x.clone(memory_format=torch.contiguous_format)
    B, N, H, d = x.shape
    e = x.element_size()
    sb, sn, sh, sd = x.stride()
    ok = (sd == 1 and (H == 1 or sh == d) and (B == 1 or (sb > 0 and sb * e % 16 == 0))
          and (N == 1 or (sn > 0 and sn * e % 16 == 0)) and x.data_ptr() % 16 == 0)
    return x if ok else x.contiguous()


def _rope_function():
    import torch

    class _Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, positions, axes, freq, interleaved, inverse, call):
            ctx.set_materialize_grads(False)
            ctx.save_for_backward(positions)
            ctx.table = axes, freq, interleaved
            ctx.inverse, ctx.call = inverse, call
            yq, yk = call(_rows(q), None if k is None else _rows(k), positions, axes, freq, interleaved, inverse)
            return yq, yk

        @staticmethod
        def backward(ctx, dq, dk):
            positions, = ctx.saved_tensors
            if not ctx.needs_input_grad[0]:
                dq = None
            if not ctx.needs_input_grad[1]:
                dk = None

            def back(x, y):
                if torch.is_grad_enabled():  # a gradient of the gradient is wanted
                    return _Rope.apply(x, y, positions, *ctx.table, not ctx.inverse, ctx.call)
                return ctx.call(_rows(x), None if y is None else _rows(y), positions, *ctx.table, not ctx.inverse)

            if dq is None:  # only k's output was used, or only k's gradient is wanted
                gq, gk = None, (None if dk is None else back(dk, None)[0])
            else:
                gq, gk = back(dq, dk)
            return gq, gk, None, None, None, None, None, None

    return _Rope


_ROPE_FN = None


def rope(q, k, positions, axes, freq, interleaved=False, call=None):
    """eio.rope, differentiable in q and k (any number of times).  Returns (q, k) rotated.
    May be captured into a CUDA graph, backward included, with leaves of no other autograd graph that
    is still alive.  `call` replaces the library call, with the signature of default_rope."""
    global _ROPE_FN
    if _ROPE_FN is None:
        _ROPE_FN = _rope_function()
    from . import _axes
    axes, freq = np.array(_axes(axes)), np.array(freq, dtype=np.float64)  # the backward's own copy
    return _ROPE_FN.apply(q, k, positions, axes, freq, interleaved, False, call or default_rope)
