"""PyTorch autograd wrappers: the library's forward and backward entry points
as one differentiable function (argument marshalling only; both directions
run in the library's kernels).

    o = linear_attention(q, k, v, causal=True)     # q, k: [B,H,N,Dk], v: [B,H,N,Dv]
    o.backward(g)                                   # la_causal_bwd fills q.grad, k.grad, v.grad
    qo, ko = qk_norm_rope(q, k, pos, table, wq, wk) # q: [B,N,Hq,D], k: [B,N,Hk,D], head-major out

Either of q and k of qk_norm_rope may be None. A training step captured into a CUDA
graph calls the library's backward entries (la_*_bwd) itself.

The attention backward takes Dk, Dv <= 64 (the library refuses wider heads with
LA_ERR_UNSUPPORTED). Gradients have the inputs' dtype.
"""
import torch
from torch.autograd.function import once_differentiable

from . import (LA_PHI_ELU1, la_causal_bwd, la_causal_fwd, la_noncausal_bwd,
               la_noncausal_fwd, la_qk_norm_rope_bwd, la_qk_norm_rope_fwd)


class _LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal, eps, phi):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        fwd = la_causal_fwd if causal else la_noncausal_fwd
        o = fwd(q, k, v, eps=eps, phi=phi)
        ctx.save_for_backward(q, k, v)
        ctx.causal, ctx.eps, ctx.phi = causal, eps, phi
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v = ctx.saved_tensors
        bwd = la_causal_bwd if ctx.causal else la_noncausal_bwd
        dq, dk, dv = bwd(q, k, v, do.contiguous().to(v.dtype), eps=ctx.eps, phi=ctx.phi)
        return dq, dk, dv, None, None, None


def linear_attention(q, k, v, causal=True, eps=1e-6, phi=LA_PHI_ELU1):
    """Differentiable elu+1 linear attention (or another feature map via `phi`)."""
    return _LinearAttention.apply(q, k, v, bool(causal), float(eps), int(phi))


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, pos, table, wq, wk, norm, eps, interleaved):
        qo, ko = la_qk_norm_rope_fwd(q, k, pos, table, wq=wq, wk=wk, norm=norm, eps=eps,
                                     interleaved=interleaved)
        # Without the norm the gradient needs nothing of q and k.
        ctx.save_for_backward(*((q, k) if norm else (None, None)), pos, table, wq, wk)
        ctx.given = q is not None, k is not None
        ctx.how = dict(norm=norm, eps=eps, interleaved=interleaved)
        return qo, ko

    @staticmethod
    @once_differentiable
    def backward(ctx, dqo, dko):
        q, k, pos, table, wq, wk = ctx.saved_tensors
        # A side that was not given has no gradient (one whose output was not used gets zeros).
        dqo = dqo.contiguous() if ctx.given[0] else None
        dko = dko.contiguous() if ctx.given[1] else None
        dq, dk, dwq, dwk = la_qk_norm_rope_bwd(q, k, dqo, dko, pos, table, wq=wq, wk=wk, **ctx.how)
        return (dq, dk, None, None, dwq.to(wq.dtype) if wq is not None else None,
                dwk.to(wk.dtype) if wk is not None else None, None, None, None)


def qk_norm_rope(q, k, pos, table, wq=None, wk=None, norm=True, eps=1e-6, interleaved=False):
    """Differentiable la_qk_norm_rope_fwd: q [B,N,Hq,D], k [B,N,Hk,D] -> head-major (qo, ko)."""
    return _QkNormRope.apply(q, k, pos, table, wq, wk, bool(norm), float(eps), bool(interleaved))
