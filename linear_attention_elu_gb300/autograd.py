"""PyTorch autograd wrappers: the library's forward and backward entry points
as one differentiable function (argument marshalling only; both directions
run in the library's kernels).

    o = linear_attention(q, k, v, causal=True)     # q, k: [B,H,N,Dk], v: [B,H,N,Dv]
    o.backward(g)                                   # la_causal_bwd fills q.grad, k.grad, v.grad
    qo, ko = qk_norm_rope(q, k, pos, table, wq, wk) # q: [B,N,Hq,D], k: [B,N,Hk,D], head-major out
    o = decay_attention(q, k, v, decay)             # q, k: [B,H,N,Dk], v: [B,H,N,Dv], decay: [H]
    y = group_norm(o_rows, H, w, b, z)              # o_rows: [B N,1,H D], z: the gate

Either of q and k of qk_norm_rope may be None. A training step captured into a CUDA
graph calls the library's backward entries (la_*_bwd) itself.

The attention backward takes Dk, Dv <= 64 (the library refuses wider heads with
LA_ERR_UNSUPPORTED). Gradients have the inputs' dtype.
"""
import torch
from torch.autograd.function import once_differentiable

from . import (LA_PHI_ELU1, la_causal_bwd, la_causal_fwd, la_decay_attn_bwd, la_decay_attn_fwd,
               la_group_norm_bwd, la_group_norm_fwd, la_noncausal_bwd, la_noncausal_fwd,
               la_qk_norm_rope_bwd, la_qk_norm_rope_fwd)


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


def _adjacent(t):
    """t itself where a row's values are adjacent, else a copy (a gradient may come expanded)."""
    return t if t.shape[-1] <= 1 or t.stride(-1) == 1 else t.contiguous()


def _whole_pieces(t):
    """A gradient in rows of whole 16-byte pieces: t itself, or a copy where only its strides or its
    place in memory stand against that (behind a torch.cat, say). Without them the tensor-core kernels
    of the decayed attention and the wide groups of the norm, which the forward pass had, are closed to it."""
    e = t.element_size()
    if t.shape[-1] * e % 16 or t.numel() == 0:
        return _adjacent(t)
    rows = zip(t.shape[:-1], t.stride()[:-1])
    if t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(n == 1 or s * e % 16 == 0 for n, s in rows):
        return t
    return t.clone(memory_format=torch.contiguous_format)


class _DecayAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, decay, scale, lengths, token_major):
        o = None
        if token_major:
            B, H, N, Dv = v.shape
            make = torch.empty if lengths is None else torch.zeros
            o = make((B, N, H, Dv), dtype=v.dtype, device=v.device).transpose(1, 2)
        o = la_decay_attn_fwd(q, k, v, decay, scale, lengths, o=o)
        ctx.save_for_backward(q, k, v, decay, lengths)
        ctx.scale = scale
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, decay, lengths = ctx.saved_tensors
        do = _whole_pieces(do.to(v.dtype))
        if do.stride(2) == 0:                   # one row for all tokens (a sum over them): rows of their own
            do = do.contiguous()
        dq, dk, dv = la_decay_attn_bwd(q, k, v, do, decay, ctx.scale, lengths)
        return dq, dk, dv, None, None, None, None


def decay_attention(q, k, v, decay, scale=1.0, lengths=None, token_major=False):
    """Differentiable la_decay_attn_fwd from a state of zero (the decay is a constant).

    token_major: the outputs lie as [B,N,H,Dv] in memory (the rows that the group norm and a
    projection take); their shape is [B,H,N,Dv] either way."""
    if decay.requires_grad:
        raise ValueError("the decay is a constant: no gradient with respect to it")
    q, k, v = (_adjacent(t) for t in (q, k, v))
    return _DecayAttention.apply(q, k, v, decay, float(scale), lengths, bool(token_major))


class _GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, groups, w, b, z, silu, eps):
        y, stats = la_group_norm_fwd(x, groups, w, b, z, silu, eps, return_stats=True)
        ctx.save_for_backward(x, w, b, z, stats)
        ctx.groups, ctx.silu = groups, silu
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, b, z, stats = ctx.saved_tensors
        dx, dw, db, dz = la_group_norm_bwd(x, ctx.groups, _whole_pieces(dy.to(x.dtype)), stats, w, b, z, ctx.silu)
        return (dx, None, dw.to(w.dtype) if dw is not None else None, db.to(b.dtype) if db is not None else None,
                dz, None, None)


def group_norm(x, groups, w=None, b=None, z=None, silu=False, eps=1e-5):
    """Differentiable la_group_norm_fwd: y = act(w xh + b) silu(z) of channels-last rows x [B,N,C]."""
    x, z = _adjacent(x), None if z is None else _adjacent(z)
    return _GroupNorm.apply(x, int(groups), w, b, z, bool(silu), float(eps))
