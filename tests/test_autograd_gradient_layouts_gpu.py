"""Gradients that reach the decayed attention and the group norm as views: parts of a joined tensor,
off a 16-byte boundary, expanded. Each gives the bits of the same gradient in a tensor of its own (the
kernels and their order of sums are the same), and no layout is refused that the forward pass took."""
import pytest
import torch

from test_decay_attn_gpu import problem as attn_problem
from test_group_norm_gpu import DT
from test_group_norm_gpu import problem as norm_problem

pytestmark = pytest.mark.gpu


def views(t):
    """t as views: behind 3 other columns, off a boundary, with the last two axes exchanged in memory."""
    e = torch.zeros(*t.shape[:-1], 3, dtype=t.dtype, device=t.device)
    flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.flatten()
    return [torch.cat([e, t], -1)[..., 3:], flat[1:].view(t.shape), t.transpose(-1, -2).contiguous().transpose(-1, -2)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N,C,G", [(1, 256, 1), (1, 1024, 2), (1, 99, 3), (1, 512, 8), (40, 64, 4)])
def test_group_norm(N, C, G, dt):
    from linear_attention_elu_gb300.autograd import group_norm
    p, dy = norm_problem(5, N, C, dt, 61)
    if N == 1 and C == 99:
        p["z"] = None

    def gradients(g):
        x = {n: None if t is None else t.clone().requires_grad_() for n, t in p.items()}
        group_norm(x["x"], G, x["w"], x["b"], x["z"], silu=True).backward(g)
        return [t.grad for t in x.values() if t is not None]

    want = gradients(dy)
    for v in views(dy):
        assert all(torch.equal(a, b) for a, b in zip(gradients(v), want))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 20])
def test_decay_attention(D, dt):
    from linear_attention_elu_gb300.autograd import decay_attention
    (q, k, v, do), decay, _ = attn_problem(2, 3, 200, D, D, dt, 67)

    def gradients(g):
        x = [t.clone().requires_grad_() for t in (q, k, v)]
        decay_attention(*x, decay, 0.125).backward(g)
        return [t.grad for t in x]

    want = gradients(do.contiguous())
    for g in views(do):
        assert all(torch.equal(a, b) for a, b in zip(gradients(g), want))
    # A sum over tokens, heads or sequences leaves one row for all of them.
    for axis in (0, 1, 2):
        one = do.narrow(axis, 0, 1).contiguous()
        g = one.expand(do.shape)
        assert g.stride(axis) == 0
        assert all(torch.equal(a, b) for a, b in zip(gradients(g), gradients(g.contiguous())))


def test_joined_outputs():
    # The gradient of a joined tensor's part, as autograd makes it.
    from linear_attention_elu_gb300.autograd import group_norm
    p, _ = norm_problem(6, 1, 256, "bf16", 71)
    e = torch.randn(6, 1, 3, device="cuda").to(DT["bf16"]).requires_grad_()
    x = p["x"].clone().requires_grad_()
    out = torch.cat([e, group_norm(x, 1, p["w"], p["b"], p["z"])], -1)
    w = torch.randn_like(out)
    (out * w).sum().backward()
    y = p["x"].clone().requires_grad_()
    group_norm(y, 1, p["w"], p["b"], p["z"]).backward(w[..., 3:].contiguous())
    assert torch.equal(x.grad, y.grad)
