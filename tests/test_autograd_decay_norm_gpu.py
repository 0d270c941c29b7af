"""The differentiable decayed attention and group norm, and the two together behind the
rotation as a layer uses them."""
import numpy as np
import pytest
import torch

from oracle import token_mixing as tm
from test_decay_attn_gpu import limits, near
from test_decay_attn_gpu import problem as attn_problem
from workloads import to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("token_major", [False, True])
def test_decay_attention_gradients(la, token_major, dt):
    from linear_attention_elu_gb300.autograd import decay_attention
    (q, k, v, do), decay, _ = attn_problem(2, 3, 150, 64, 64, dt, 5)
    x = [t.clone().requires_grad_() for t in (q, k, v)]
    o = decay_attention(*x, decay, 0.125, token_major=token_major)
    assert o.transpose(1, 2).is_contiguous() == token_major
    o.backward(do)
    a = [to_f64(t) for t in (q, k, v, do)]
    ref = tm.decay_attn_bwd(*a, to_f64(decay), 0.125)
    mag = tm.decay_attn_bwd(*map(np.abs, a), to_f64(decay), 0.125)
    for t, r, m in zip(x, ref, mag):
        near(t.grad, r, limits(150, 64, dt, r, m), "gradient")


def test_shared_keys_sum_over_heads_and_expanded_gradients(la):
    from linear_attention_elu_gb300.autograd import decay_attention
    (q, k, v, _), decay, _ = attn_problem(2, 4, 70, 64, 64, "f32", 6)
    q, k, v = q.clone().requires_grad_(), k[:, :1].clone().requires_grad_(), v[:, :1].clone().requires_grad_()
    decay_attention(q, k.expand(-1, 4, -1, -1), v.expand(-1, 4, -1, -1), decay).sum().backward()
    wide = [to_f64(q), np.repeat(to_f64(k), 4, 1), np.repeat(to_f64(v), 4, 1), np.ones((2, 4, 70, 64))]
    dq, dk, dv = tm.decay_attn_bwd(*wide, to_f64(decay))
    mq, mk, mv = tm.decay_attn_bwd(*map(np.abs, wide), to_f64(decay))
    near(q.grad, dq, limits(70, 64, "f32", dq, mq), "dq")
    for t, r, m in ((k, dk, mk), (v, dv, mv)):
        near(t.grad, r.sum(1, keepdims=True), limits(70, 64, "f32", r, m).sum(1, keepdims=True), "shared")


def test_a_decay_that_wants_a_gradient_is_refused(la):
    from linear_attention_elu_gb300.autograd import decay_attention
    q = torch.zeros(1, 2, 4, 64, device="cuda")
    with pytest.raises(ValueError):
        decay_attention(q, q, q, (-torch.ones(2, device="cuda")).requires_grad_())


@pytest.mark.parametrize("form", ["scripted", "differences"])
def test_rotation_attention_norm_and_gate_together(la, form):
    """One layer's mixing: rotation, decayed attention, per-head norm with a gate."""
    from linear_attention_elu_gb300.autograd import decay_attention, group_norm, qk_norm_rope
    B, N, H, D = 2, 70, 3, 32
    g = torch.Generator().manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    proj, w, b, dy = r(B, N, 4 * H * D), 1 + 0.2 * r(H * D), 0.1 * r(H * D), r(B, N, H * D)
    decay, freq = -torch.exp2(-4 * torch.rand(H, generator=g)), [100.0 ** (-i / 16) for i in range(16)]
    pos = torch.arange(N, dtype=torch.int32).expand(B, N).contiguous()

    def layer(p, w, b):
        q, k, v, z = p.unflatten(2, (4, H * D)).unbind(2)
        qo, ko = qk_norm_rope(q.unflatten(2, (H, D)), k.unflatten(2, (H, D)), pos.cuda(),
                              la.la_rope_table(freq), norm=False)
        o = decay_attention(qo, ko, v.unflatten(2, (H, D)).transpose(1, 2), decay.cuda(), D ** -0.5, token_major=True)
        rows = o.transpose(1, 2).reshape(B * N, 1, H * D)
        return group_norm(rows, H, w, b, z.reshape(B * N, 1, H * D)).view(B, N, H * D)

    def exact(p, w, b):
        q, k, v, z = np.split(p, 4, -1)
        cut = lambda t: t.reshape(B, N, H, D)  # noqa: E731
        qo, ko = (tm.norm_rope(cut(t), None, pos.numpy()[..., None], freq, [0] * 16, norm=False) for t in (q, k))
        o, _ = tm.decay_attn(qo, ko, cut(v).transpose(0, 2, 1, 3), decay.numpy().astype(np.float64), D ** -0.5)
        rows = o.transpose(0, 2, 1, 3).reshape(B * N, 1, H * D)
        return tm.group_norm(rows, H, w, b, z.reshape(B * N, 1, H * D))[0].reshape(B, N, H * D)

    x = [t.cuda().requires_grad_() for t in (proj, w, b)]
    y = layer(*x)
    ref = exact(*(to_f64(t) for t in (proj, w, b)))
    if form == "scripted":
        # fp32 throughout: a few hundred roundings of values of order one.
        assert np.abs(to_f64(y) - ref).max() <= 600 * 2.0 ** -24 * np.abs(ref).max()
        return
    # The gradient along a direction against the difference of the definition in 64 bits.
    (y * dy.cuda()).sum().backward()
    a = [to_f64(t) for t in (proj, w, b)]
    for i in range(3):
        d = np.random.default_rng(i).standard_normal(a[i].shape)
        loss = lambda s: (exact(*(t + s * d if j == i else t for j, t in enumerate(a))) * to_f64(dy)).sum()  # noqa: E731,B023
        diff, dot = (loss(1e-6) - loss(-1e-6)) / 2e-6, (to_f64(x[i].grad) * d).sum()
        size = np.linalg.norm(to_f64(x[i].grad)) * np.linalg.norm(d)
        assert abs(diff - dot) <= 1e-4 * size / np.sqrt(d.size) + 1e-5 * abs(diff)
