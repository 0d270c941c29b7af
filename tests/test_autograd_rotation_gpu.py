"""The rotation's gradients where no norm is taken, and those of a zero row."""
import numpy as np
import pytest
import torch

from oracle import token_mixing as tm
from test_qk_rope_gpu import TOL, close, problem
from workloads import to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("given", ["both", "q", "k"])
def test_rotation_alone_keeps_no_inputs(la, given, dt):
    # Without the norm the gradient is the turned-back output gradient: nothing of q and k
    # is needed, and nothing of them is kept.
    from linear_attention_elu_gb300.autograd import qk_norm_rope
    q, k, pos, f, ax, _, _, _ = problem(2, 9, 4, 2, 64, 32, 1, dt, 71)
    table = la.la_rope_table(f, ax)
    q = q.clone().requires_grad_() if given != "k" else None
    k = k.clone().requires_grad_() if given != "q" else None
    qo, ko = qk_norm_rope(q, k, pos.cuda(), table, norm=False)
    out = qo if qo is not None else ko
    assert not any(t is not None and t.is_floating_point() for t in out.grad_fn.saved_tensors)
    outs = [t for t in (qo, ko) if t is not None]
    gos = [torch.randn_like(t) for t in outs]
    torch.autograd.backward(outs, gos)
    for x, go in zip([t for t in (q, k) if t is not None], gos):
        ref, _ = tm.norm_rope_bwd(to_f64(x), None, to_f64(go), pos.numpy(), f, ax, False)
        close(x.grad, ref, TOL[dt])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_backward_entry_without_inputs(la, dt):
    q, k, pos, f, ax, _, _, _ = problem(2, 9, 4, 2, 64, 32, 1, dt, 72)
    table, pos = la.la_rope_table(f, ax), pos.cuda()
    dqo, dko = (torch.randn(2, h, 9, 64, device="cuda").to(q.dtype) for h in (4, 2))
    want = la.la_qk_norm_rope_bwd(q, k, dqo, dko, pos, table, norm=False)
    got = la.la_qk_norm_rope_bwd(None, None, dqo, dko, pos, table, norm=False)
    one = la.la_qk_norm_rope_bwd(None, None, None, dko, pos, table, norm=False)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert one[0] is None and torch.equal(one[1], want[1])
    with pytest.raises(ValueError):
        la.la_qk_norm_rope_bwd(None, None, dqo, dko, pos, table)      # the norm needs q and k


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gradient_of_a_zero_row(la, dt):
    # r = 1 / sqrt(eps) and x = 0: dx = r w g, and the row adds nothing to dw.
    q, k, pos, f, ax, wq, wk, _ = problem(1, 6, 2, 2, 64, 32, 1, dt, 73)
    q = q.clone()
    q[0, 1] = 0
    table = la.la_rope_table(f, ax)
    dqo, dko = (torch.randn(1, 2, 6, 64, device="cuda").to(q.dtype) for _ in range(2))
    dq, _, dwq, _ = la.la_qk_norm_rope_bwd(q, k, dqo, dko, pos.cuda(), table, wq, wk)
    torch.cuda.synchronize()
    rx, rw = tm.norm_rope_bwd(to_f64(q), to_f64(wq), to_f64(dqo), pos.numpy(), f, ax)
    close(dq[0, 1], rx[0, 1], 2 * TOL[dt])
    mag = np.abs(to_f64(q)) * np.abs(to_f64(dqo)).max(-1).transpose(0, 2, 1)[..., None] \
        / np.sqrt((to_f64(q) ** 2).mean(-1, keepdims=True) + 1e-6)
    assert (np.abs(to_f64(dwq) - rw) <= 2 * 160 * 2.0 ** -24 * mag.sum((0, 1, 2))).all()
