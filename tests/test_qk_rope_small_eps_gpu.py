"""la_qk_norm_rope_bwd at eps = 0 against the float64 oracle (oracle/token_mixing.py).

The bounds of test_qk_rope_gpu.py: dx within twice 2.5e-6 (bf16: 2^-8 more) of the larger
of the row's gradient and its two terms, dw within 2 * 160 * 2^-24 of the sum of the
magnitudes of its terms."""
import numpy as np
import pytest
import torch

from oracle import token_mixing as tm
from test_qk_rope_gpu import TOL, problem
from workloads import to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


def check(x, w, go, dx, dw, pos, f, ax, inter, dt):
    x64, w64, go64 = to_f64(x), to_f64(w), to_f64(go)
    rx, rw = tm.norm_rope_bwd(x64, w64, go64, pos, f, ax, True, 0.0, inter)
    r = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True))
    g = np.abs(go64).max(-1).transpose(0, 2, 1)[..., None]
    size = np.maximum(np.abs(rx).max(-1, keepdims=True), r * g * np.abs(w64).max())
    assert (np.abs(to_f64(dx) - rx) / size).max() <= 2 * TOL[dt]
    mag = (np.abs(x64) * r * g).sum((0, 1, 2))
    assert (np.abs(to_f64(dw) - rw) <= 2 * 160 * 2.0 ** -24 * mag).all()


SHAPES = [
    # B, N, Hq, Hk, D, R: odd head counts, token counts that leave a tile partly filled
    (1, 3, 3, 1, 64, 32),
    (2, 33, 1, 1, 128, 64),
    (1, 7, 5, 3, 96, 36),
    (3, 50, 2, 1, 32, 12),
    (1, 5, 3, 1, 20, 10),              # the row kernel
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward_without_an_epsilon(la, shape, inter, dt):
    B, N, Hq, Hk, D, R = shape
    q, k, pos, f, ax, wq, wk, _ = problem(B, N, Hq, Hk, D, R, 1, dt, N + D)
    table, how = la.la_rope_table(f, ax), dict(wq=wq, wk=wk, eps=0.0, interleaved=inter)
    qo, ko = la.la_qk_norm_rope_fwd(q, k, pos.cuda(), table, **how)
    dqo, dko = torch.randn_like(qo), torch.randn_like(ko)
    dq, dk, dwq, dwk = la.la_qk_norm_rope_bwd(q, k, dqo, dko, pos.cuda(), table, **how)
    torch.cuda.synchronize()
    check(q, wq, dqo, dq, dwq, pos.numpy(), f, ax, inter, dt)
    check(k, wk, dko, dk, dwk, pos.numpy(), f, ax, inter, dt)
