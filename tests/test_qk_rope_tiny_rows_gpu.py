"""la_qk_norm_rope_bwd of rows so small that their inverse norm's cube is past fp32's range.
Bounds of test_qk_rope_small_eps_gpu.py."""
import pytest
import torch

from test_qk_rope_gpu import problem
from test_qk_rope_small_eps_gpu import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D,R", [(64, 32), (20, 10)])
@pytest.mark.parametrize("scale", [2.0 ** -50, 2.0 ** -60])
def test_rows_whose_inverse_norm_cubed_passes_fp32(la, scale, D, R, dt):
    # 1 / |x| near 2^50: its cube is past fp32's range, the gradient, near |g| / |x|, is not.
    q, k, pos, f, ax, wq, wk, _ = problem(1, 9, 2, 1, D, R, 1, dt, D)
    q, k = q.clone(), k.clone()
    q[0, 2] *= scale
    k[0, 5:] *= scale
    table, how = la.la_rope_table(f, ax), dict(wq=wq, wk=wk, eps=0.0)
    qo, ko = la.la_qk_norm_rope_fwd(q, k, pos.cuda(), table, **how)
    dqo, dko = torch.randn_like(qo), torch.randn_like(ko)
    dq, dk, dwq, dwk = la.la_qk_norm_rope_bwd(q, k, dqo, dko, pos.cuda(), table, **how)
    torch.cuda.synchronize()
    check(q, wq, dqo, dq, dwq, pos.numpy(), f, ax, False, dt)
    check(k, wk, dko, dk, dwk, pos.numpy(), f, ax, False, dt)
