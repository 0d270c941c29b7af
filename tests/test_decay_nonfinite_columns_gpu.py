"""Infinities and NaN in a token of la_decay_attn_fwd: what they reach, and as what."""
import pytest
import torch

from test_decay_attn_gpu import problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("N,Dk,Dv", [(300, 64, 64), (1500, 64, 64), (90, 128, 128), (400, 64, 128)])
def test_what_a_value_reaches(N, Dk, Dv, value, dt):
    import linear_attention_elu_gb300 as la
    (q, k, v, _), _, S0 = problem(2, 2, N, Dk, Dv, dt, 73, "head")
    decay = torch.tensor([-0.001, -0.02], device="cuda")
    at, col = N // 2, 5
    S, T = torch.empty_like(S0), torch.empty_like(S0)
    clean = la.la_decay_attn_fwd(q, k, v, decay, 0.125, S0=S0, S_out=S)
    for what in ("q", "k", "v"):
        x = dict(q=q.clone(), k=k.clone(), v=v.clone())
        x[what][1, 0, at, col] = value
        o = la.la_decay_attn_fwd(*x.values(), decay, 0.125, S0=S0, S_out=T)
        assert torch.equal(o[0], clean[0]) and torch.equal(o[1, 1], clean[1, 1]) and torch.equal(o[1, 0, :at], clean[1, 0, :at])
        hit = slice(col, col + 1) if what == "v" else slice(None)
        rows = slice(at, at + 1) if what == "q" else slice(at, None)
        bad = o[1, 0, rows, hit]
        assert not torch.isfinite(bad).any()
        if dt == "bf16":
            assert torch.isnan(bad).all()
        left = o[1, 0].clone()
        left[rows, hit] = clean[1, 0, rows, hit]
        assert torch.equal(left, clean[1, 0])
        # The state: a row for k, a column for v.
        state = T.clone()
        if what != "q":
            part = (slice(None), col) if what == "v" else (col,)
            assert not torch.isfinite(T[1, 0][part]).any()
            state[1, 0][part] = S[1, 0][part]
        assert torch.equal(state, S)
