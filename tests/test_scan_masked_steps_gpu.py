"""Tokens masked out of the selective scan by their step size: with the softplus, a step
of minus infinity or of a type's lowest value is a step size of 0, and the token changes
nothing. Against the float64 oracle, with the bounds of test_selective_scan_gpu.py."""
import numpy as np
import pytest
import torch

from test_selective_scan_gpu import check, oracle, problem

pytestmark = pytest.mark.gpu

TOKEN = ("x", "Bm", "Cm", "step", "z")
MASKS = [float("-inf"), torch.finfo(torch.bfloat16).min, torch.finfo(torch.float32).min, -2.5e38]


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


def masked(p, N, value):
    """Left padding of sequence 0, tokens within it and its last one; all of sequence 1."""
    p["step"] = p["step"].clone()
    p["step"][0, :min(37, N - 1)] = value
    p["step"][0, 60:70] = value
    p["step"][0, N - 1] = value
    p["step"][1] = value
    return p


# One launch and segments; the tensor cores (bf16, whole 16-byte rows) and the recurrence.
@pytest.mark.parametrize("dt,S,P", [("bf16", 128, 64), ("bf16", 33, 20), ("f32", 64, 64)])
@pytest.mark.parametrize("N", [150, 1500])
@pytest.mark.parametrize("value", MASKS)
def test_masked_tokens_change_nothing(la, dt, S, P, N, value):
    p = masked(problem(2, N, 2, 1, S, P, dt, N + S), N, value)
    S_out = torch.empty(2, 2, S, P, device="cuda")
    y = la.la_selective_scan_fwd(**p, S_out=S_out)
    torch.cuda.synchronize()
    check(y, S_out, oracle(p), N, S, dt)
    assert torch.equal(S_out[1], p["S0"][1])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("value", MASKS)
def test_masked_single_tokens_change_nothing(la, dt, value):
    p = problem(3, 1, 2, 1, 64, 64, dt, 21)
    q = {k: (v[:, 0] if k in TOKEN else v) for k, v in p.items() if k != "S0"}
    q["step"] = q["step"].clone()
    q["step"][1] = value
    p["step"] = q["step"].unsqueeze(1)
    state = p["S0"].clone()
    y = la.la_selective_scan_step(**q, S=state)
    torch.cuda.synchronize()
    check(y.unsqueeze(1), state, oracle(p), 1, 64, dt)
    assert torch.equal(state[1], p["S0"][1])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_steps_that_are_not_numbers_stay_visible(la, dt):
    # A step of NaN is no mask: what follows it is NaN, what stands before it is not.
    p = problem(1, 40, 1, 1, 64, 64, dt, 22)
    p["step"] = p["step"].clone()
    p["step"][0, 20] = float("nan")
    S_out = torch.empty(1, 1, 64, 64, device="cuda")
    y = la.la_selective_scan_fwd(**p, S_out=S_out)
    torch.cuda.synchronize()
    assert y[:, 20:].isnan().all() and S_out.isnan().all() and torch.isfinite(y[:, :20]).all()


def test_large_steps_are_themselves(la):
    # softplus(v) = v in fp32 from v = 17 on, up to the largest.
    big = torch.tensor([17.0, 100.0, 1e20, 3e38], device="cuda")
    n = big.numel()
    one = torch.ones(1, n, 1, 1, device="cuda")
    S = torch.empty(1, n, 1, 1, device="cuda")
    y = la.la_selective_scan_fwd(one.view(1, 1, n, 1), big.view(1, 1, n), -torch.ones(n, device="cuda"),
                                 one[:, :1], one[:, :1], S_out=S)
    torch.cuda.synchronize()
    assert np.allclose(S.flatten().cpu(), big.cpu(), rtol=2.0 ** -22, atol=0)
    assert np.allclose(y.flatten().cpu(), big.cpu(), rtol=2.0 ** -22, atol=0)
