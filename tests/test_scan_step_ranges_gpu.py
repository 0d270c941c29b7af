"""Batches and states of la_selective_scan_step that need no bound: more than 65535 heads
in all, and states on any 4-byte boundary where no 16-byte access reads them. Against the
float64 oracle, with the bounds of test_selective_scan_gpu.py."""
import pytest
import torch

from test_selective_scan_gpu import check, oracle, problem

pytestmark = pytest.mark.gpu

TOKEN = ("x", "Bm", "Cm", "step", "z")


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


def run(la, p, state, S, dt):
    q = {k: (v[:, 0] if k in TOKEN else v) for k, v in p.items() if k != "S0"}
    y = la.la_selective_scan_step(**q, S=state)
    torch.cuda.synchronize()
    check(y.unsqueeze(1), state, oracle(p), 1, S, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,S,P", [(2048, 33, 8, 8), (65537, 1, 3, 5)])
def test_more_heads_than_a_grid_is_high(la, B, H, S, P, dt):
    p = problem(B, 1, H, 1, S, P, dt, 61)
    run(la, p, p["S0"].clone(), S, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_a_sequence_of_a_batch_of_odd_states(la, dt):
    # One sequence's state of a batch: 33 x 5 floats, 4-byte aligned.
    p = problem(1, 1, 1, 1, 33, 5, dt, 62)
    states = torch.zeros(3, 1, 33, 5, device="cuda")
    states[1] = p["S0"][0]
    assert states[1:2].data_ptr() % 16 != 0
    run(la, p, states[1:2], 33, dt)
    assert (states[0] == 0).all() and (states[2] == 0).all()
