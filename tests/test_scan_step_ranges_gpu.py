"""Batches and states of la_selective_scan_step that need no bound: more than 65535 heads
in all. Against the float64 oracle, with the bounds of test_selective_scan_gpu.py."""
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
