"""Large and small steps in one chunk of the selective scan, against the float64 oracle.

Bounds as in test_selective_scan_gpu.py, and for the tensor-core path the decays between
tokens of a chunk: an exponent there is a difference of sums over at most 32 tokens of
exponents held within 127, so below 4096 in magnitude, in fp32; a sum is rounded at most
seven times on its way, by 2^-13 each at most, so a decay is off by 14 2^-13 ln 2 of
itself at most."""
import math

import numpy as np
import pytest
import torch

from test_selective_scan_gpu import DT, oracle, problem
from workloads import to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


def check(y, S, ref, N, Sn, dt):
    ry, rS, ym, Sm = ref
    f = (8 * N + Sn + 32) * 2.0 ** -24
    if dt == "bf16":
        ty = (2.0 ** -8 + f + 14 * 2.0 ** -13 * math.log(2)) * ym * 1.01 + 2.0 ** -8 * np.abs(ry)
        tS = (2.0 ** -16 + f) * Sm
    else:
        ty, tS = f * ym, f * Sm
    ey, eS = np.abs(to_f64(y) - ry), np.abs(to_f64(S) - rS)
    assert (ey <= ty + 1e-30).all(), (ey - ty).max()
    assert (eS <= tS + 1e-30).all(), (eS - tS).max()


def run(la, step, rate, dt, S=64, seed=31):
    """Steps given directly [N]; a bf16 problem takes them as rounded."""
    N = len(step)
    p = problem(1, N, 2, 1, S, 64, dt, seed)
    p["step"] = torch.tensor(step, device="cuda").to(DT[dt]).view(1, N, 1).expand(1, N, 2).contiguous()
    p["A"] = torch.tensor([rate, -1.0], device="cuda")
    p["dt_bias"] = None
    S_out = torch.empty(1, 2, S, 64, device="cuda")
    y = la.la_selective_scan_fwd(**p, S_out=S_out, softplus=False)
    torch.cuda.synchronize()
    check(y, S_out, oracle(p, use_softplus=False), N, S, dt)


# A reset of the state (one token of a very large exponent) and slow decays after it: within
# a block of 32 tokens, on its borders, and with the slow tokens in later blocks.
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("at", [0, 5, 31, 32, 64, 95, 127])
@pytest.mark.parametrize("exponent", [3e4, 1e5, 1e6, 1e7])
def test_slow_decays_after_a_reset(la, dt, at, exponent):
    step = [1e-5] * 200
    step[at] = exponent / 1e3
    run(la, step, -1e3, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("at", [0, 40, 127])
def test_an_exponent_past_the_largest_number(la, dt, at):
    step = [1.25e-38] * 200                # times the rate 3.75
    step[at] = step[at + 3] = 10.0         # minus infinity
    run(la, step, -3e38, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rate,large,small", [(-16.0, 10.0, 0.01), (-100.0, 3.0, 0.001)])
@pytest.mark.parametrize("order", ["half", "turns", "end"])
def test_large_and_small_steps_in_one_chunk(la, dt, rate, large, small, order):
    N = 384
    big = {"half": lambda t: t % 128 < 64, "turns": lambda t: t % 3 == 0, "end": lambda t: t % 128 > 90}[order]
    run(la, [large if big(t) else small for t in range(N)], rate, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_resets_in_segments(la, dt):
    # Long enough to be cut into segments; a reset every 300 tokens.
    run(la, [1e6 if t % 300 == 17 else 1e-4 for t in range(3100)], -100.0, dt, S=128)
