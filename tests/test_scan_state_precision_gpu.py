"""The state that the bf16 scan returns is an fp32 state: a single token's contribution,
alone in its sequence (every other step is masked), against 64 bits.

Bound, in units of 2^-24 of each entry: the step size 4 (its softplus), its product with
the value 1, what three bf16 terms leave of that product 1/2, and the sum of the three
terms' products in fp32 with at most 2 (a truncated last place) each for them and for the
sums that pass the entry on to the end (first pass, chaining): below 16. Two terms alone
would leave up to 128."""
import numpy as np
import pytest
import torch

from oracle import token_mixing as tm
from test_selective_scan_gpu import problem
from workloads import to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


@pytest.mark.parametrize("S,P", [(128, 64), (64, 64), (16, 128)])
@pytest.mark.parametrize("N,at", [(1, 0), (150, 0), (150, 77), (150, 149), (1500, 3), (1500, 700), (1500, 1499)])
def test_one_token(la, N, at, S, P):
    p = problem(2, N, 4, 2, S, P, "bf16", N + at + S)
    step = torch.full_like(p["step"], float("-inf"))
    step[:, at] = p["step"][:, at]
    p.update(step=step, S0=None)
    S_out = torch.empty(2, 4, S, P, device="cuda")
    la.la_selective_scan_fwd(**p, S_out=S_out)
    torch.cuda.synchronize()
    d = tm.softplus(to_f64(step[:, at]) + to_f64(p["dt_bias"]))
    want = d[:, :, None, None] * to_f64(p["Bm"][:, at]).repeat(2, 1)[..., None] * to_f64(p["x"][:, at])[:, :, None]
    assert (np.abs(to_f64(S_out) - want) <= 16 * 2.0 ** -24 * np.abs(want)).all()
