"""The same call of the selective scan again and again gives the same bits: outputs and
states do not depend on how its warps, copies and tensor-core products happen to meet."""
import pytest
import torch

from test_selective_scan_gpu import problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


SHAPES = [
    # B, N, H, G, S, P
    (1, 300, 303, 1, 64, 64),          # two units per CTA, the last CTA one
    (1, 140, 304, 1, 64, 16),
    (2, 129, 152, 2, 128, 128),        # both units of a CTA of one head
    (1, 700, 306, 2, 16, 8),
    (1, 4000, 32, 1, 128, 64),         # segments
    (8, 333, 16, 1, 128, 64),          # one unit per CTA
]


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_same_bits_every_time(la, shape, gate):
    B, N, H, G, S, P = shape
    p = problem(B, N, H, G, S, P, "bf16", N + H)
    if not gate:
        p["z"] = None
    want, state = torch.empty(B, H, S, P, device="cuda"), torch.empty(B, H, S, P, device="cuda")
    first = la.la_selective_scan_fwd(**p, S_out=want)
    for _ in range(100):
        y = la.la_selective_scan_fwd(**p, S_out=state)
        assert torch.equal(y, first) and torch.equal(state, want)
