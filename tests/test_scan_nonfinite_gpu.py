"""Infinities and NaN in a token's values of the selective scan: outputs before the token,
and of other columns and heads, are those without it; the token's column is not finite from
there on, its state included. Bounds as in test_selective_scan_gpu.py."""
import pytest
import torch

from test_selective_scan_gpu import check, oracle, problem

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


SHAPES = [
    # dt, N, H, S, P
    ("bf16", 150, 2, 128, 64),         # one unit per CTA
    ("bf16", 300, 306, 64, 64),        # two
    ("bf16", 140, 152, 64, 128),       # both of one head
    ("bf16", 1500, 2, 128, 64),        # segments
    ("bf16", 150, 2, 33, 20),          # the recurrence
    ("f32", 150, 2, 64, 64),
    ("f32", 1500, 2, 64, 64),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("at,value", [(0, NAN), (77, INF), (77, -INF), (77, NAN), (127, NAN), (130, INF)])
def test_values_that_are_not_finite_stay_behind_their_token(la, shape, gate, at, value):
    dt, N, H, S, P = shape
    p = problem(1, N, H, 1, S, P, dt, N + H)
    if not gate:
        p["z"] = None
    p["x"] = p["x"].clone()
    cols = [0, 13, P - 1]
    p["x"][0, at, 1, cols] = 0
    ref = oracle(p)
    p["x"][0, at, 1, cols] = value
    S_out = torch.empty(1, H, S, P, device="cuda")
    y = la.la_selective_scan_fwd(**p, S_out=S_out)
    torch.cuda.synchronize()
    assert not torch.isfinite(y[0, at:, 1, cols]).any() and not torch.isfinite(S_out[0, 1][:, cols]).any()
    # What does not depend on them is held to the bounds.
    y, S_out = y.clone(), S_out.clone()
    y[0, at:, 1, cols] = 0
    S_out[0, 1][:, cols] = 0
    ry, rS, ym, Sm = ref
    for r in (ry, ym):
        r[0, at:, 1, cols] = 0
    for r in (rS, Sm):
        r[0, 1][:, cols] = 0
    check(y, S_out, ref, N, S, dt)


def test_every_column_at_once_and_two_tokens(la):
    p = problem(1, 200, 2, 1, 128, 64, "bf16", 41)
    p["x"] = p["x"].clone()
    ref = oracle(dict(p, x=p["x"].clone()))
    p["x"][0, 100, 0] = NAN
    p["x"][0, 40, 1, 7], p["x"][0, 20, 1, 7] = INF, NAN
    S_out = torch.empty(1, 2, 128, 64, device="cuda")
    y = la.la_selective_scan_fwd(**p, S_out=S_out)
    torch.cuda.synchronize()
    bad = torch.zeros(y.shape, dtype=torch.bool)
    bad[0, 100:, 0] = True
    bad[0, 20:, 1, 7] = True
    assert torch.equal(~torch.isfinite(y).cpu(), bad)
    ry, rS, ym, Sm = ref
    y, S_out = y.cpu().masked_fill(bad, 0), S_out.cpu()
    for r in (ry, ym):
        r[bad.numpy()] = 0
    assert not torch.isfinite(S_out[0, 0]).any() and not torch.isfinite(S_out[0, 1, :, 7]).any()
    for r in (rS, Sm):
        r[0, 0], r[0, 1, :, 7] = 0, 0
    S_out[0, 0], S_out[0, 1, :, 7] = 0, 0
    check(y, S_out, ref, 200, 128, "bf16")


@pytest.mark.parametrize("S,P", [(128, 64), (64, 40), (33, 20)])
def test_in_the_last_chunk_of_a_padded_batch(la, S, P):
    p = problem(2, 300, 2, 1, S, P, "bf16", 42)
    p["x"] = p["x"].clone()
    n = [200, 300]
    p["x"][0, 150, 1, 5], p["x"][0, 250] = 0, INF          # behind the length: not there
    ref = [oracle({k: (v[b:b + 1, :n[b]] if k in ("x", "Bm", "Cm", "step", "z") else v[b:b + 1] if k == "S0" else v)
                   for k, v in p.items()}) for b in range(2)]
    p["x"][0, 150, 1, 5] = NAN
    y = torch.full((2, 300, 2, P), 5.0, dtype=torch.bfloat16, device="cuda")
    S_out = torch.empty(2, 2, S, P, device="cuda")
    la.la_selective_scan_fwd(**p, lengths=torch.tensor(n, dtype=torch.int32, device="cuda"), y=y, S_out=S_out)
    torch.cuda.synchronize()
    assert (y[0, 200:] == 5).all()
    assert not torch.isfinite(y[0, 150:200, 1, 5]).any() and not torch.isfinite(S_out[0, 1, :, 5]).any()
    y[0, 150:200, 1, 5], S_out[0, 1, :, 5] = 0, 0
    ref[0][0][0, 150:, 1, 5] = ref[0][2][0, 150:, 1, 5] = 0
    ref[0][1][0, 1, :, 5] = ref[0][3][0, 1, :, 5] = 0
    for b in range(2):
        check(y[b:b + 1, :n[b]], S_out[b:b + 1], ref[b], n[b], S, "bf16")
