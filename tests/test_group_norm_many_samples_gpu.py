"""Group norm of many samples with few tokens each, against the float64 oracle: the backward's blocks
take several samples each, and the weights' gradients are sums over all of them."""
import pytest
import torch

from test_group_norm_gpu import check, la, problem  # noqa: F401

pytestmark = pytest.mark.gpu


# More samples than blocks at once (two or three per SM); groups of whole and of odd widths, several
# blocks of channels, single values.
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("shape", [(1000, 2, 64, 4), (457, 3, 320, 32), (913, 17, 40, 5), (600, 5, 35, 5), (500, 2, 2100, 300),
                                   (700, 33, 48, 1), (20000, 2, 8, 2)])
def test_matches_oracle(la, shape, gate, dt):  # noqa: F811
    B, N, C, G = shape
    p, dy = problem(B, N, C, dt, B + N + C)
    if not gate:
        p["z"] = None
    check(la, p, G, dy, silu=(C + gate) % 2 == 0, dt=dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_the_same_bits_every_time(la, dt):  # noqa: F811
    p, dy = problem(3000, 4, 96, dt, 3)
    y, s = la.la_group_norm_fwd(p["x"], 8, p["w"], p["b"], p["z"], True, return_stats=True)
    want = la.la_group_norm_bwd(p["x"], 8, dy, s, p["w"], p["b"], p["z"], True)
    ws = la.group_norm_workspace(3000, 4, 96, 8)
    for _ in range(3):
        ws.fill_(255)                                       # whatever it held
        got = la.la_group_norm_bwd(p["x"], 8, dy, s, p["w"], p["b"], p["z"], True, ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
