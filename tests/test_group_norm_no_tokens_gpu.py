"""la_group_norm_fwd without tokens: nothing to write but the statistics, which are zeros and not
whatever the buffer held."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B", [0, 1, 3])
def test_statistics_of_no_tokens(B, dt):
    import linear_attention_elu_gb300 as la
    x, w = torch.empty(B, 0, 8, device="cuda", dtype=dt), torch.ones(8, device="cuda", dtype=dt)
    buf = torch.full((B + 2, 2, 2), 7.0, device="cuda")
    given = buf[1:B + 1]
    y, s = la.la_group_norm_fwd(x, 2, w, w, stats=given, return_stats=True)
    assert y.shape == x.shape and s is given
    assert (la.la_group_norm_fwd(x, 2, w, w, return_stats=True)[1] == 0).all()
    assert (buf[1:B + 1] == 0).all() and (buf[0] == 7).all() and (buf[B + 1:] == 7).all()
    dx, dw, db, _ = la.la_group_norm_bwd(x, 2, x, s, w, w)
    assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all()
    if B == 0:
        return
    # Captured: the statistics are part of the graph.
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.la_group_norm_fwd(x, 2, w, w, stats=buf[1:B + 1])
    buf.fill_(5.0)
    graph.replay()
    torch.cuda.synchronize()
    assert (buf[1:B + 1] == 0).all() and (buf[0] == 5).all()
