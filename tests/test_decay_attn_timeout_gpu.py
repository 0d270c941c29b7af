"""The decayed attention's bounded waits: with its loads withheld (the workspace header's test
hook) every wait gives up, the status says so, and the context stays usable."""
import pytest
import torch

from test_decay_attn_gpu import problem

pytestmark = pytest.mark.gpu

MAX_SPIN_WORD, HOLD_WORD = 4, 5   # uint32 index of max_spin and hold_item in the header


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("B,N", [(1, 1500), (40, 200)])       # with segments, without
def test_withheld_loads_time_out(la, B, N, backward, D):
    (q, k, v, do), decay, _ = problem(B, 2, N, D, D, "bf16", 3, "head")
    ws = la.workspace(la.LA_OP_DECAY_ATTN_BWD if backward else la.LA_OP_DECAY_ATTN, B, 2, N, D, D, q.dtype)

    def call():
        if backward:
            return la.la_decay_attn_bwd(q, k, v, do, decay, ws=ws)
        return [la.la_decay_attn_fwd(q, k, v, decay, ws=ws)]

    want = call()
    assert la.la_query_status(ws) == 0
    hdr = ws[:256].view(torch.int32)
    hdr[MAX_SPIN_WORD] = 1000  # 1 ms
    hdr[HOLD_WORD] = 1
    call()
    assert la.la_query_status(ws) == la.LA_ERR_TIMEOUT
    assert la.la_query_status(ws) == 0          # the status word was cleared
    la.la_workspace_init(ws)                     # default limit, hook off
    got = call()
    assert la.la_query_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
