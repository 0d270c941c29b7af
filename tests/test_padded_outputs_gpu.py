"""Padded batches of the convolution and the scan without a y of the caller's: the rows
past each length of the tensor that the call makes are zero."""
import pytest
import torch

from test_selective_scan_gpu import DT, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


def leave_nan(shape, dtype):
    """Leaves NaN in memory that the next allocation of this size is given."""
    torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    torch.cuda.synchronize()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_scan(la, dt):
    p = problem(3, 200, 2, 1, 64, 64, dt, 51)
    n = [200, 0, 130]
    leave_nan((3, 200, 2, 64), DT[dt])
    y = la.la_selective_scan_fwd(**p, lengths=torch.tensor(n, dtype=torch.int32, device="cuda"))
    for b in range(3):
        assert (y[b, n[b]:] == 0).all() and torch.isfinite(y[b]).all()
        assert n[b] == 0 or (y[b, :n[b]] != 0).any()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_convolution(la, dt):
    x, w = torch.randn(3, 50, 64, device="cuda").to(DT[dt]), torch.randn(64, 4, device="cuda").to(DT[dt])
    n = [50, 0, 21]
    leave_nan((3, 50, 64), DT[dt])
    y = la.la_short_conv_fwd(x, w, lengths=torch.tensor(n, dtype=torch.int32, device="cuda"))
    for b in range(3):
        assert (y[b, n[b]:] == 0).all() and torch.isfinite(y[b]).all()
        assert n[b] == 0 or (y[b, :n[b]] != 0).any()
