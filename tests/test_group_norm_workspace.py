"""The group norm's workspace grows with the samples by their groups' statistics alone (no GPU)."""
import pytest


@pytest.mark.parametrize("B,N,C,G", [(65536, 4, 320, 32), (65536, 16, 64, 8), (1 << 20, 2, 512, 8), (3, 4096, 320, 32)])
def test_workspace_of_many_samples(B, N, C, G):
    import linear_attention_elu_gb300 as la
    # A pair of values per sample and group for each of its blocks of rows, and the weights' sums of
    # at most three blocks per SM, at most 160 SMs; rounded up to 256 bytes.
    blocks = B if B > 3 * 160 else 3 * 160
    assert la.la_group_norm_workspace_size(B, N, C, G) <= 4 * 2 * (blocks * G + 3 * 160 * C) + 256
