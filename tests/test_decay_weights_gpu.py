"""Weights of la_decay_attn_fwd's scores between neighbouring tokens on the tensor cores."""
import numpy as np
import pytest
import torch

from oracle import token_mixing as tm
from test_decay_attn_gpu import near
from workloads import to_f64

pytestmark = pytest.mark.gpu

EACH = 2.0 ** -16                                            # what two bf16 terms leave of a score


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


@pytest.mark.parametrize("B", [1, 40])
@pytest.mark.parametrize("l", [-0.5, -0.9, -1.0, -1.3])
def test_weights_within_a_block_of_tokens(la, l, B):
    """Two terms that cancel, so that the weight of one shows: a token `gap` back, and the token itself
    with minus that weight in its key. A weight 2^x, x = gap l log2 e, is off by half a step of x and of
    log2 f (2^-23 |x| ln 2 in all) and by 2^-22 of its exponential; each term by 2^-16 of itself."""
    H, N, D, x0 = 8, 64, 64, 40.0
    gaps = [3, 9, 17, 20, 25, 28, 30, 31]
    q, k, v = (torch.zeros(B, H, N, D) for _ in range(3))
    at = 31                                                  # the last row of a block of 32
    for h, gap in enumerate(gaps):
        w = float(np.exp(np.float64(np.float32(l)) * gap))
        q[:, h, at, h], k[:, h, at - gap, h], k[:, h, at, h] = 1.0, 2.0 ** x0, -w * 2.0 ** x0
        v[:, h, at - gap], v[:, h, at] = 1.0, 1.0
    q, k, v = (t.bfloat16().cuda() for t in (q, k, v))
    decay = torch.full((H,), l, device="cuda")
    a, d = [to_f64(t) for t in (q, k, v)], to_f64(decay)
    ref, mag = (tm.decay_attn(*(f(t) for t in a), d)[0] for f in (np.asarray, np.abs))
    x = np.array(gaps) * abs(l) / np.log(2)
    each = (EACH + 2.0 ** -22 + 2.0 ** -23 * x * np.log(2))[None, :, None, None]
    o = la.la_decay_attn_fwd(q, k, v, decay)
    near(o[:, :, at:at + 1], ref[:, :, at:at + 1], 1.01 * each * mag[:, :, at:at + 1] + 2.0 ** -8 * np.abs(ref[:, :, at:at + 1]), "o")
