"""What bf16 outputs and gradients of la_decay_attn_fwd / _bwd lose beside their own rounding on the
tensor cores: the same in calls of every size, for every sequence of them.

Per element, from the sum of magnitudes `mag` of its terms (the oracle run on absolute values).
Two bf16 terms leave half a step twice of a value, 2^-8 of 2^-8: of a weighted score 2^-16, of the
state where it is read 2^-16, and 2^-16 of what each token added to a state that is not returned. The
fp32 sums and weights add f = (D + N / 16 + 192) 2^-24 as in test_decay_attn_gpu.py, and the output is
rounded once (2^-8). In sequences of one chunk from zero the state plays no part.
"""
import numpy as np
import pytest
import torch

from oracle import token_mixing as tm
from test_decay_attn_gpu import near, problem
from workloads import to_f64

pytestmark = pytest.mark.gpu

EACH = 2.0 ** -16


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


def check(got, ref, mag, D, N, terms, what):
    f = (D + N / 16 + 192) * 2.0 ** -24
    near(got, ref, (terms * EACH + f) * 1.01 * mag + 2.0 ** -8 * np.abs(ref), what)


def both_ways(la, x, decay, lengths=None, terms=1):
    """Outputs and gradients against the oracle, `terms` values of two bf16 terms on each term's way."""
    q, k, v, do = x
    N, Dk, Dv = q.shape[2], q.shape[3], v.shape[3]
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    a, d = [to_f64(t) for t in x], to_f64(decay)
    ref, mag = (tm.decay_attn(*(f(t) for t in a[:3]), d, 0.125, lengths)[0] for f in (np.asarray, np.abs))
    check(la.la_decay_attn_fwd(q, k, v, decay, 0.125, n), ref, mag, Dk, N, terms, "o")
    got = la.la_decay_attn_bwd(*x, decay, 0.125, n)
    ref, mag = (tm.decay_attn_bwd(*(f(t) for t in a), d, 0.125, lengths) for f in (np.asarray, np.abs))
    for g, r, m, D, what in zip(got, ref, mag, (Dv, Dv, Dk), ("dq", "dk", "dv")):
        check(g, r, m, D, N, terms, what)


# Short sequences in numbers; the few-rows calls of test_decay_attn_gpu.py have the same bound.
@pytest.mark.parametrize("shape", [(550, 2, 1, 64, 64), (40, 16, 3, 64, 64), (9, 16, 128, 64, 64), (80, 4, 100, 64, 40),
                                   (5, 8, 128, 128, 128), (12, 8, 40, 64, 128), (12, 8, 77, 128, 64)])
def test_short_sequences_in_a_large_batch(la, shape):
    x, decay, _ = problem(*shape, "bf16", 47)
    both_ways(la, x, decay)


def test_a_sequence_alone_and_in_a_batch(la):
    # Short sequences among padding: one of them alone has 60 rows, the call 8 x 4 x 128.
    x, decay, _ = problem(8, 4, 128, 64, 64, "bf16", 53)
    both_ways(la, x, decay, lengths=[60, 1, 128, 0, 17, 100, 2, 31])
    both_ways(la, [t[:1, :, :60] for t in x], decay)


# The state in two terms, the tokens that made it in two: three values on a term's way at most.
@pytest.mark.parametrize("shape", [(1, 1, 1024, 64, 64), (2, 2, 300, 64, 64), (8, 8, 520, 64, 48), (2, 8, 1500, 64, 64),
                                   (4, 4, 400, 64, 128), (4, 4, 400, 128, 64), (1, 2, 1300, 40, 128)])
def test_states_that_are_read_lose_no_more(la, shape):
    x, decay, _ = problem(*shape, "bf16", 59)
    both_ways(la, x, decay, terms=3)
