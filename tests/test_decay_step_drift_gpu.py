"""la_decay_attn_step over thousands of tokens against the float64 recurrence.

A step rounds each element of the state once to fp32, off by at most half a step, 2^-24 of the
element. Where the token added has as many digits as the state, the direction is as good as
random, and n such roundings, each carried over the steps behind it, leave the root of the sum of
their squares; taken at their largest that is sqrt(sum_t (f^(n-t) 2^-24 S_t)^2), and roundings spread
evenly over a step leave 3^-1/2 of it. The factor itself adds nothing to that: a factor off by
its own rounding (2^-25 and more, always the same way) would be n 2^-25 off, 8 to 100 times as much here.

A product of two bf16 values has 16 digits: it leaves the last places of a larger state as they
are, and what the decay rounds there can go the same way for thousands of steps, so that the
bound is the sum of the half steps, sum_t f^(n-t) 2^-24 |S_t|. What bf16 adds to the test is the bits: those
of the same values held in fp32.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TOKENS = 8192


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,Dk,Dv", [(2, 16, 16), (2, 16, 17)])
def test_a_slow_decay_does_not_drift(B, Dk, Dv, dt):
    import linear_attention_elu_gb300 as la
    l = np.array([-1e-6, -2.0 ** -12, -1.3e-5, 0.0], np.float32)
    H = len(l)
    g = torch.Generator().manual_seed(7)
    k = (0.05 * torch.randn(TOKENS, B, H, Dk, generator=g)).to(dt)
    v = torch.randn(TOKENS, B, H, Dv, generator=g).to(dt)
    S0 = 4 * torch.randn(B, H, Dk, Dv, generator=g)
    decay = torch.from_numpy(l).cuda()

    def steps(kd, vd):
        S, o = S0.cuda(), torch.empty(B, H, Dv, dtype=kd.dtype, device="cuda")
        for t in range(TOKENS):
            la.la_decay_attn_step(kd[t], kd[t], vd[t], decay, S, o=o)
        return S

    S = steps(k.cuda(), v.cuda())
    if dt == torch.bfloat16:
        assert torch.equal(S, steps(k.float().cuda(), v.float().cuda()))
    f = np.exp(l.astype(np.float64))[:, None, None]
    ref, squares, sums = S0.double().numpy(), np.zeros(S0.shape), np.zeros(S0.shape)
    k, v = k.double().numpy(), v.double().numpy()
    for t in range(TOKENS):
        ref = f * ref + k[t][..., :, None] * v[t][..., None, :]
        squares = f * f * squares + (2.0 ** -24 * ref) ** 2
        sums = f * sums + 2.0 ** -24 * np.abs(ref)
    rms = lambda x: np.sqrt((x * x).mean((0, 2, 3)))  # noqa: E731
    err, most = rms(S.double().cpu().numpy() - ref), rms(np.sqrt(squares) if dt == torch.float32 else sums)
    assert (err <= most).all(), err / most
