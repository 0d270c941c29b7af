"""Pins of the float64 decayed attention and group norm: closed forms, sums written out
term by term, and central differences of the gradients."""
import numpy as np
import pytest

from oracle import token_mixing as tm


def rand(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def test_decay_attn_is_its_double_sum():
    B, H, N, Dk, Dv = 2, 3, 7, 4, 5
    q, k, v = rand(1, B, H, N, Dk), rand(2, B, H, N, Dk), rand(3, B, H, N, Dv)
    S0, l = rand(4, B, H, Dk, Dv), -np.array([0.0, 0.3, 40.0])
    lengths = [7, 4]
    o, S = tm.decay_attn(q, k, v, l, 0.5, lengths, S0)
    for b in range(B):
        for h in range(H):
            n = lengths[b]
            for t in range(N):
                want = np.zeros(Dv)
                if t < n:
                    want = np.exp(l[h] * (t + 1)) * q[b, h, t] @ S0[b, h]
                    for j in range(t + 1):
                        want = want + np.exp(l[h] * (t - j)) * (q[b, h, t] @ k[b, h, j]) * v[b, h, j]
                assert np.allclose(o[b, h, t], 0.5 * want, rtol=1e-12, atol=1e-14)
            end = np.exp(l[h] * n) * S0[b, h]
            for j in range(n):
                end = end + np.exp(l[h] * (n - 1 - j)) * np.outer(k[b, h, j], v[b, h, j])
            assert np.allclose(S[b, h], end, rtol=1e-12, atol=1e-14)


def test_decay_of_nothing_and_without_decay():
    q, k, v = rand(1, 1, 2, 6, 3), rand(2, 1, 2, 6, 3), rand(3, 1, 2, 6, 4)
    o, S = tm.decay_attn(q, k, v, [0.0, -np.inf])
    assert np.allclose(S[0, 0], np.einsum("td,te->de", k[0, 0], v[0, 0]))
    assert np.allclose(o[0, 1], (q[0, 1] * k[0, 1]).sum(-1, keepdims=True) * v[0, 1])
    S0 = rand(4, 1, 2, 3, 4)
    assert np.array_equal(tm.decay_attn(q[:, :, :0], k[:, :, :0], v[:, :, :0], [0.0, -1.0], S0=S0)[1], S0)


@pytest.mark.parametrize("lengths", [None, [5, 0]])
def test_decay_gradients_by_differences(lengths):
    B, H, N, Dk, Dv = 2, 2, 5, 3, 4
    x = [rand(i, B, H, N, D) for i, D in ((1, Dk), (2, Dk), (3, Dv))]
    do, l = rand(4, B, H, N, Dv), np.array([-0.2, -1.5])
    loss = lambda q, k, v: (tm.decay_attn(q, k, v, l, 0.7, lengths)[0] * do).sum()  # noqa: E731
    got = tm.decay_attn_bwd(*x, do, l, 0.7, lengths)
    for i in range(3):
        for at in np.ndindex(*x[i].shape):
            e = np.zeros_like(x[i])
            e[at] = 1e-5
            up, down = ([t + s * e if j == i else t for j, t in enumerate(x)] for s in (1, -1))
            assert abs((loss(*up) - loss(*down)) / 2e-5 - got[i][at]) < 1e-8


@pytest.mark.parametrize("use_silu", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_group_norm_statistics_and_gradients(use_silu, gate):
    B, N, C, G = 2, 3, 8, 4
    x, w, b, dy = 3 + rand(1, B, N, C), rand(2, C), rand(3, C), rand(4, B, N, C)
    z = rand(5, B, N, C) if gate else None
    plain, stats = tm.group_norm(x, G, eps=0.0)
    for g in range(G):
        v = plain[..., 2 * g:2 * g + 2].reshape(B, -1)
        assert np.allclose(v.mean(1), 0) and np.allclose(v.std(1), 1)
        assert np.allclose(stats[:, g, 0], x[..., 2 * g:2 * g + 2].mean((1, 2)))
    run = lambda x, w, b, z: (tm.group_norm(x, G, w, b, z, use_silu)[0] * dy).sum()  # noqa: E731
    grads = tm.group_norm_bwd(x, G, dy, w, b, z, use_silu)
    args = [x, w, b, z]
    for i, got in enumerate(grads):
        if got is None:
            assert i == 3 and not gate
            continue
        for at in np.ndindex(*args[i].shape):
            e = np.zeros_like(args[i])
            e[at] = 1e-5
            up, down = ([t + s * e if j == i else t for j, t in enumerate(args)] for s in (1, -1))
            assert abs((run(*up) - run(*down)) / 2e-5 - got[at]) < 1e-7
