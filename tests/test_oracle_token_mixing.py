"""Pins of the token-mixing oracle (oracle/token_mixing.py): values worked out
by hand, properties of the definitions, and gradients against differences."""
import numpy as np
import pytest

from oracle import token_mixing as tm


def test_rotation_worked_example():
    # One pair at position 3 with 0.5 radians per position: (1, 2) turned by 1.5 radians.
    x = np.array([[[[1.0, 2.0, 7.0]]]])
    out = tm.norm_rope(x, None, np.array([[[3]]]), [0.5], [0], norm=False)
    c, s = np.cos(1.5), np.sin(1.5)
    assert np.allclose(out[0, 0, 0], [c - 2 * s, 2 * c + s, 7.0], atol=1e-15)


def test_norm_worked_example():
    # Row (3, 4): mean square 12.5; weights (2, 1).
    x = np.array([[[[3.0, 4.0]]]])
    out = tm.norm_rope(x, [2.0, 1.0], np.zeros((1, 1, 1), int), [1.0], [0], eps=0.0)
    assert np.allclose(out[0, 0, 0], [6 / np.sqrt(12.5), 4 / np.sqrt(12.5)], atol=1e-15)


@pytest.mark.parametrize("inter", [False, True])
def test_products_depend_on_position_differences(inter):
    # With one axis, q_m . k_n of rotated rows depends on m - n only.
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 1, 8))
    f = [1.0, 0.3, 0.1]
    dot = lambda m, n: (tm.norm_rope(q, None, [[[m]]], f, [0, 0, 0], False, 0, inter)  # noqa: E731
                        * tm.norm_rope(k, None, [[[n]]], f, [0, 0, 0], False, 0, inter)).sum()
    assert abs(dot(7, 3) - dot(1004, 1000)) < 1e-12
    assert abs(dot(7, 3) - dot(3, 7)) > 1e-3


def test_axes_rotate_their_own_pairs():
    # Moving along axis 1 changes only the pairs of axis 1.
    x = np.random.default_rng(1).standard_normal((1, 1, 1, 8))
    at = lambda p: tm.norm_rope(x, None, [[p]], [1.0, 0.5, 1.0, 0.5], [0, 0, 1, 1], False, 0, True)  # noqa: E731
    d = np.abs(at([2, 5]) - at([2, 6]))[0, 0, 0] > 1e-9
    assert d.tolist() == [False] * 4 + [True] * 4


@pytest.mark.parametrize("norm,weighted,inter", [(True, True, False), (True, False, True),
                                                 (False, False, False)])
def test_gradients_match_differences(norm, weighted, inter):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((2, 3, 2, 6))
    w = rng.standard_normal(6) if weighted else None
    go = rng.standard_normal((2, 2, 3, 6))
    pos = rng.integers(-5, 50, (2, 3, 2))
    f, ax = [1.0, 0.2], [0, 1]
    dx, dw = tm.norm_rope_bwd(x, w, go, pos, f, ax, norm, 1e-6, inter)
    loss = lambda x, w: (tm.norm_rope(x, w, pos, f, ax, norm, 1e-6, inter) * go).sum()  # noqa: E731
    h = 1e-6
    for idx in [(0, 0, 0, 0), (1, 2, 1, 5), (0, 1, 1, 2), (1, 0, 0, 3)]:
        e = np.zeros_like(x)
        e[idx] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[idx]) < 1e-7
    if weighted:
        for i in range(6):
            e = np.zeros(6)
            e[i] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_conv_worked_example_and_state():
    # Two taps, one channel: y_t = 2 x_{t-1} + 3 x_t + 1.
    y, s = tm.short_conv(np.array([[[1.0], [2.0], [4.0]]]), [[2.0, 3.0]], [1.0], act=False)
    assert y[0, :, 0].tolist() == [4.0, 9.0, 17.0] and s[0, :, 0].tolist() == [4.0]
    # In two pieces through the state, and token by token, it is the same.
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((2, 9, 4)), rng.standard_normal((4, 4))
    full, last = tm.short_conv(x, w)
    state = np.zeros((2, 3, 4))
    parts = []
    for a, b in ((0, 2), (2, 3), (3, 9)):
        y, state = tm.short_conv(x[:, a:b], w, state=state)
        parts.append(y)
    assert np.allclose(np.concatenate(parts, 1), full, atol=1e-14) and np.allclose(state, last)


def test_conv_lengths():
    x = np.random.default_rng(4).standard_normal((3, 5, 2))
    s0 = np.random.default_rng(5).standard_normal((3, 2, 2))
    y, s = tm.short_conv(x, np.ones((2, 3)), lengths=[0, 1, 5], state=s0)
    assert (y[0] == 0).all() and np.array_equal(s[0], s0[0])
    assert np.array_equal(s[1], np.stack((s0[1, 1], x[1, 0]))) and (y[1, 1:] == 0).all()
    assert np.array_equal(s[2], x[2, 3:])


def test_scan_worked_example():
    # One state, one channel, step 1, A = -ln 2: S_t = S_{t-1} / 2 + B_t x_t.
    one = np.ones((1, 3, 1))
    x = np.array([[[[8.0]], [[2.0]], [[1.0]]]])
    y, S = tm.selective_scan(x, one, [-np.log(2.0)], one[..., None], 3 * one[..., None],
                             D=[10.0], use_softplus=False)
    assert np.allclose(y[0, :, 0, 0], [3 * 8 + 80, 3 * 6 + 20, 3 * 4 + 10]) and np.allclose(S, 4.0)


def test_scan_without_decay_is_a_prefix_sum():
    # A = 0 and step 1: y_t = sum_{j <= t} (C_t . B_j) x_j, causal linear attention's numerator.
    rng = np.random.default_rng(6)
    x, Bm, Cm = (rng.standard_normal((2, 7, 4, 3)), rng.standard_normal((2, 7, 2, 5)),
                 rng.standard_normal((2, 7, 2, 5)))
    y, S = tm.selective_scan(x, np.ones((2, 7, 4)), np.zeros(4), Bm, Cm, use_softplus=False)
    Bh, Ch = Bm.repeat(2, 2), Cm.repeat(2, 2)
    ref = np.einsum("bths,bjhs,tj,bjhp->bthp", Ch, Bh, np.tril(np.ones((7, 7))), x)
    assert np.allclose(y, ref, atol=1e-12)
    assert np.allclose(S, np.einsum("bjhs,bjhp->bhsp", Bh, x), atol=1e-12)


def test_scan_in_pieces_and_lengths():
    rng = np.random.default_rng(7)
    B, N, H, P, G, S = 2, 8, 2, 3, 1, 4
    x, z = rng.standard_normal((2, B, N, H, P))
    dt = rng.standard_normal((B, N, H))
    Bm, Cm = rng.standard_normal((2, B, N, G, S))
    A, D, bias = -np.ones(H), np.ones(H), rng.standard_normal(H)
    S0 = rng.standard_normal((B, H, S, P))
    full, last = tm.selective_scan(x, dt, A, Bm, Cm, D, z, bias, S0=S0)
    y1, s1 = tm.selective_scan(x[:, :3], dt[:, :3], A, Bm[:, :3], Cm[:, :3], D, z[:, :3], bias, S0=S0)
    y2, s2 = tm.selective_scan(x[:, 3:], dt[:, 3:], A, Bm[:, 3:], Cm[:, 3:], D, z[:, 3:], bias, S0=s1)
    assert np.allclose(np.concatenate((y1, y2), 1), full) and np.allclose(s2, last)
    y, s = tm.selective_scan(x, dt, A, Bm, Cm, D, z, bias, lengths=[3, 0], S0=S0)
    assert np.allclose(y[0, :3], full[0, :3]) and (y[0, 3:] == 0).all() and (y[1] == 0).all()
    assert np.allclose(s[0], s1[0]) and np.array_equal(s[1], S0[1])
