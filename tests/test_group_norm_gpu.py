"""la_group_norm_fwd / _bwd against the float64 oracle (oracle/token_mixing.py).

Tolerances, per element. A sum over a group passes at most kDepth roundings on its way
(8 values of a thread, the joins of its tiles, the rows and channels of a block, the blocks):
128 for the sizes here. So a mean is off by kDepth 2^-24 of the group's largest magnitude X,
and with the inverse deviation r (off by kDepth 2^-24 of itself, and by the mean's error in
the deviations) xh by kDepth 2^-24 (X r + |xh|) =: e_xh; u = w xh + b by |w| e_xh and its
roundings; silu and its derivative (Lipschitz constants 1.1 and 0.5) by that and a few 2^-22
of the hardware exponential and reciprocal. bf16 outputs are rounded once (2^-8).
"""
import numpy as np
import pytest
import torch

from oracle import token_mixing as tm
from workloads import to_f64

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
E = 128 * 2.0 ** -24


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


def problem(B, N, C, dt, seed, lead=0, mean=0.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (r(B, N, C) * (0.5 + torch.rand(C, generator=g)) + mean * r(C)).to(DT[dt]).cuda()
    z = r(B, N, lead + C).to(DT[dt]).cuda()[..., lead:]
    return dict(x=x, w=(1 + 0.2 * r(C)).to(DT[dt]).cuda(), b=(0.1 * r(C)).to(DT[dt]).cuda(), z=z), \
        r(B, N, C).to(DT[dt]).cuda()


def dsilu(z):
    s = tm._logistic(z)
    return s + z * s * (1 - s)


def check(la, p, G, dy, silu, dt, **kw):
    """Both directions, each output against its tolerance."""
    x, w, b, z = (p[n] for n in "xwbz")
    B, N, C = x.shape
    y, stats = la.la_group_norm_fwd(x, G, w, b, z, silu, return_stats=True, **kw)
    dx, dw, db, dz = la.la_group_norm_bwd(x, G, dy, stats, w, b, z, silu)
    torch.cuda.synchronize()
    X, W, Bc, Z, DY = (None if t is None else to_f64(t) for t in (x, w, b, z, dy))
    ry, rs = tm.group_norm(X, G, W, Bc, Z, silu)
    rdx, rdw, rdb, rdz = tm.group_norm_bwd(X, G, DY, W, Bc, Z, silu)
    wide = lambda t: np.repeat(t, C // G, -1)[:, None]  # noqa: E731
    top = np.abs(X).reshape(B, N, G, -1).max((1, 3))
    mean, r = rs[..., 0], rs[..., 1]
    half = 2.0 ** -8 if dt == "bf16" else 0.0

    def near(got, ref, tol, what):
        err = np.abs(to_f64(got) - ref)
        assert np.isfinite(err).all() and (err <= tol + 1e-30).all(), (what, (err - tol).max(), (err / (tol + 1e-30)).max())

    near(stats[..., 0], mean, E * top, "mean")
    near(stats[..., 1], r, E * r * (1 + top * r), "r")
    W1, B1 = (1.0 if W is None else W), (0.0 if Bc is None else Bc)
    xh = (X - wide(mean)) * wide(r)
    e_xh = E * (wide(top * r) + np.abs(xh) * (1 + wide(top * r)))
    u = W1 * xh + B1
    e_u = np.abs(W1) * e_xh + 2.0 ** -22 * (np.abs(W1 * xh) + np.abs(B1))
    a = tm.silu(u) if silu else u
    e_a = 1.1 * e_u + 2.0 ** -19 * np.abs(u) if silu else e_u
    gate = 1.0 if Z is None else tm.silu(Z)
    e_gate = 0.0 if Z is None else 2.0 ** -19 * np.abs(Z)
    e_y = e_a * np.abs(gate) + np.abs(a) * e_gate
    near(y, ry, 1.01 * e_y + (half + 2.0 ** -23) * np.abs(ry), "y")
    if Z is not None:
        near(dz, rdz, np.abs(DY) * (1.2 * e_a + 2.0 ** -19 * np.abs(a) * (1 + np.abs(Z))) + (half + 2.0 ** -22) * np.abs(rdz), "dz")
    else:
        assert dz is None
    slope = dsilu(u) if silu else np.ones_like(u)
    h = DY * gate * slope
    e_h = np.abs(DY) * (np.abs(gate) * (0.6 * e_u + 2.0 ** -19 * (1 + np.abs(u)) if silu else 0.0) + 1.1 * e_gate) \
        + 2.0 ** -22 * np.abs(h)
    rows = E * 4                                        # a thread's rows, the blocks' rows
    if dw is not None:
        near(dw, rdw, (rows * np.abs(h * xh) + e_h * np.abs(xh) + np.abs(h) * e_xh).sum((0, 1)), "dw")
    if db is not None:
        near(db, rdb, (rows * np.abs(h) + e_h).sum((0, 1)), "db")
    g, e_g = h * W1, e_h * np.abs(W1) + 2.0 ** -23 * np.abs(h * W1)
    over = lambda t: wide(t.reshape(B, N, G, -1).mean((1, 3)))  # noqa: E731
    s2, m2 = over(g * xh), over(np.abs(g * xh))
    e1 = over(e_g) + E * over(np.abs(g))
    e2 = over(e_g * np.abs(xh) + np.abs(g) * e_xh) + E * m2
    parts = np.abs(g) + np.abs(over(g)) + np.abs(xh * s2)
    e_dx = wide(r) * (e_g + e1 + np.abs(xh) * e2 + e_xh * np.abs(s2)) + E * wide(r) * (1 + wide(top * r)) * parts
    near(dx, rdx, 1.01 * e_dx + half * np.abs(rdx), "dx")
    return y, stats, dx, dw, db, dz


SHAPES = [
    # B, N, C, G
    (37, 1, 512, 8),           # heads of single tokens
    (5, 1, 1024, 8),
    (3, 1, 96, 3),             # groups of 32
    (9, 1, 1152, 12),          # 96: lanes past the group's end, more slots than threads
    (4, 1, 99, 3),             # 33: no whole pieces
    (2, 1, 2048, 2),           # a group of 1024
    (7, 1, 6, 6),              # groups of one channel (deviation 0)
    (700, 1, 64, 1),
    (3, 1, 4160, 65),          # more slots than a block
    (2, 64, 320, 32),          # groups of 10
    (1, 1000, 64, 8),
    (3, 17, 224, 32),          # groups of 7
    (2, 33, 35, 5),            # odd everything
    (1, 5, 3000, 3),           # groups of 1000, several blocks of channels
    (1, 2, 4096, 16),
    (2, 9, 2100, 300),         # groups of 7 over several blocks of channels
    (2, 4096, 8, 2),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_oracle(la, shape, gate, dt):
    B, N, C, G = shape
    p, dy = problem(B, N, C, dt, B + N + C)
    if not gate:
        p["z"] = None
    check(la, p, G, dy, silu=(C + gate) % 2 == 0, dt=dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N,C,G", [(1, 256, 4), (50, 64, 4)])
def test_without_weights(la, N, C, G, dt):
    p, dy = problem(3, N, C, dt, 5)
    p.update(w=None, b=None)
    out = check(la, p, G, dy, True, dt)
    assert out[3] is None and out[4] is None


@pytest.mark.parametrize("N,C,G", [(1, 512, 8), (300, 40, 4)])
def test_a_large_mean_costs_no_digits(la, N, C, G):
    p, dy = problem(4, N, C, "f32", 9)
    p["x"] += 1000.0
    check(la, p, G, dy, True, "f32")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N,C,G", [(1, 256, 4), (70, 48, 4)])
def test_strided_and_unaligned_rows(la, N, C, G, dt):
    p, dy = problem(6, N, C, dt, 15, lead=3)                 # z not on a 16-byte boundary
    wide = torch.zeros(6, N, 2 * C + 16, device="cuda", dtype=DT[dt])
    wide[..., 8:8 + C] = p["x"]
    p["x"] = wide[..., 8:8 + C]                             # whole pieces
    y = check(la, p, G, dy, True, dt)[0]
    out = torch.full((6, N, C + 8), 3.0, device="cuda").to(DT[dt])
    got = la.la_group_norm_fwd(p["x"], G, p["w"], p["b"], p["z"], True, y=out[..., :C])
    assert torch.equal(got, y) and (out[..., C:] == 3).all()
    # Sequences next to one another within a token.
    q = {k: v for k, v in p.items()}
    q["x"] = p["x"].transpose(0, 1).contiguous().transpose(0, 1)
    check(la, q, G, dy, False, dt)


def test_non_finite_rows_stay_their_own(la):
    p, dy = problem(9, 1, 256, "f32", 21)
    y = la.la_group_norm_fwd(p["x"], 4, p["w"], p["b"], p["z"])
    p["x"][4, 0, 70] = float("nan")
    got = la.la_group_norm_fwd(p["x"], 4, p["w"], p["b"], p["z"])
    assert torch.isnan(got[4, 0, 64:128]).all()
    got[4, 0, 64:128] = y[4, 0, 64:128]
    assert torch.equal(got, y)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_empty_calls(la, dt):
    w = torch.ones(8, device="cuda", dtype=DT[dt])
    for shape in ((0, 4, 8), (3, 0, 8)):
        x = torch.empty(shape, device="cuda", dtype=DT[dt])
        y, s = la.la_group_norm_fwd(x, 2, w, w, return_stats=True)
        assert y.shape == x.shape
        dx, dw, db, dz = la.la_group_norm_bwd(x, 2, x, s, w, w)
        assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all() and dz is None


@pytest.mark.parametrize("N,C,G", [(1, 512, 8), (600, 64, 4)])
def test_streams_graphs_and_repeats(la, N, C, G):
    p, dy = problem(40, N, C, "bf16", 33)
    call = lambda ws, **kw: la.la_group_norm_fwd(p["x"], G, p["w"], p["b"], p["z"], True, return_stats=True, ws=ws, **kw)  # noqa: E731
    back = lambda s, ws, **kw: la.la_group_norm_bwd(p["x"], G, dy, s, p["w"], p["b"], p["z"], True, ws=ws, **kw)  # noqa: E731
    ws = la.group_norm_workspace(40, N, C, G)
    y, s = call(ws)
    g = back(s, ws)
    torch.cuda.synchronize()
    got = []
    for st in [torch.cuda.Stream() for _ in range(2)]:
        st.wait_stream(torch.cuda.current_stream())
        u, t = call(None, stream=st)
        got.append((u, t, *back(t, None, stream=st)))
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, (y, s, *g)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        u, t = call(ws)
        r = back(t, ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((u, t, *r), (y, s, *g)))
