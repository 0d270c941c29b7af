"""Outputs of the token-mixing entries that overlap an input or one another are refused
before any CUDA call (no pointer here is read): ranges of one buffer a few values apart,
rows that share some of their values, an output inside a dense input. Column ranges that
interleave without sharing a value are not overlaps; such calls are refused here by a later
check, or pass (the GPU tests run them)."""
import pytest

F = 1 << 24            # aligned, never dereferenced
FAR = 1 << 24          # between buffers
BAD, WS = 1, 3


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


def at(i):
    return F + i * FAR


def conv(la, **kw):
    """bf16 [2, 40, 64], every tensor far from the others."""
    a = dict(x=at(0), xb=40 * 64, xt=64, w=at(1), bias=at(2), silu=1, lengths=at(3), s0=at(4), s1=at(5), y=at(6),
             yb=40 * 64, yt=64, B=2, N=40, C=64, W=4, dt=1, stream=None)
    a.update(kw)
    return la._lib.la_short_conv_fwd(*a.values())


@pytest.mark.parametrize("kw", [
    dict(y=at(0)), dict(y=at(0) + 2), dict(y=at(0) + 128), dict(y=at(0) - 128), dict(y=at(0) + 2 * 40 * 64 * 2 - 2),
    dict(y=at(1) + 16), dict(y=at(2) - 64), dict(y=at(3)), dict(y=at(4) + 128), dict(y=at(5) + 128),
    dict(s1=at(0) + 256), dict(s1=at(1)), dict(s1=at(2)), dict(s1=at(3)), dict(s1=at(4) + 64),
    # Rows of one buffer of 160 values: x holds 0..63, y 32..95.
    dict(xb=40 * 160, xt=160, yb=40 * 160, yt=160, y=at(0) + 64),
    # y a token later, and a sequence later, in such rows.
    dict(xb=40 * 160, xt=160, yb=40 * 160, yt=160, y=at(0) + 320 + 10),
    dict(B=3, xb=40 * 160, xt=160, yb=40 * 160, yt=160, y=at(0) + 40 * 320 - 64),
    # A dense y inside a strided x, and the other way round.
    dict(xb=40 * 160, xt=160, y=at(0) + 320 * 3 + 100),
    dict(yb=40 * 160, yt=160, y=at(0) - 640),
    # Token-major batches: sequences next to one another within a token.
    dict(xb=64, xt=128, yb=64, yt=128, y=at(0) + 64),
])
def test_convolution_refuses(la, kw):
    assert conv(la, **kw) == BAD


def conv_step(la, **kw):
    a = dict(x=at(0), xb=64, w=at(1), bias=at(2), silu=1, state=at(3), y=at(4), yb=64, B=8, C=64, W=4, dt=1, stream=None)
    a.update(kw)
    return la._lib.la_short_conv_step(*a.values())


@pytest.mark.parametrize("kw", [
    dict(y=at(0) + 16), dict(y=at(0) - 128), dict(y=at(0), yb=80), dict(y=at(1)), dict(y=at(2) + 2),
    dict(y=at(3) + 128), dict(state=at(0)), dict(state=at(1) + 4), dict(state=at(2)),
])
def test_convolution_step_refuses(la, kw):
    assert conv_step(la, **kw) == BAD


def scan(la, **kw):
    """bf16, B=2 N=40 H=2 S=P=64; the workspace stands (far away) and is large enough."""
    a = dict(x=at(0), xb=40 * 128, xt=128, step=at(1), sb=80, st=2, A=at(2), Bm=at(3), bb=40 * 64, bt=64, Cm=at(4),
             cb=40 * 64, ct=64, D=at(5), z=at(6), zb=40 * 128, zt=128, bias=at(7), softplus=1, lengths=at(8), S0=at(9),
             S_out=at(10), y=at(11), yb=40 * 128, yt=128, B=2, H=2, G=1, N=40, S=64, P=64, dt=1, ws=at(12),
             wsb=1 << 23, stream=None)
    a.update(kw)
    return la._lib.la_selective_scan_fwd(*a.values())


@pytest.mark.parametrize("kw", [
    dict(y=at(0)), dict(y=at(0) + 16), dict(y=at(0) - 256), dict(y=at(6) + 256), dict(y=at(1)), dict(y=at(2)),
    dict(y=at(3) + 128), dict(y=at(4) - 16), dict(y=at(5)), dict(y=at(7)), dict(y=at(8)), dict(y=at(9) + 4096),
    dict(y=at(10) + 1024), dict(S_out=at(0)), dict(S_out=at(1)), dict(S_out=at(2)), dict(S_out=at(3) + 64),
    dict(S_out=at(4)), dict(S_out=at(5)), dict(S_out=at(6) + 16), dict(S_out=at(7)), dict(S_out=at(8)),
    dict(S_out=at(9) + 16),
    # x and y as overlapping column ranges of one projection.
    dict(xb=40 * 512, xt=512, yb=40 * 512, yt=512, y=at(0) + 128),
])
def test_scan_refuses(la, kw):
    assert scan(la, **kw) == BAD


def scan_step(la, **kw):
    a = dict(x=at(0), xb=128, step=at(1), sb=2, A=at(2), Bm=at(3), bb=64, Cm=at(4), cb=64, D=at(5), z=at(6), zb=128,
             bias=at(7), softplus=1, S=at(8), y=at(9), yb=128, B=4, H=2, G=1, Sn=64, P=64, dt=1, stream=None)
    a.update(kw)
    return la._lib.la_selective_scan_step(*a.values())


@pytest.mark.parametrize("kw", [
    dict(y=at(0) + 16), dict(y=at(6) + 128), dict(y=at(1)), dict(y=at(2)), dict(y=at(3)), dict(y=at(4) + 64), dict(y=at(5)),
    dict(y=at(7)), dict(y=at(8) + 64), dict(S=at(0)), dict(S=at(1)), dict(S=at(2)), dict(S=at(3)), dict(S=at(4)),
    dict(S=at(5)), dict(S=at(6)), dict(S=at(7)),
])
def test_scan_step_refuses(la, kw):
    assert scan_step(la, **kw) == BAD


def rope_fwd(la, **kw):
    """bf16, B=2 N=40 Hq=4 Hk=2 D=64."""
    a = dict(q=at(0), qb=40 * 256, qt=256, k=at(1), kb=40 * 128, kt=128, wq=at(2), wk=at(3), pos=at(4), axes=1,
             table=at(5), pairs=32, qo=at(6), ko=at(7), B=2, N=40, Hq=4, Hk=2, D=64, dt=1, norm=1, eps=1e-6, layout=0,
             stream=None)
    a.update(kw)
    return la._lib.la_qk_norm_rope_fwd(*a.values())


@pytest.mark.parametrize("kw", [
    dict(qo=at(0)), dict(qo=at(0) + 512), dict(ko=at(0)), dict(ko=at(1) + 2), dict(qo=at(1) - 64), dict(qo=at(2)),
    dict(ko=at(3)), dict(ko=at(4)), dict(qo=at(5)), dict(ko=at(6) + 1024),
    # q and k as column ranges of a projection of 512 values per token, ko in its other columns.
    dict(qb=40 * 512, qt=512, k=at(0) + 512, kb=40 * 512, kt=512, ko=at(0) + 1024 * 3 + 700),
])
def test_rotation_refuses(la, kw):
    assert rope_fwd(la, **kw) == BAD


def rope_bwd(la, **kw):
    a = dict(q=at(0), qb=40 * 256, qt=256, k=at(1), kb=40 * 128, kt=128, wq=at(2), wk=at(3), pos=at(4), axes=1,
             table=at(5), pairs=32, dqo=at(6), dko=at(7), dq=at(8), dqb=40 * 256, dqt=256, dk=at(9), dkb=40 * 128,
             dkt=128, dwq=at(10), dwk=at(11), B=2, N=40, Hq=4, Hk=2, D=64, dt=1, norm=1, eps=1e-6, layout=0, ws=at(12),
             wsb=1 << 23, stream=None)
    a.update(kw)
    return la._lib.la_qk_norm_rope_bwd(*a.values())


@pytest.mark.parametrize("kw", [
    dict(dq=at(6)), dict(dq=at(7) + 64), dict(dk=at(6)), dict(dk=at(7)), dict(dq=at(0) + 512), dict(dq=at(1)),
    dict(dk=at(1) + 2), dict(dk=at(8) + 128), dict(dq=at(2)), dict(dk=at(3)), dict(dq=at(4)), dict(dk=at(5)),
    dict(dq=at(0), dqb=40 * 320, dqt=320),                # q's place with other strides
    # dq and dk as column ranges of one projection gradient that share 32 columns.
    dict(dqb=40 * 512, dqt=512, dk=at(8) + 512 - 64, dkb=40 * 512, dkt=512),
])
def test_rotation_backward_refuses(la, kw):
    assert rope_bwd(la, **kw) == BAD


def test_ranges_that_interleave_are_no_overlap(la):
    # Column ranges side by side, in rows of one buffer: only the missing workspace is refused.
    rows = dict(xb=40 * 512, xt=512, yb=40 * 512, yt=512, ws=None)
    assert scan(la, y=at(0) + 256, **rows) == WS
    assert scan(la, y=at(0) - 256, **rows) == WS
    assert rope_bwd(la, dqb=40 * 512, dqt=512, dk=at(8) + 512, dkb=40 * 512, dkt=512, ws=None) == WS
    assert rope_bwd(la, dq=at(0), ws=None) == WS           # in q's own place


@pytest.mark.gpu
def test_outputs_in_their_inputs_place_and_between_columns(la):
    # What the refusals leave: steps and gradients that replace their own input, and an output
    # in columns of the buffer that holds the inputs, give the bits of separate buffers.
    import torch
    g = torch.Generator(device="cuda").manual_seed(81)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, w, state = r(3, 64), r(64, 4), r(3, 3, 64)
    s1, s2, x2 = state.clone(), state.clone(), x.clone()
    want = la.la_short_conv_step(x, w, s1)
    assert torch.equal(la.la_short_conv_step(x2, w, s2, y=x2), want) and torch.equal(s1, s2)

    xs, Bm, Cm, step, z = r(3, 2, 64), r(3, 1, 64), r(3, 1, 64), r(3, 2), r(3, 2, 64)
    A, S = -torch.ones(2, device="cuda"), torch.randn(3, 2, 64, 64, generator=g, device="cuda")
    want = la.la_selective_scan_step(xs, step, A, Bm, Cm, S.clone(), z=z)
    for place in (xs, z):
        a, b = xs.clone(), z.clone()
        got = la.la_selective_scan_step(a, step, A, Bm, Cm, S.clone(), z=b, y=a if place is xs else b)
        assert torch.equal(got, want)

    buf = r(2, 150, 512)
    x4, y4 = buf[..., :128].unflatten(2, (2, 64)), buf[..., 128:256].unflatten(2, (2, 64))
    B4, C4, d4 = buf[..., 256:320].unflatten(2, (1, 64)), buf[..., 320:384].unflatten(2, (1, 64)), buf[..., 384:386]
    want = la.la_selective_scan_fwd(x4, d4, A, B4, C4)
    assert torch.equal(la.la_selective_scan_fwd(x4, d4, A, B4, C4, y=y4), want)
    want = la.la_short_conv_fwd(buf[..., :64], w)
    assert torch.equal(la.la_short_conv_fwd(buf[..., :64], w, y=buf[..., 448:]), want)

    q, k = r(2, 33, 4, 64), r(2, 33, 2, 64)
    dqo, dko = r(2, 4, 33, 64), r(2, 2, 33, 64)
    pos = torch.arange(33, dtype=torch.int32, device="cuda").repeat(2, 1)
    table = la.la_rope_table([10000.0 ** (-i / 32) for i in range(32)])
    for D in (64, 60):                     # the vector kernels and the row kernel
        t = la.la_rope_table([10000.0 ** (-i / 30) for i in range(30)]) if D == 60 else table
        a, b, go, ko = (v[..., :D].contiguous() for v in (q, k, dqo, dko))
        want = la.la_qk_norm_rope_bwd(a, b, go, ko, pos, t)
        got = la.la_qk_norm_rope_bwd(a, b, go, ko, pos, t, dq=a, dk=b)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
