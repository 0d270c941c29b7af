"""Refusals of the token-mixing entries: every call here fails its checks before
any CUDA call, so no GPU is needed and no pointer is read."""
import ctypes

import pytest
import torch

F = 1 << 20   # aligned, never dereferenced
BAD, UNSUP, WS = 1, 2, 3


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


def rope_fwd(la, **kw):
    a = dict(q=F, qb=0, qt=64, k=F, kb=0, kt=64, wq=F, wk=F, pos=F, axes=1, table=F, pairs=32, qo=F, ko=F,
             B=1, N=4, Hq=1, Hk=1, D=64, dt=1, norm=1, eps=1e-6, layout=0, stream=None)
    a.update(kw)
    return la._lib.la_qk_norm_rope_fwd(*a.values())


def rope_bwd(la, **kw):
    a = dict(q=F, qb=0, qt=64, k=F, kb=0, kt=64, wq=F, wk=F, pos=F, axes=1, table=F, pairs=32, dqo=F, dko=F,
             dq=F, dqb=256, dqt=64, dk=F, dkb=256, dkt=64, dwq=F, dwk=F, B=2, N=4, Hq=1, Hk=1, D=64, dt=1,
             norm=1, eps=1e-6, layout=0, ws=F, wsb=1 << 30, stream=None)
    a.update(kw)
    return la._lib.la_qk_norm_rope_bwd(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), BAD), (dict(ko=None), BAD), (dict(q=F + 1), BAD), (dict(wk=F + 1), BAD),
    (dict(pos=None), BAD), (dict(pos=F + 2), BAD), (dict(table=None), BAD), (dict(table=F + 8), BAD),
    (dict(pairs=33), BAD), (dict(pairs=-1), BAD), (dict(axes=0), BAD), (dict(axes=5), UNSUP),
    (dict(D=0), BAD), (dict(D=129, pairs=4), UNSUP), (dict(dt=2), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=float("nan")), BAD), (dict(layout=2), BAD), (dict(norm=0), BAD), (dict(B=-1), BAD),
    (dict(Hq=65535), UNSUP), (dict(B=1 << 20, N=1 << 20), UNSUP),
])
def test_rope_forward_refuses(la, kw, want):
    assert rope_fwd(la, **kw) == want


def test_rope_empty_calls_touch_nothing(la):
    none = dict(q=None, k=None, wq=None, wk=None, pos=None, table=None, qo=None, ko=None)
    assert rope_fwd(la, B=0, **none) == 0
    assert rope_fwd(la, N=0, **none) == 0
    assert rope_fwd(la, Hq=0, Hk=0, **none) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(dqo=None), BAD), (dict(dk=None), BAD), (dict(q=None), BAD), (dict(dwq=F + 1), BAD),
    (dict(norm=0), BAD), (dict(ws=None), WS), (dict(ws=F + 16), WS), (dict(wsb=512), WS),
    (dict(dqt=32), BAD),                      # rows of one sequence overlap
    (dict(dqb=128), BAD),                     # sequences overlap
    (dict(dkb=32, dkt=64), BAD),
])
def test_rope_backward_refuses(la, kw, want):
    assert rope_bwd(la, **kw) == want


def test_rope_table_values_and_refusals(la):
    import math
    t = la.la_rope_table([2 * math.pi / 4, 0.0, 2 * math.pi * 1.5, -2 * math.pi / 8], [0, 1, 2, 3], device="cpu")
    steps = [int(v) % (1 << 64) for v in t[:, 0]]
    for got, want in zip(steps, (1 << 62, 0, 1 << 63, 7 << 61)):
        assert min((got - want) % (1 << 64), (want - got) % (1 << 64)) <= 1 << 13   # double rounding of 1/2pi
    assert t[:, 1].tolist() == [0, 1, 2, 3]
    for f, ax in (([float("inf")], None), ([1.0], [4]), ([1.0], [-1])):
        with pytest.raises(la.LinAttnError):
            la.la_rope_table(f, ax, device="cpu")
    with pytest.raises(ValueError):
        la.la_rope_table([1.0, 2.0], [0], device="cpu")


def test_rope_workspace_size(la):
    n = la.la_qk_norm_rope_bwd_workspace_size(1, 1, 8, 8, 64)
    assert n % 256 == 0 and n >= 4 * 148 * 2 * 64 * 4
    assert la.la_qk_norm_rope_bwd_workspace_size(1, 1, 3000, 8, 64) >= 3008 * 2 * 64 * 4
    size = ctypes.c_size_t(0)
    assert la._lib.la_qk_norm_rope_bwd_workspace_size(1, 1, 1, 1, 129, ctypes.byref(size)) == UNSUP
    assert la._lib.la_qk_norm_rope_bwd_workspace_size(1, 1, 1, 1, 64, None) == BAD


def test_rope_wrappers_refuse_before_any_launch(la):
    q = torch.zeros(1, 4, 2, 64)
    pos, table = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(32, 2, dtype=torch.int64)
    with pytest.raises(ValueError):                       # host tensors
        la.la_qk_norm_rope_fwd(q, q, pos, table)
    with pytest.raises(ValueError):
        la.la_qk_norm_rope_fwd(None, None, pos, table)
    with pytest.raises(TypeError):
        la.la_qk_norm_rope_fwd(q, q.double(), pos, table)


def conv_fwd(la, **kw):
    a = dict(x=F, xb=1000, xt=64, w=F, bias=F, silu=1, lengths=None, s0=F, s1=F + (1 << 19), y=F + 16, yb=1000,
             yt=64, B=2, N=4, C=64, W=4, dt=1, stream=None)
    a.update(kw)
    return la._lib.la_short_conv_fwd(*a.values())


def conv_step(la, **kw):
    a = dict(x=F, xb=64, w=F, bias=F, silu=1, state=F, y=F, yb=64, B=2, C=64, W=4, dt=1, stream=None)
    a.update(kw)
    return la._lib.la_short_conv_step(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), BAD), (dict(w=None), BAD), (dict(y=None), BAD), (dict(y=F), BAD), (dict(x=F + 1), BAD),
    (dict(bias=F + 1), BAD), (dict(lengths=F + 2), BAD), (dict(s1=F + 64), BAD), (dict(yt=32), BAD),
    (dict(yb=100), BAD), (dict(W=5), UNSUP), (dict(W=1), UNSUP), (dict(W=0), BAD), (dict(C=0), BAD),
    (dict(dt=3), BAD), (dict(N=-1), BAD), (dict(B=1 << 20, N=1 << 20), UNSUP), (dict(B=0, x=None), 0),
])
def test_conv_forward_refuses(la, kw, want):
    assert conv_fwd(la, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(state=None), BAD), (dict(x=None), BAD), (dict(y=F + 1), BAD), (dict(W=8), UNSUP), (dict(yb=63), BAD),
    (dict(C=-1), BAD), (dict(B=0, x=None), 0),
])
def test_conv_step_refuses(la, kw, want):
    assert conv_step(la, **kw) == want


def test_conv_wrappers_refuse_before_any_launch(la):
    x, w = torch.zeros(2, 4, 64), torch.zeros(64, 4)
    with pytest.raises(ValueError):                       # host tensors
        la.la_short_conv_fwd(x, w)
    with pytest.raises(ValueError):
        la.la_short_conv_fwd(x, torch.zeros(32, 4))
    with pytest.raises(TypeError):
        la.la_short_conv_step(torch.zeros(2, 64).half(), w, torch.zeros(2, 3, 64))


def scan_fwd(la, **kw):
    a = dict(x=F, xb=1 << 14, xt=128, step=F, sb=8, st=2, A=F, Bm=F, bb=256, bt=64, Cm=F, cb=256, ct=64, D=F, z=F,
             zb=1 << 14, zt=128, bias=F, softplus=1, lengths=None, S0=F, S_out=F, y=F + 16, yb=512, yt=128, B=2, H=2,
             G=1, N=4, S=64, P=64, dt=1, ws=F, wsb=1 << 30, stream=None)
    a.update(kw)
    return la._lib.la_selective_scan_fwd(*a.values())


def scan_step(la, **kw):
    a = dict(x=F, xb=128, step=F, sb=2, A=F, Bm=F, bb=64, Cm=F, cb=64, D=F, z=F, zb=128, bias=F, softplus=1, S=F, y=F,
             yb=128, B=2, H=2, G=1, Sn=64, P=64, dt=1, stream=None)
    a.update(kw)
    return la._lib.la_selective_scan_step(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), BAD), (dict(A=None), BAD), (dict(Bm=F + 1), BAD), (dict(Cm=None), BAD), (dict(step=None), BAD),
    (dict(y=None), BAD), (dict(y=F), BAD), (dict(z=F + 16), BAD), (dict(S_out=F + 64), BAD), (dict(S0=F + 2), BAD),
    (dict(D=F + 2), BAD), (dict(lengths=F + 1), BAD), (dict(yt=64), BAD), (dict(yb=500), BAD),
    (dict(G=0), BAD), (dict(H=3, G=2), BAD), (dict(S=0), BAD), (dict(P=-1), BAD), (dict(dt=2), BAD),
    (dict(S=129), UNSUP), (dict(P=192), UNSUP), (dict(B=40000), UNSUP), (dict(ws=None), WS), (dict(ws=F + 8), WS),
    (dict(wsb=255), WS), (dict(B=0, x=None), 0), (dict(H=0, x=None), 0), (dict(N=0, x=None, y=None), 0),
])
def test_scan_forward_refuses(la, kw, want):
    assert scan_fwd(la, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(S=None), BAD), (dict(S=F + 4), BAD), (dict(x=None), BAD), (dict(y=F + 1), BAD), (dict(A=None), BAD),
    (dict(yb=100), BAD), (dict(H=3, G=2), BAD), (dict(Sn=200), UNSUP), (dict(B=0, x=None), 0),
])
def test_scan_step_refuses(la, kw, want):
    assert scan_step(la, **kw) == want


def test_scan_workspace_and_launches(la):
    assert la.la_workspace_size(la.LA_OP_SELECTIVE_SCAN, 2, 64, 0, 128, 64, la.LA_BF16) == 256
    assert la.la_workspace_size(la.LA_OP_SELECTIVE_SCAN, 1, 8, 8192, 128, 64, la.LA_BF16) % 256 == 0
    assert la.la_launch_count(la.LA_OP_SELECTIVE_SCAN, 1, 8, 0, 128, 64, la.LA_BF16) == 0
    for N in (1, 60):                                     # too short to be cut into segments
        assert la.la_launch_count(la.LA_OP_SELECTIVE_SCAN, 1, 1, N, 64, 64, la.LA_F32) == 1
    with pytest.raises(la.LinAttnError):
        la.la_workspace_size(la.LA_OP_SELECTIVE_SCAN, 1, 8, 64, 129, 64, la.LA_BF16)


def test_scan_wrappers_refuse_before_any_launch(la):
    x, step, A = torch.zeros(2, 4, 2, 64), torch.zeros(2, 4, 2), -torch.ones(2)
    Bm = torch.zeros(2, 4, 1, 64)
    with pytest.raises(ValueError):                       # host tensors
        la.la_selective_scan_fwd(x, step, A, Bm, Bm)
    with pytest.raises(ValueError):
        la.la_selective_scan_fwd(x, step[:, :3], A, Bm, Bm)
    with pytest.raises(TypeError):
        la.la_selective_scan_fwd(x, step.bfloat16(), A, Bm, Bm)
    with pytest.raises(ValueError):
        la.la_selective_scan_step(x[:, 0], step[:, 0], A, Bm[:, 0], Bm[:, 0], None)


def test_sequences_whose_roundings_pass_an_int(la):
    far = (1 << 30) + 1
    assert conv_fwd(la, B=1, N=far) == UNSUP
    assert conv_fwd(la, B=1, N=2147483647, C=1) == UNSUP
    for N in (far, 2147483647):
        assert scan_fwd(la, B=1, N=N) == UNSUP
        for dt in (la.LA_F32, la.LA_BF16):
            with pytest.raises(la.LinAttnError):
                la.la_workspace_size(la.LA_OP_SELECTIVE_SCAN, 1, 2, N, 64, 64, dt)
            with pytest.raises(la.LinAttnError):
                la.la_launch_count(la.LA_OP_SELECTIVE_SCAN, 1, 2, N, 64, 64, dt)
