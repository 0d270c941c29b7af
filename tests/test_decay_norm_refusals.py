"""Refusals of the decayed attention and of the group norm: every call here fails its checks
before any CUDA call, so no GPU is needed and no pointer is read."""
import ctypes

import pytest
import torch

F, FAR = 1 << 24, 1 << 24        # aligned, never dereferenced; between buffers
BAD, UNSUP, WS = 1, 2, 3


def at(i):
    return F + i * FAR


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


def strides(*v):
    return (ctypes.c_int64 * len(v))(*v)


HEAD = (2 * 40 * 64, 40 * 64, 64)                # [2, 2, 40, 64] head-major
TOK = (40 * 512, 64, 512)                        # column ranges of rows of 512


def fwd(la, q=at(0), k=at(1), v=at(2), decay=at(3), scale=1.0, lengths=at(4), S0=at(5), S1=at(6), o=at(7), st=HEAD * 4, B=2,
        H=2, N=40, Dk=64, Dv=64, dt=1, ws=at(8), wsb=1 << 23):
    return la._lib.la_decay_attn_fwd(q, k, v, decay, scale, lengths, S0, S1, o, strides(*st) if st else None, B, H, N, Dk, Dv,
                                     dt, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), BAD), (dict(k=at(1) + 1), BAD), (dict(v=None), BAD), (dict(decay=None), BAD), (dict(decay=at(3) + 2), BAD),
    (dict(lengths=at(4) + 1), BAD), (dict(S0=at(5) + 2), BAD), (dict(o=None), BAD), (dict(st=None), BAD), (dict(dt=2), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(B=-1), BAD), (dict(N=-1), BAD), (dict(Dk=0), BAD),
    (dict(Dv=-3), BAD), (dict(Dk=129), UNSUP), (dict(Dv=256), UNSUP), (dict(H=65536), UNSUP), (dict(B=300, H=300), UNSUP),
    (dict(N=(1 << 30) + 1), UNSUP), (dict(ws=None), WS), (dict(ws=at(8) + 16), WS), (dict(wsb=255), WS),
    (dict(S1=at(5) + 64), BAD),                          # S_out across S0
    (dict(B=0, q=None), 0), (dict(H=0, q=None), 0), (dict(N=0, q=None, o=None, S0=None, S1=None), 0),
    # Output rows that share values.
    (dict(st=HEAD * 3 + (HEAD[0], HEAD[1], 32)), BAD), (dict(st=HEAD * 3 + (HEAD[0], HEAD[1] - 8, 64)), BAD),
    (dict(st=HEAD * 3 + (HEAD[1], HEAD[1], 64)), BAD), (dict(st=HEAD * 3 + (HEAD[0], 0, 64)), BAD),
    (dict(st=HEAD * 3 + (-HEAD[0], HEAD[1], 64)), BAD),
    # Outputs on inputs.
    (dict(o=at(0)), BAD), (dict(o=at(1) + 128), BAD), (dict(o=at(2) - 64), BAD), (dict(o=at(3)), BAD), (dict(o=at(4)), BAD),
    (dict(o=at(5) + 64), BAD), (dict(o=at(6)), BAD), (dict(o=at(8) + 128), BAD), (dict(S1=at(0)), BAD), (dict(S1=at(1)), BAD),
    (dict(S1=at(3)), BAD), (dict(S1=at(8)), BAD), (dict(ws=at(0)), BAD), (dict(ws=at(5)), BAD),
    (dict(st=TOK * 4, o=at(0) + 64), BAD), (dict(st=TOK * 4, o=at(0) + 1024), BAD),
    (dict(st=(TOK[0], 64, 512) * 3 + (64 * 4, 64 * 8, 40 * 512), o=at(0)), BAD),
])
def test_forward_refuses(la, kw, want):
    assert fwd(la, **kw) == want


def bwd(la, q=at(0), k=at(1), v=at(2), g=at(3), decay=at(4), scale=1.0, lengths=at(5), dq=at(6), dk=at(7), dv=at(8),
        st=HEAD * 7, B=2, H=2, N=40, Dk=64, Dv=64, dt=1, ws=at(9), wsb=1 << 23):
    return la._lib.la_decay_attn_bwd(q, k, v, g, decay, scale, lengths, dq, dk, dv, strides(*st) if st else None, B, H, N, Dk,
                                     Dv, dt, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), BAD), (dict(g=None), BAD), (dict(dv=None), BAD), (dict(dk=at(7) + 1), BAD), (dict(decay=None), BAD),
    (dict(st=None), BAD), (dict(lengths=at(5) + 2), BAD), (dict(scale=float("nan")), BAD), (dict(Dk=200), UNSUP),
    (dict(ws=None), WS), (dict(wsb=0), WS), (dict(B=0, q=None), 0), (dict(N=0, q=None), 0),
    (dict(st=HEAD * 5 + (HEAD[0], HEAD[1], 63) + HEAD), BAD), (dict(st=HEAD * 6 + (HEAD[0], 0, 64)), BAD),
    (dict(dq=at(0)), BAD), (dict(dq=at(3)), BAD), (dict(dk=at(6)), BAD), (dict(dv=at(7) + 64), BAD), (dict(dv=at(6) - 2), BAD),
    (dict(dk=at(4)), BAD), (dict(dv=at(9) + 128), BAD), (dict(ws=at(2)), BAD),
])
def test_backward_refuses(la, kw, want):
    assert bwd(la, **kw) == want


def step(la, q=at(0), k=at(1), v=at(2), decay=at(3), scale=1.0, S=at(4), o=at(5), st=(128, 64) * 4, B=2, H=2, Dk=64, Dv=64,
         dt=1):
    return la._lib.la_decay_attn_step(q, k, v, decay, scale, S, o, strides(*st) if st else None, B, H, Dk, Dv, dt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), BAD), (dict(v=at(2) + 1), BAD), (dict(S=None), BAD), (dict(S=at(4) + 4), BAD), (dict(decay=None), BAD),
    (dict(o=None), BAD), (dict(st=None), BAD), (dict(Dk=0), BAD), (dict(Dv=129), UNSUP), (dict(dt=5), BAD),
    (dict(scale=float("-inf")), BAD), (dict(o=at(0) + 64), BAD), (dict(o=at(4)), BAD), (dict(S=at(0)), BAD), (dict(S=at(3)), BAD),
    (dict(st=(128, 64) * 3 + (128, 32)), BAD), (dict(st=(128, 64) * 3 + (64, 64)), BAD), (dict(B=0, q=None), 0),
    (dict(B=1 << 16, H=1 << 16), UNSUP),
])
def test_step_refuses(la, kw, want):
    assert step(la, **kw) == want


def test_workspace_and_launches(la):
    for op, most in ((la.LA_OP_DECAY_ATTN, 3), (la.LA_OP_DECAY_ATTN_BWD, 9)):
        for dt in (la.LA_F32, la.LA_BF16):
            assert la.la_workspace_size(op, 2, 8, 0, 64, 64, dt) == 256
            assert la.la_workspace_size(op, 1, 2, 9000, 64, 128, dt) % 256 == 0
            assert la.la_launch_count(op, 2, 8, 0, 64, 64, dt) == 0
            # (On the tensor cores dk and dv of heads up to 64 wide come from one launch.)
            assert la.la_launch_count(op, 2, 8, 1, 64, 64, dt) == most // 3
            assert la.la_launch_count(op, 20, 8, 100, 64, 64, dt) >= most // 3 - (most == 9 and dt == la.LA_BF16)
            assert la.la_launch_count(op, 2, 8, 1, 128, 128, dt) == most // 3
            assert la.la_launch_count(op, 1, 1, 9000, 64, 64, dt) <= most
            for bad in ((1, 1, 10, 129, 64), (1, 1, (1 << 30) + 1, 64, 64), (70000, 1, 4, 64, 64)):
                with pytest.raises(la.LinAttnError):
                    la.la_workspace_size(op, *bad, dt)


def test_decay_wrappers_refuse_before_any_launch(la):
    q, decay = torch.zeros(2, 3, 4, 64), -torch.ones(3)
    with pytest.raises(ValueError):                       # host tensors
        la.la_decay_attn_fwd(q, q, q, decay)
    with pytest.raises(ValueError):
        la.la_decay_attn_fwd(q, q[:, :, :3], q, decay)
    with pytest.raises(ValueError):
        la.la_decay_attn_fwd(q, q, q[0], decay)
    with pytest.raises(TypeError):
        la.la_decay_attn_bwd(q, q.bfloat16(), q, q, decay)
    with pytest.raises(TypeError):
        la.la_decay_attn_step(q[:, :, 0].half(), q[:, :, 0].half(), q[:, :, 0].half(), decay, None)


def norm(la, x=at(0), xb=40 * 64, xt=64, w=at(1), b=at(2), z=at(3), zb=40 * 64, zt=64, y=at(4), yb=40 * 64, yt=64, stats=at(5),
         B=2, N=40, C=64, G=4, dt=1, silu=1, eps=1e-5, ws=at(6), wsb=1 << 23):
    return la._lib.la_group_norm_fwd(x, xb, xt, w, b, z, zb, zt, y, yb, yt, stats, B, N, C, G, dt, silu, eps, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), BAD), (dict(y=None), BAD), (dict(x=at(0) + 1), BAD), (dict(w=at(1) + 1), BAD), (dict(z=at(3) + 1), BAD),
    (dict(stats=at(5) + 4), BAD), (dict(C=65), BAD), (dict(G=0), BAD), (dict(C=0), BAD), (dict(B=-1), BAD), (dict(dt=2), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(G=1, C=1025), UNSUP), (dict(B=1 << 20, N=1 << 20), UNSUP),
    (dict(ws=None), WS), (dict(ws=at(6) + 8), WS), (dict(wsb=16), WS), (dict(yt=32), BAD), (dict(yb=100), BAD),
    (dict(y=at(0)), BAD), (dict(y=at(0) + 64), BAD), (dict(y=at(3)), BAD), (dict(y=at(1)), BAD), (dict(y=at(5)), BAD),
    (dict(y=at(6) + 256), BAD), (dict(stats=at(0)), BAD), (dict(stats=at(6)), BAD), (dict(ws=at(2)), BAD),
    (dict(N=1, C=129, G=1, xb=129, zb=129, yb=129), UNSUP), (dict(N=1, C=256, G=1, xb=260, zb=256, yb=256), UNSUP),
    (dict(N=1, C=256, G=1, xb=256, zb=256, yb=256, z=at(3) + 2), UNSUP), (dict(B=0, x=None), 0), (dict(N=0, x=None), 0),
])
def test_norm_refuses(la, kw, want):
    assert norm(la, **kw) == want


def norm_bwd(la, x=at(0), w=at(1), b=at(2), z=at(3), dy=at(4), stats=at(5), dx=at(6), dxb=40 * 64, dxt=64, dz=at(7), dzb=40 * 64,
             dzt=64, dw=at(8), db=at(9), B=2, N=40, C=64, G=4, dt=1, silu=1, ws=at(10), wsb=1 << 23):
    return la._lib.la_group_norm_bwd(x, 40 * 64, 64, w, b, z, 40 * 64, 64, dy, 40 * 64, 64, stats, dx, dxb, dxt, dz, dzb, dzt, dw,
                                     db, B, N, C, G, dt, silu, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), BAD), (dict(dy=None), BAD), (dict(dx=None), BAD), (dict(stats=None), BAD), (dict(dz=None), BAD),
    (dict(z=None), BAD), (dict(dw=at(8) + 2), BAD), (dict(dy=at(4) + 1), BAD), (dict(dxt=63), BAD), (dict(dzb=64), BAD),
    (dict(G=3), BAD), (dict(ws=None), WS), (dict(wsb=100), WS), (dict(dx=at(0)), BAD), (dict(dx=at(4) + 2), BAD),
    (dict(dz=at(3)), BAD), (dict(dz=at(6) + 128), BAD), (dict(dw=at(1)), BAD), (dict(db=at(8) + 4), BAD), (dict(dw=at(5)), BAD),
    (dict(dx=at(10)), BAD), (dict(db=at(10) + 64), BAD), (dict(ws=at(3)), BAD),
])
def test_norm_backward_refuses(la, kw, want):
    assert norm_bwd(la, **kw) == want


def test_norm_workspace(la):
    assert la.la_group_norm_workspace_size(0, 4, 64, 4) == 0
    for N in (1, 40):
        n = la.la_group_norm_workspace_size(2, N, 64, 4)
        assert n > 0 and n % 256 == 0
    size = ctypes.c_size_t(0)
    assert la._lib.la_group_norm_workspace_size(1, 1, 64, 5, ctypes.byref(size)) == BAD
    assert la._lib.la_group_norm_workspace_size(1, 1, 64, 4, None) == BAD


def test_norm_wrappers_refuse_before_any_launch(la):
    x = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError):                       # host tensors
        la.la_group_norm_fwd(x, 4)
    for groups in (0, 5):
        with pytest.raises(ValueError):
            la.la_group_norm_fwd(x, groups)
    with pytest.raises(TypeError):
        la.la_group_norm_fwd(x.half(), 4)
