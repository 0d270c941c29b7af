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
