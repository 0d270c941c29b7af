"""la_qk_norm_rope_fwd / _bwd against the float64 oracle (oracle/token_mixing.py).

Tolerances, relative to the row's largest output magnitude. The arithmetic is
fp32 from exact inputs and exactly reduced angles: about 20 fp32 roundings per
value plus a 7-step sum in the norm, far below 32 * 2^-24 (+ 2^-22 for sincospi
and its argument) = 2.2e-6; bf16 outputs add half a step, 2^-8. A value can
reach sqrt(2) times what it is made of and cancel, which the row maximum
absorbs. The weight gradients are sums of up to n rows: fp32 sums in a tree of
partials, bounded by (rows per thread + 32) * 2^-24 of the sum of magnitudes;
the tests have fewer than 2^7 rows per thread.
"""
import numpy as np
import pytest
import torch

from oracle import token_mixing as tm
from workloads import to_f64

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": 2.5e-6, "bf16": 2.0 ** -8 + 2.5e-6}


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


def problem(B, N, Hq, Hk, D, R, axes, dt, seed, far=0, lead=0):
    """q, k as column ranges of one projection (lead: columns before q), positions, frequencies."""
    g = torch.Generator().manual_seed(seed)
    proj = torch.randn(B, N, lead + (Hq + 2 * Hk) * D, generator=g).to(DT[dt]).cuda()
    q = proj[:, :, lead:lead + Hq * D].unflatten(2, (Hq, D))
    k = proj[:, :, lead + Hq * D:lead + (Hq + Hk) * D].unflatten(2, (Hk, D))
    pos = torch.randint(-far - 3, far + 2000, (B, N, axes), generator=g, dtype=torch.int32)
    f = [10000.0 ** (-i / max(R, 1)) for i in range(R)]
    ax = [i % axes for i in range(R)]
    wq, wk = (1 + 0.3 * torch.randn(2, D, generator=g)).to(DT[dt]).cuda()
    return q, k, pos, f, ax, wq, wk, g


def close(got, ref, tol):
    ref = np.asarray(ref)
    scale = np.maximum(np.abs(ref).max(-1, keepdims=True), 1e-30)
    err = np.abs(to_f64(got) - ref) / scale
    assert err.max(initial=0.0) <= tol, err.max()


SHAPES = [
    # B, N, Hq, Hk, D, R, axes, far, lead
    (2, 33, 4, 2, 64, 32, 1, 0, 0),
    (1, 1, 1, 1, 64, 32, 1, 2 ** 30, 0),          # one row, far position
    (3, 1, 8, 8, 64, 24, 1, 0, 8),                # single tokens, part of the head
    (2, 70, 3, 1, 128, 64, 3, 0, 0),
    (1, 50, 2, 2, 96, 36, 2, 0, 0),               # R a multiple of 4 only, 12 lanes of 16
    (2, 17, 2, 1, 32, 12, 4, 0, 0),
    (2, 9, 2, 3, 64, 30, 1, 0, 0),                # R not a multiple of 4: row kernel
    (2, 9, 2, 1, 20, 10, 2, 0, 0),                # D not a multiple of 8
    (1, 7, 1, 2, 64, 32, 1, 0, 3),                # rows not 16-byte aligned
    (2, 5, 2, 2, 1, 0, 1, 0, 0),                  # nothing to rotate
    (1, 1500, 1, 1, 8, 4, 1, 10 ** 6, 0),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward_match_oracle(la, shape, norm, inter, dt):
    B, N, Hq, Hk, D, R, axes, far, lead = shape
    q, k, pos, f, ax, wq, wk, g = problem(B, N, Hq, Hk, D, R, axes, dt, 7 * N + D, far, lead)
    wq, wk = (wq, wk) if norm else (None, None)
    table = la.la_rope_table(f, ax)
    how = dict(wq=wq, wk=wk, norm=norm, interleaved=inter)
    qo, ko = la.la_qk_norm_rope_fwd(q, k, pos.cuda(), table, **how)
    dqo, dko = torch.randn_like(qo), torch.randn_like(ko)
    # Gradients land in column ranges of one projection gradient; what lies between stays.
    dproj = torch.full((B, N, lead + (Hq + 2 * Hk) * D), 7.0, dtype=q.dtype, device="cuda")
    dq = dproj[:, :, lead:lead + Hq * D].unflatten(2, (Hq, D))
    dk = dproj[:, :, lead + Hq * D:lead + (Hq + Hk) * D].unflatten(2, (Hk, D))
    got = la.la_qk_norm_rope_bwd(q, k, dqo, dko, pos.cuda(), table, dq=dq, dk=dk, **how)
    torch.cuda.synchronize()
    p = pos.numpy()
    for out, x, w, go, dx, dw in ((qo, q, wq, dqo, got[0], got[2]), (ko, k, wk, dko, got[1], got[3])):
        x64, w64 = to_f64(x), to_f64(w) if norm else None
        close(out, tm.norm_rope(x64, w64, p, f, ax, norm, 1e-6, inter), TOL[dt])
        rx, rw = tm.norm_rope_bwd(x64, w64, to_f64(go), p, f, ax, norm, 1e-6, inter)
        # dx is a difference of two terms, each up to |g| |w| r sqrt(D) in the worst case:
        # compare with the larger of them.
        if norm:
            r = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + 1e-6)
            size = np.maximum(np.abs(rx).max(-1, keepdims=True),
                              r * np.abs(to_f64(go)).max(-1).transpose(0, 2, 1)[..., None] * np.abs(w64).max())
        else:
            size = np.maximum(np.abs(rx).max(-1, keepdims=True), 1e-30)
        assert (np.abs(to_f64(dx) - rx) / size).max() <= 2 * TOL[dt]
        if norm:
            g64 = np.abs(to_f64(go)).transpose(0, 2, 1, 3)
            mag = (np.abs(x64) * g64.max(-1, keepdims=True) / np.sqrt((x64 ** 2).mean(-1, keepdims=True))).sum((0, 1, 2))
            assert (np.abs(to_f64(dw) - rw) <= 2 * 160 * 2.0 ** -24 * mag).all()
        else:
            assert dw is None
    assert (dproj[:, :, :lead] == 7).all() and (dproj[:, :, lead + (Hq + Hk) * D:] == 7).all()


def test_far_positions_lose_nothing(la):
    # The rotation at p and at p + 2^31 - 2^20 differs from the oracle by fp32 rounding only.
    f = [1.0, 0.7, 1e-3, 1e-5]
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 999999937]], dtype=torch.int32)
    x = torch.randn(1, 4, 1, 8, device="cuda")
    qo, _ = la.la_qk_norm_rope_fwd(x, None, pos.cuda(), la.la_rope_table(f), norm=False)
    close(qo, tm.norm_rope(to_f64(x), None, pos.numpy()[..., None], f, [0] * 4, False), TOL["f32"])


def test_zero_rows_and_infinite_rows_stay_apart(la):
    # A zero row has norm sqrt(eps): output and gradient stay finite. A row of NaN and one
    # of infinities change no other row.
    q, k, pos, f, ax, wq, wk, _ = problem(1, 6, 2, 2, 64, 32, 1, "bf16", 5)
    q = q.clone()
    q[0, 1] = 0
    table = la.la_rope_table(f, ax)
    ref, _ = la.la_qk_norm_rope_fwd(q, k, pos.cuda(), table, wq, wk)
    assert torch.isfinite(ref).all()
    q[0, 3], q[0, 4] = float("nan"), float("inf")
    out, _ = la.la_qk_norm_rope_fwd(q, k, pos.cuda(), table, wq, wk)
    keep = [0, 1, 2, 5]
    assert torch.equal(out[:, :, keep], ref[:, :, keep]) and out[:, :, 3].isnan().all()


def test_one_side_only_and_empty(la):
    q, k, pos, f, ax, wq, wk, _ = problem(2, 5, 4, 2, 64, 32, 1, "bf16", 6)
    table = la.la_rope_table(f, ax)
    both = la.la_qk_norm_rope_fwd(q, k, pos.cuda(), table, wq, wk)
    assert torch.equal(la.la_qk_norm_rope_fwd(q, None, pos.cuda(), table, wq)[0], both[0])
    assert torch.equal(la.la_qk_norm_rope_fwd(None, k, pos.cuda(), table, None, wk)[1], both[1])
    e = q[:, :0]
    out = la.la_qk_norm_rope_fwd(e, None, pos[:, :0].contiguous().cuda(), table, wq)[0]
    assert out.shape == (2, 4, 0, 64)
    g = la.la_qk_norm_rope_bwd(e, None, out, None, pos[:, :0].contiguous().cuda(), table, wq)
    assert (g[2] == 0).all()


def test_same_bits_twice_on_another_stream_and_in_a_graph(la):
    q, k, pos, f, ax, wq, wk, _ = problem(2, 300, 4, 2, 64, 32, 1, "bf16", 8)
    table, pos = la.la_rope_table(f, ax), pos.cuda()
    run = lambda **kw: la.la_qk_norm_rope_bwd(q, k, qo, ko, pos, table, wq, wk, **kw)  # noqa: E731
    qo, ko = la.la_qk_norm_rope_fwd(q, k, pos, table, wq, wk)
    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    ws = la.qk_norm_rope_workspace(2, 300, 4, 2, 64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run(ws=ws)
    ws.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, other, captured):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_autograd_feeds_linear_attention(la):
    # Projection -> norm and rotation -> causal linear attention, differentiated end to
    # end: the projection's gradient equals the chain of the library's own entries.
    from linear_attention_elu_gb300.autograd import linear_attention, qk_norm_rope
    B, N, H, D = 2, 130, 2, 64
    g = torch.Generator().manual_seed(3)
    proj = torch.randn(B, N, 3 * H * D, generator=g).cuda().requires_grad_()
    wq, wk = (torch.ones(D, device="cuda", requires_grad=True) for _ in range(2))
    table = la.la_rope_table([10000.0 ** (-i / 32) for i in range(32)])
    pos = torch.arange(N, dtype=torch.int32, device="cuda").expand(B, N).contiguous()
    q, k, v = (t.unflatten(2, (H, D)) for t in proj.split(H * D, 2))
    qo, ko = qk_norm_rope(q, k, pos, table, wq, wk)
    o = linear_attention(qo, ko, v.transpose(1, 2))
    do = torch.randn(o.shape, generator=g).cuda()
    o.backward(do)
    with torch.no_grad():
        dqo, dko, dv = la.la_causal_bwd(qo.detach(), ko.detach(), v.transpose(1, 2).contiguous(), do)
        dq, dk, dwq, dwk = la.la_qk_norm_rope_bwd(q, k, dqo, dko, pos, table, wq, wk)
    ref = torch.cat((dq.flatten(2), dk.flatten(2), dv.transpose(1, 2).flatten(2)), 2)
    # The fp32 backward of the attention adds in an order of its own per call at most.
    assert torch.allclose(proj.grad, ref, rtol=1e-4, atol=1e-5)
    assert torch.allclose(wq.grad, dwq, rtol=1e-4, atol=1e-4)
    assert torch.allclose(wk.grad, dwk, rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("given", ["q", "k", "unused"])
def test_autograd_of_one_side(la, given):
    # One side alone, and both with only one output used.
    from linear_attention_elu_gb300.autograd import qk_norm_rope
    q, k, pos, f, ax, wq, wk, _ = problem(2, 9, 4, 2, 64, 32, 1, "f32", 9)
    table, pos = la.la_rope_table(f, ax), pos.cuda()
    q, k, wq, wk = (t.clone().requires_grad_() for t in (q, k, wq, wk))
    if given == "q":
        qo, ko = qk_norm_rope(q, None, pos, table, wq)
        assert ko is None
    elif given == "k":
        qo, ko = qk_norm_rope(None, k, pos, table, None, wk)
        assert qo is None
    else:
        qo, ko = qk_norm_rope(q, k, pos, table, wq, wk)
    out, x, w = (ko, k, wk) if given == "k" else (qo, q, wq)
    go = torch.randn_like(out)
    out.backward(go)
    rx, rw = tm.norm_rope_bwd(to_f64(x), to_f64(w), to_f64(go), pos.cpu().numpy(), f, ax)
    assert np.allclose(to_f64(x.grad), rx, rtol=0, atol=2.0 ** -18 * np.abs(rx).max())
    assert np.allclose(to_f64(w.grad), rw, rtol=0, atol=2.0 ** -16 * np.abs(rw).max())
    if given == "unused":
        assert (k.grad == 0).all() and (wk.grad == 0).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
def test_backward_of_many_tokens(la, dt, inter):
    # More token tiles than blocks, so that a block walks several: rows equal those of pieces
    # bit for bit; the weight gradients are the pieces' sums. Either is an fp32 sum of the same
    # terms in a tree of fewer than 2^7 additions deep, the pieces' five sums add five more.
    B, N, D, step = 1, 60001, 32, 12000
    q, k, pos, f, ax, wq, wk, g = problem(B, N, 2, 1, D, 12, 2, dt, 5)
    table, pos = la.la_rope_table(f, ax), pos.cuda()
    how = dict(wq=wq, wk=wk, interleaved=inter)
    qo, ko = la.la_qk_norm_rope_fwd(q, k, pos, table, **how)
    dqo, dko = torch.randn_like(qo), torch.randn_like(ko)
    dq, dk, dwq, dwk = la.la_qk_norm_rope_bwd(q, k, dqo, dko, pos, table, **how)
    sums = [torch.zeros(D, device="cuda", dtype=torch.float64) for _ in range(2)]
    for t in range(0, N, step):
        s = slice(t, min(t + step, N))
        part = (q[:, s], k[:, s], pos[:, s].contiguous(), table)
        po, ro = la.la_qk_norm_rope_fwd(*part, **how)
        assert torch.equal(po, qo[:, :, s]) and torch.equal(ro, ko[:, :, s])
        pq, pk, pwq, pwk = la.la_qk_norm_rope_bwd(*part[:2], dqo[:, :, s].contiguous(), dko[:, :, s].contiguous(),
                                                  *part[2:], **how)
        assert torch.equal(pq, dq[:, s]) and torch.equal(pk, dk[:, s])
        sums[0] += pwq
        sums[1] += pwk
    for x, do, dw, want in ((q, dqo, dwq, sums[0]), (k, dko, dwk, sums[1])):
        r = torch.rsqrt(x.double().square().mean(-1, keepdim=True) + 1e-6)
        # |g| of a pair is at most the two gradients' magnitudes together.
        size = (do.double().abs().amax(-1).transpose(1, 2)[..., None] * 2 * (x.double() * r).abs()).sum((0, 1, 2))
        assert ((dw - want).abs() <= 2 * 128 * 2.0 ** -24 * size).all()
