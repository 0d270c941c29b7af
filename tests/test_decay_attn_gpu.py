"""la_decay_attn_fwd / _bwd / _step against the float64 oracle (oracle/token_mixing.py).

Tolerances, per element, from the sum of magnitudes `mag` of the terms that make it (the
oracle run on absolute values). fp32: a term passes a product sum of Dk and one of 64 terms,
a weight off by a few 2^-22 (its hardware exponential) or, per chunk of 64 or 128 tokens that
it is carried over, two roundings and a product sum of the chunk:
(Dk + N / 16 + 192) 2^-24 mag. bf16 inputs are exact; the tensor-core path rounds the weighted
scores and the state where it is read to bf16, half a step (2^-8) of each term, what a token
adds to a state that is only read to two terms (2^-16 of it is left), to a state that is
returned to three (2^-24); the output is rounded once more (2^-8).
"""
import numpy as np
import pytest
import torch

from oracle import token_mixing as tm
from workloads import to_f64

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def la():
    import linear_attention_elu_gb300 as m
    return m


def problem(B, H, N, Dk, Dv, dt, seed, layout="tok", lead=0):
    """q, k, v and dout [B,H,N,D]: column ranges of a projection, or head-major tensors."""
    g = torch.Generator().manual_seed(seed)
    proj = torch.randn(B, N, lead + H * (2 * Dk + 2 * Dv), generator=g).to(DT[dt]).cuda()
    out, at = [], lead
    for D in (Dk, Dk, Dv, Dv):
        t = proj[..., at:at + H * D].unflatten(2, (H, D)).transpose(1, 2)
        out.append(t if layout == "tok" else t.contiguous())
        at += H * D
    decay = -torch.exp2(-8 * torch.rand(H, generator=g)).cuda()
    S0 = torch.randn(B, H, Dk, Dv, generator=g).cuda()
    return out, decay, S0


def limits(N, Dk, dt, ref, mag):
    f = (Dk + N / 16 + 192) * 2.0 ** -24
    return f * mag if dt == "f32" else (2.0 ** -8 + 2.0 ** -15 + f) * 1.01 * mag + 2.0 ** -8 * np.abs(ref)


def near(got, ref, tol, what):
    err = np.abs(to_f64(got) - ref)
    assert np.isfinite(err).all() and (err <= tol + 1e-30).all(), (what, (err - tol).max(), (err / (tol + 1e-30)).max())


def check_fwd(la, x, decay, S0, dt, scale=0.125, lengths=None, **kw):
    q, k, v = x[:3]
    B, H, N, Dk = q.shape
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    S = torch.full((B, H, Dk, v.shape[3]), float("nan"), device="cuda")
    ws = la.workspace(la.LA_OP_DECAY_ATTN, B, H, N, Dk, v.shape[3], q.dtype)
    o = la.la_decay_attn_fwd(q, k, v, decay, scale, n, S0, S, ws=ws, **kw)
    torch.cuda.synchronize()
    assert la.la_query_status(ws) == 0
    a = [to_f64(t) for t in (q, k, v)]
    s0 = None if S0 is None else to_f64(S0)
    ro, rS = tm.decay_attn(*a, to_f64(decay), scale, lengths, s0)
    mo, mS = tm.decay_attn(*map(np.abs, a), to_f64(decay), scale, lengths, None if s0 is None else np.abs(s0))
    near(o, ro, limits(N, Dk, dt, ro, mo), "o")
    near(S, rS, (Dk + N / 16 + 192) * 2.0 ** -24 * mS, "S")
    # Without a state to return, the same outputs to their own tolerance.
    o2 = la.la_decay_attn_fwd(q, k, v, decay, scale, n, S0, None, ws=ws, **kw)
    near(o2, ro, limits(N, Dk, dt, ro, mo), "o without S_out")
    return o


def check_bwd(la, x, decay, dt, scale=0.125, lengths=None, grads=(None, None, None)):
    q, k, v, do = x
    B, H, N, Dk = q.shape
    Dv = v.shape[3]
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    ws = la.workspace(la.LA_OP_DECAY_ATTN_BWD, B, H, N, Dk, Dv, q.dtype)
    got = la.la_decay_attn_bwd(q, k, v, do, decay, scale, n, *grads, ws=ws)
    torch.cuda.synchronize()
    assert la.la_query_status(ws) == 0
    a = [to_f64(t) for t in x]
    ref = tm.decay_attn_bwd(*a, to_f64(decay), scale, lengths)
    mag = tm.decay_attn_bwd(*map(np.abs, a), to_f64(decay), scale, lengths)
    for g, r, m, D, what in zip(got, ref, mag, (Dv, Dv, Dk), ("dq", "dk", "dv")):
        near(g, r, limits(N, D, dt, r, m), what)
    return got


SHAPES = [
    # B, H, N, Dk, Dv, layout, lead
    (2, 3, 40, 64, 64, "tok", 0),
    (1, 2, 1, 64, 128, "head", 0),       # one token
    (2, 2, 129, 128, 64, "tok", 0),      # one token past a chunk
    (1, 2, 1100, 64, 64, "head", 0),     # segments
    (1, 1, 900, 128, 128, "tok", 0),
    (2, 2, 130, 80, 48, "tok", 0),       # widths of whole 16-byte pieces
    (2, 3, 65, 33, 20, "tok", 0),        # neither
    (1, 2, 128, 64, 64, "tok", 3),       # rows not 16-byte aligned
    (1, 1, 300, 1, 1, "head", 0),
    (3, 5, 257, 8, 8, "tok", 0),
    (1, 1, 64, 65, 66, "head", 0),
    (2, 70, 5, 128, 8, "tok", 0),
    (1, 1, 1300, 64, 128, "tok", 0),     # segments of every pair of widths
    (1, 1, 1300, 128, 64, "head", 0),
    (1, 2, 1500, 24, 56, "tok", 0),
    (1, 1, 4100, 64, 64, "head", 0),     # more segments than a CTA joins itself
    (1, 1, 3000, 128, 128, "head", 0),
    (9, 4, 40, 64, 64, "tok", 0),        # short sequences, more than 1024 rows in all
    (4, 4, 130, 64, 48, "head", 0),
    (550, 2, 1, 64, 64, "tok", 0),
    (5, 2, 129, 128, 64, "tok", 0),
    (3, 3, 129, 40, 128, "head", 0),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_matches_oracle(la, shape, state, dt):
    B, H, N, Dk, Dv, layout, lead = shape
    x, decay, S0 = problem(B, H, N, Dk, Dv, dt, N + Dk + Dv, layout, lead)
    check_fwd(la, x, decay, S0 if state else None, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward_matches_oracle(la, shape, dt):
    B, H, N, Dk, Dv, layout, lead = shape
    x, decay, _ = problem(B, H, N, Dk, Dv, dt, 7 + N + Dk + Dv, layout, lead)
    check_bwd(la, x, decay, dt)


# At most 1024 rows: the scores are two bf16 terms, so that what is lost of a term is 2^-16 of it
# (half a step twice: 2^-8 of 2^-8), beside o's own rounding. Sequences of one chunk, from zero:
# the state plays no part.
@pytest.mark.parametrize("shape", [(1, 1, 1, 64, 64), (1, 2, 3, 64, 128), (2, 8, 4, 128, 64), (1, 8, 128, 64, 64),
                                   (1, 3, 100, 128, 128), (3, 4, 20, 32, 48)])
def test_few_rows_lose_nothing_but_the_rounding_of_the_output(la, shape):
    x, decay, _ = problem(*shape, "bf16", 43)
    a, d = [to_f64(t) for t in x], to_f64(decay)
    N = shape[2]

    def check(got, ref, mag, D, what):
        f = (D + N / 16 + 192) * 2.0 ** -24
        near(got, ref, (2.0 ** -16 + f) * 1.01 * mag + 2.0 ** -8 * np.abs(ref), what)

    ref, mag = (tm.decay_attn(*(f(t) for t in a[:3]), d, 0.125)[0] for f in (np.asarray, np.abs))
    check(la.la_decay_attn_fwd(*x[:3], decay, 0.125), ref, mag, shape[3], "o")
    got = la.la_decay_attn_bwd(*x, decay, 0.125)
    ref, mag = (tm.decay_attn_bwd(*(f(t) for t in a), d, 0.125) for f in (np.asarray, np.abs))
    for g, r, m, D, what in zip(got, ref, mag, (shape[4], shape[4], shape[3]), ("dq", "dk", "dv")):
        check(g, r, m, D, what)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(80, 4, 70, 64, 96), (60, 3, 131, 33, 40), (45, 4, 66, 100, 127), (2, 90, 65, 128, 31)])
def test_more_heads_than_sms(la, shape, dt):
    x, decay, S0 = problem(*shape, dt, 41, lead=1)
    check_fwd(la, x, decay, S0, dt)
    check_bwd(la, x, decay, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_slow_and_fast_decays(la, dt):
    # Factors of one (no decay), almost one, tiny, and exactly zero.
    x, _, S0 = problem(1, 6, 520, 64, 64, dt, 3)
    decay = torch.tensor([0.0, -1e-6, -1e-3, -30.0, -3e38, -float("inf")], device="cuda")
    check_fwd(la, x, decay, S0, dt)
    check_bwd(la, x, decay, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N,lengths", [(300, [300, 0, 1, 257, 128]), (40, [3, 40, 500, -2, 39])])
def test_lengths_leave_rows_behind_them(la, N, lengths, dt):
    B = len(lengths)
    x, decay, S0 = problem(B, 2, N, 64, 64, dt, 11)
    keep = [min(max(n, 0), N) for n in lengths]
    for t in x:                                         # nothing behind a length counts
        for b, n in enumerate(keep):
            t[b, :, n:] = float("nan")
    o = torch.full((B, N, 2, 64), 7.0, device="cuda").to(DT[dt]).transpose(1, 2)
    clean = [torch.nan_to_num(t) for t in x]
    # (A call that returns the state sums it in more terms: both calls here do.)
    got = la.la_decay_attn_fwd(*x[:3], decay, 0.125, torch.tensor(lengths, dtype=torch.int32, device="cuda"), S0,
                               torch.empty_like(S0), o=o)
    assert got is o
    want = check_fwd(la, clean, decay, S0, dt, lengths=lengths)
    grads = [torch.full((B, 2, N, 64), 7.0, device="cuda").to(DT[dt]) for _ in range(3)]
    la.la_decay_attn_bwd(*x, decay, 0.125, torch.tensor(lengths, dtype=torch.int32, device="cuda"), *grads)
    refs = check_bwd(la, clean, decay, dt, lengths=lengths)
    for t, r in zip([o] + grads, [want] + list(refs)):
        for b, n in enumerate(keep):
            assert torch.equal(t[b, :, :n], r[b, :, :n]) and (t[b, :, n:] == 7).all()
            assert (r[b, :, n:] == 0).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_lengths_across_segments(la, D, dt):
    x, decay, S0 = problem(4, 2, 1500, D, D, dt, 12)
    lengths = [1500, 700, 0, 129]
    check_fwd(la, x, decay, S0, dt, lengths=lengths)
    check_bwd(la, x, decay, dt, lengths=lengths)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,D", [(1, 1500, 64), (1, 4100, 64), (3, 130, 128)])
def test_state_in_place(la, B, N, D, dt):
    (q, k, v, _), decay, S0 = problem(B, 2, N, D, D, dt, 14)
    want, S = torch.empty_like(S0), S0.clone()
    o = la.la_decay_attn_fwd(q, k, v, decay, S0=S0, S_out=want)
    for _ in range(3):
        S.copy_(S0)
        got = la.la_decay_attn_fwd(q, k, v, decay, S0=S, S_out=S)
        assert torch.equal(got, o) and torch.equal(S, want)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["q", "k", "v", "do"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("N,D", [(300, 64), (1100, 64), (300, 128)])
def test_values_that_are_not_finite_reach_no_earlier_token(la, N, D, what, value, dt):
    x, decay, _ = problem(1, 2, N, D, D, dt, 13, "head")
    at = N // 2
    clean = la.la_decay_attn_fwd(*x[:3], decay, 0.125)
    grads = la.la_decay_attn_bwd(*x, decay, 0.125)
    y = [t.clone() for t in x]
    y["q k v do".split().index(what)][0, :, at, 5] = value
    o = la.la_decay_attn_fwd(*y[:3], decay, 0.125)
    assert torch.equal(o[:, :, :at], clean[:, :, :at])
    if what == "q":
        assert torch.equal(o[:, :, at + 1:], clean[:, :, at + 1:])
    if what != "do":
        assert not torch.isfinite(o[:, :, at]).all()
    dq, dk, dv = la.la_decay_attn_bwd(*y, decay, 0.125)
    # dq sums over earlier tokens, dk and dv over later ones.
    assert torch.equal(dq[:, :, :at], grads[0][:, :, :at])
    for g, r in ((dk, grads[1]), (dv, grads[2])):
        assert torch.equal(g[:, :, at + 1:], r[:, :, at + 1:])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_pieces_and_steps_continue_a_prompt(la, dt):
    x, decay, _ = problem(2, 3, 200, 64, 64, dt, 17)
    q, k, v = x[:3]
    whole = torch.empty(2, 3, 64, 64, device="cuda")
    o = la.la_decay_attn_fwd(q, k, v, decay, S_out=whole)
    S = torch.zeros_like(whole)
    parts = [la.la_decay_attn_fwd(q[:, :, a:b], k[:, :, a:b], v[:, :, a:b], decay, S0=S, S_out=S)
             for a, b in ((0, 0), (0, 130), (130, 190))]
    steps = [la.la_decay_attn_step(q[:, :, t], k[:, :, t], v[:, :, t], decay, S) for t in range(190, 200)]
    got = torch.cat(parts + [torch.stack(steps, 2)], 2)
    a = [to_f64(t) for t in (q, k, v)]
    mag, mS = tm.decay_attn(*map(np.abs, a), to_f64(decay))
    near(got, to_f64(o), 2 * limits(200, 64, dt, to_f64(o), mag), "o")
    near(S, to_f64(whole), 2 * (64 + 13 + 192) * 2.0 ** -24 * mS, "S")


STEPS = [(1, 1, 64, 64, 0), (5, 3, 128, 128, 0), (2, 7, 33, 20, 0), (3, 2, 64, 65, 1), (2, 2, 1, 1, 0), (1, 4, 128, 4, 0),
         (300, 2, 8, 8, 0)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", STEPS)
def test_step_matches_oracle(la, shape, dt):
    B, H, Dk, Dv, lead = shape
    x, decay, S0 = problem(B, H, 1, Dk, Dv, dt, 19, lead=lead)
    q, k, v = (t[:, :, 0] for t in x[:3])
    S = S0.clone()
    o = la.la_decay_attn_step(q, k, v, decay, S, 0.3)
    a = [to_f64(t) for t in x[:3]]
    ro, rS = tm.decay_attn(*a, to_f64(decay), 0.3, S0=to_f64(S0))
    mo, mS = tm.decay_attn(*map(np.abs, a), to_f64(decay), 0.3, S0=np.abs(to_f64(S0)))
    f = (Dk + 32) * 2.0 ** -24
    near(S, rS, 8 * 2.0 ** -24 * mS, "S")
    near(o, ro[:, :, 0], f * mo[:, :, 0] + (2.0 ** -8 * np.abs(ro[:, :, 0]) if dt == "bf16" else 0), "o")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_step_in_the_place_of_an_input(la, dt):
    x, decay, S0 = problem(3, 2, 1, 64, 64, dt, 23)
    for i in range(3):
        y = [t[:, :, 0].clone() for t in x[:3]]
        want = la.la_decay_attn_step(*y, decay, S0.clone())
        got = la.la_decay_attn_step(*y, decay, S0.clone(), o=y[i])
        assert got is y[i] and torch.equal(got, want)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strides_of_every_kind(la, dt):
    # Shared keys (stride 0 over heads), shared sequences, heads outermost.
    x, decay, S0 = problem(2, 4, 140, 64, 64, dt, 29)
    q, k, v, do = x
    k1 = k[:, :1].contiguous().expand(-1, 4, -1, -1)
    v1 = v[:1].contiguous().expand(2, -1, -1, -1)
    check_fwd(la, [q, k1, v1], decay, S0, dt)
    check_bwd(la, [q, k1, v1, do], decay, dt)
    hb = [t.permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3) for t in x]
    check_fwd(la, hb, decay, S0, dt, o=torch.empty(4, 2, 140, 64, device="cuda", dtype=DT[dt]).permute(1, 0, 2, 3))
    spaced = [torch.empty(2, 4, 140, 72, device="cuda", dtype=DT[dt])[..., :64].copy_(t) for t in x]
    check_fwd(la, spaced, decay, S0, dt)
    nb = [t.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3) for t in x]     # [N, B, H, D]
    check_bwd(la, nb, decay, dt, grads=[torch.empty(140, 2, 4, 64, device="cuda", dtype=DT[dt]).permute(1, 2, 0, 3)
                                        for _ in range(3)])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gradients_into_one_projection(la, dt):
    B, H, N, D = 2, 3, 150, 64
    x, decay, _ = problem(B, H, N, D, D, dt, 31)
    buf = torch.full((B, N, 3 * H * D + 8), 5.0, device="cuda").to(DT[dt])
    grads = [buf[..., i * H * D:(i + 1) * H * D].unflatten(2, (H, D)).transpose(1, 2) for i in range(3)]
    want = check_bwd(la, x, decay, dt)
    got = check_bwd(la, x, decay, dt, grads=grads)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and (buf[..., 3 * H * D:] == 5).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_streams_graphs_and_repeats(la, dt):
    x, decay, S0 = problem(2, 2, 700, 64, 64, dt, 37)
    q, k, v, do = x
    S = torch.empty_like(S0)
    o = la.la_decay_attn_fwd(q, k, v, decay, S0=S0, S_out=S)
    g = la.la_decay_attn_bwd(q, k, v, do, decay)
    torch.cuda.synchronize()
    # Two streams at once, each call with its own workspace.
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        T = torch.empty_like(S0)
        got.append((la.la_decay_attn_fwd(q, k, v, decay, S0=S0, S_out=T, stream=s), T,
                    *la.la_decay_attn_bwd(q, k, v, do, decay, stream=s)))
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, (o, S, *g)))
    # Captured once, replayed on other data.
    ws = la.workspace(la.LA_OP_DECAY_ATTN, 2, 2, 700, 64, 64, q.dtype)
    wb = la.workspace(la.LA_OP_DECAY_ATTN_BWD, 2, 2, 700, 64, 64, q.dtype)
    y = [torch.zeros_like(t) for t in x]
    oo, gg, T = torch.empty_like(o), [torch.empty_like(t) for t in g], torch.empty_like(S)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.la_decay_attn_fwd(*y[:3], decay, S0=S0, S_out=T, o=oo, ws=ws)
        la.la_decay_attn_bwd(*y, decay, dq=gg[0], dk=gg[1], dv=gg[2], ws=wb)
        la.la_decay_attn_step(*(t[:, :, 0] for t in y[:3]), decay, T)
    for t, r in zip(y, x):
        t.copy_(r)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    la.la_decay_attn_step(*(t[:, :, 0] for t in x[:3]), decay, S)
    assert all(torch.equal(a, b) for a, b in zip([oo, T] + gg, [o, S] + list(g)))


def test_empty_calls(la):
    S0 = torch.randn(2, 3, 64, 64, device="cuda")
    S = torch.empty_like(S0)
    e = torch.empty(2, 3, 0, 64, device="cuda")
    decay = -torch.ones(3, device="cuda")
    assert la.la_decay_attn_fwd(e, e, e, decay, S0=S0, S_out=S).shape == e.shape
    assert torch.equal(S, S0)
    la.la_decay_attn_fwd(e, e, e, decay, S_out=S)
    assert (S == 0).all()
    assert [t.shape for t in la.la_decay_attn_bwd(e, e, e, e, decay)] == [e.shape] * 3
    n = torch.empty(0, 3, 5, 64, device="cuda")
    assert la.la_decay_attn_fwd(n, n, n, decay).shape == n.shape
    m = torch.empty(0, 3, 64, device="cuda")
    assert la.la_decay_attn_step(m, m, m, decay, torch.empty(0, 3, 64, 64, device="cuda")).shape == m.shape
