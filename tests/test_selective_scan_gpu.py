"""la_selective_scan_fwd / _step against the float64 oracle (oracle/token_mixing.py).

Tolerances, per element, from the sum of magnitudes `mag` of the terms that make
it (the oracle run on absolute values). fp32: a term passes at most N decays, each
off by a few 2^-24 (its exponential, its step size times the rate, which a large
decay suppresses, and the product and sum of the update): (8 N + S + 32) 2^-24 mag.
bf16 inputs are exact; the tensor-core path rounds the weighted scores and the
state to bf16 as operands of the read, half a step (2^-8) of each term, and the
output is rounded once more; for the state itself the weighted values enter as
bf16 terms whose remainder is at most 2^-16 of them.
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


def problem(B, N, H, G, S, P, dt, seed, lead=0, small=False):
    """Inputs as column ranges of the convolution's output and of the projection."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    conv = r(B, N, lead + H * P + 2 * G * S).to(DT[dt]).cuda()
    proj = r(B, N, H * P + H).to(DT[dt]).cuda()
    x = conv[..., lead:lead + H * P].unflatten(2, (H, P))
    Bm = conv[..., lead + H * P:lead + H * P + G * S].unflatten(2, (G, S))
    Cm = conv[..., lead + H * P + G * S:].unflatten(2, (G, S))
    z = proj[..., :H * P].unflatten(2, (H, P))
    step = proj[..., H * P:]
    A = -torch.exp(torch.rand(H, generator=g) * 3).cuda()
    bias = (r(H) - (5.0 if small else 2.0)).cuda()
    D = r(H).cuda()
    S0 = r(B, H, S, P).cuda()
    return dict(x=x, step=step, A=A, Bm=Bm, Cm=Cm, D=D, z=z, dt_bias=bias, S0=S0)


def to64(v):
    return None if v is None else to_f64(v)


def oracle(p, lengths=None, use_softplus=True):
    a = {k: to64(v) for k, v in p.items()}
    args = (a["x"], a["step"], a["A"], a["Bm"], a["Cm"])
    y, S = tm.selective_scan(*args, a["D"], a["z"], a["dt_bias"], use_softplus, lengths, a["S0"])
    ab = [np.abs(a["x"]), a["step"], a["A"], np.abs(a["Bm"]), np.abs(a["Cm"])]
    ym, Sm = tm.selective_scan(*ab, None if a["D"] is None else np.abs(a["D"]), None, a["dt_bias"],
                               use_softplus, lengths, None if a["S0"] is None else np.abs(a["S0"]))
    if a["z"] is not None:
        ym = ym * np.abs(tm.silu(a["z"]))
    return y, S, ym, Sm


def check(y, S, ref, N, Sn, dt):
    ry, rS, ym, Sm = ref
    f = (8 * N + Sn + 32) * 2.0 ** -24
    if dt == "bf16":
        ty, tS = (2.0 ** -8 + f) * ym * 1.01 + 2.0 ** -8 * np.abs(ry), (2.0 ** -16 + f) * Sm
    else:
        ty, tS = f * ym, f * Sm
    ey, eS = np.abs(to_f64(y) - ry), np.abs(to_f64(S) - rS)
    assert (ey <= ty + 1e-30).all(), (ey - ty).max()
    assert (eS <= tS + 1e-30).all(), (eS - tS).max()


SHAPES = [
    # B, N, H, G, S, P, lead
    (2, 40, 4, 1, 64, 64, 0),
    (1, 1, 2, 2, 128, 64, 0),        # one token
    (2, 129, 4, 2, 128, 64, 0),      # one token past a chunk
    (1, 700, 2, 1, 128, 64, 0),      # segments
    (1, 400, 3, 1, 16, 128, 0),      # odd head count, two column blocks
    (2, 130, 2, 2, 80, 48, 0),       # widths of whole 16-byte pieces
    (2, 65, 6, 3, 33, 20, 0),        # neither
    (1, 128, 2, 1, 64, 64, 4),       # rows not 16-byte aligned
    (1, 300, 1, 1, 1, 1, 0),
    (1, 257, 5, 5, 8, 8, 0),
    (3, 5, 8, 2, 128, 128, 0),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_matches_oracle(la, shape, full, dt):
    B, N, H, G, S, P, lead = shape
    p = problem(B, N, H, G, S, P, dt, N + S + P, lead)
    if not full:                       # neither skip, gate, bias nor initial state
        p.update(D=None, z=None, dt_bias=None, S0=None)
    S_out = torch.empty(B, H, S, P, device="cuda")
    y = la.la_selective_scan_fwd(**p, S_out=S_out)
    torch.cuda.synchronize()
    check(y, S_out, oracle(p), N, S, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_slow_and_fast_decays(la, dt):
    # Rates from none to so fast that a chunk's decay underflows.
    p = problem(1, 520, 4, 1, 64, 64, dt, 3)
    p["A"] = torch.tensor([0.0, -1e-4, -50.0, -1e4], device="cuda")
    S_out = torch.empty(1, 4, 64, 64, device="cuda")
    y = la.la_selective_scan_fwd(**p, S_out=S_out)
    torch.cuda.synchronize()
    assert torch.isfinite(y).all() and torch.isfinite(S_out).all()
    check(y, S_out, oracle(p), 520, 64, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_steps_given_directly(la, dt):
    p = problem(2, 150, 2, 1, 64, 64, dt, 4)
    p["step"], p["dt_bias"] = p["step"].abs() * 0.1, None
    S_out = torch.empty(2, 2, 64, 64, device="cuda")
    y = la.la_selective_scan_fwd(**p, S_out=S_out, softplus=False)
    torch.cuda.synchronize()
    check(y, S_out, oracle(p, use_softplus=False), 150, 64, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("S,P,lead", [(128, 64, 0), (20, 12, 1)])
def test_ragged_rows_are_neither_read_nor_written(la, dt, S, P, lead):
    n = [300, 0, 1, 128, 129, 290]
    B, N, H = len(n), 300, 2
    p = problem(B, N, H, 1, S, P, dt, 5, lead)
    for b in range(B):
        for k in ("x", "Bm", "Cm", "step", "z"):
            p[k][b, n[b]:] = float("nan")
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    y = torch.full((B, N, H, P), 5.0, dtype=DT[dt], device="cuda")
    S_out = torch.empty(B, H, S, P, device="cuda")
    la.la_selective_scan_fwd(**p, lengths=lengths, S_out=S_out, y=y)
    torch.cuda.synchronize()
    for b in range(B):
        assert (y[b, n[b]:] == 5).all(), b
        q = {k: (v[b:b + 1, :n[b]] if k in ("x", "Bm", "Cm", "step", "z") else v) for k, v in p.items()}
        q["S0"] = p["S0"][b:b + 1]
        check(y[b:b + 1, :n[b]], S_out[b:b + 1], oracle(q), max(n[b], 1), S, dt)
    assert torch.equal(S_out[1], p["S0"][1])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("S,P", [(128, 64), (16, 32), (33, 20), (64, 128)])
def test_steps_continue_a_prompt(la, dt, S, P):
    # A prompt in two pieces with the state updated in place, then single tokens.
    B, N, H, G = 2, 150, 4, 2
    p = problem(B, N, H, G, S, P, dt, 6)
    tok = ("x", "Bm", "Cm", "step", "z")
    part = lambda a, b: {k: (v[:, a:b] if k in tok else v) for k, v in p.items()}  # noqa: E731
    state = p["S0"].clone()
    outs = []
    for a, b in ((0, 60), (60, 140)):
        q = part(a, b)
        q["S0"] = state
        outs.append(la.la_selective_scan_fwd(**q, S_out=state))
    for t in range(140, N):
        q = {k: (v[:, t] if k in tok else v) for k, v in p.items() if k != "S0"}
        outs.append(la.la_selective_scan_step(**q, S=state).unsqueeze(1))
    torch.cuda.synchronize()
    check(torch.cat(outs, 1), state, oracle(p), N, S, dt)


def test_empty_prompt_keeps_the_state(la):
    p = problem(2, 4, 2, 1, 64, 64, "bf16", 7)
    for k in ("x", "Bm", "Cm", "step", "z"):
        p[k] = p[k][:, :0]
    S_out = torch.empty_like(p["S0"])
    y = la.la_selective_scan_fwd(**p, S_out=S_out)
    assert y.shape == (2, 0, 2, 64) and torch.equal(S_out, p["S0"])


@pytest.mark.parametrize("N", [100, 900])
def test_same_bits_on_another_stream_and_in_graphs_that_share_a_workspace(la, N):
    p = problem(2, N, 2, 1, 128, 64, "bf16", 8)
    ws = la.workspace(la.LA_OP_SELECTIVE_SCAN, 2, 2, N, 128, 64, torch.bfloat16)
    first = la.la_selective_scan_fwd(**p, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = la.la_selective_scan_fwd(**p, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    outs, graphs = [torch.zeros_like(first) for _ in range(2)], []
    for y in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            la.la_selective_scan_fwd(**p, y=y, ws=ws)
        graphs.append(graph)
    for graph in graphs + graphs:
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, other) and torch.equal(first, outs[0]) and torch.equal(first, outs[1])
    assert la.la_query_status(ws) == la.LA_OK


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_convolution_and_scan_together(la, dt):
    # The two as a layer uses them: the convolution's output [B, N, H P + 2 G S] is read
    # in place by the scan; a prompt, then tokens.
    B, N, H, G, S, P = 2, 140, 4, 1, 64, 64
    C = H * P + 2 * G * S
    g = torch.Generator().manual_seed(9)
    proj = torch.randn(B, N + 3, C + H * P + H, generator=g).to(DT[dt]).cuda()
    w = (0.5 * torch.randn(C, 4, generator=g)).to(DT[dt]).cuda()
    p = problem(B, 1, H, G, S, P, dt, 10)
    xin, z, step = proj[..., :C], proj[..., C:C + H * P].unflatten(2, (H, P)), proj[..., C + H * P:]
    common = dict(A=p["A"], D=p["D"], dt_bias=p["dt_bias"])

    def cut(u, d):
        return dict(x=u[..., :H * P].unflatten(d, (H, P)), Bm=u[..., H * P:H * P + G * S].unflatten(d, (G, S)),
                    Cm=u[..., H * P + G * S:].unflatten(d, (G, S)))

    u, cs = la.la_short_conv_fwd(xin[:, :N], w, return_state=True)
    S_out = torch.empty(B, H, S, P, device="cuda")
    ys = [la.la_selective_scan_fwd(step=step[:, :N], z=z[:, :N], S_out=S_out, **cut(u, 2), **common)]
    us = [u]
    for t in range(N, N + 3):
        ut = la.la_short_conv_step(xin[:, t], w, cs)
        ys.append(la.la_selective_scan_step(step=step[:, t], z=z[:, t], S=S_out, **cut(ut, 1), **common).unsqueeze(1))
        us.append(ut.unsqueeze(1))
    torch.cuda.synchronize()
    u64, _ = tm.short_conv(to_f64(xin), to_f64(w))
    u = torch.cat(us, 1)
    mag = np.abs(to_f64(w)).sum(1) * np.abs(to_f64(xin)).max()
    assert (np.abs(to_f64(u) - u64) <= 2.0 ** -20 * mag + (2.0 ** -8 * np.abs(u64) if dt == "bf16" else 0)).all()
    q = dict(p, step=step, z=z, S0=None, **cut(u, 2))
    check(torch.cat(ys, 1), S_out, oracle(q), N + 3, S, dt)


@pytest.mark.parametrize("N,H", [(300, 2), (4096, 2)])
def test_withheld_loads_time_out_and_the_context_survives(la, N, H):
    # The header's test hook withholds the loads: every bounded wait runs out, the call
    # ends and the status says so (one launch, and the segmented form).
    p = problem(1, N, H, 1, 128, 64, "bf16", 12)
    ws = la.workspace(la.LA_OP_SELECTIVE_SCAN, 1, H, N, 128, 64, torch.bfloat16)
    hdr = ws[:256].view(torch.int32)
    hdr[4], hdr[5] = 2000, 1               # 2 ms, withhold
    la.la_selective_scan_fwd(**p, ws=ws)
    assert la.la_query_status(ws) == la.LA_ERR_TIMEOUT
    la.la_workspace_init(ws)
    S_out = torch.empty(1, H, 128, 64, device="cuda")
    y = la.la_selective_scan_fwd(**p, S_out=S_out, ws=ws)
    assert la.la_query_status(ws) == la.LA_OK
    if N < 1000:
        check(y, S_out, oracle(p), N, 128, "bf16")


MANY = [
    # B, N, H, G, S, P: enough units for two per CTA
    (1, 140, 304, 1, 64, 16),
    (1, 300, 303, 1, 64, 64),          # the last CTA has one unit
    (2, 129, 152, 2, 128, 128),        # both units of a CTA belong to one head
    (1, 700, 306, 2, 16, 8),           # odd unit counts per group
]


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("shape", MANY)
def test_many_heads_match_oracle(la, shape, gate):
    B, N, H, G, S, P = shape
    p = problem(B, N, H, G, S, P, "bf16", N + H)
    if not gate:
        p["z"] = None
    S_out = torch.empty(B, H, S, P, device="cuda")
    y = la.la_selective_scan_fwd(**p, S_out=S_out)
    torch.cuda.synchronize()
    check(y, S_out, oracle(p), N, S, "bf16")


def test_many_heads_ragged(la):
    n = [260, 0, 129]
    B, N, H, S, P = len(n), 300, 104, 64, 64
    p = problem(B, N, H, 1, S, P, "bf16", 14)
    for b in range(B):
        for k in ("x", "Bm", "Cm", "step", "z"):
            p[k][b, n[b]:] = float("inf")
    y = torch.full((B, N, H, P), 5.0, dtype=torch.bfloat16, device="cuda")
    state = p["S0"].clone()
    la.la_selective_scan_fwd(**dict(p, S0=state), lengths=torch.tensor(n, dtype=torch.int32, device="cuda"),
                             S_out=state, y=y)
    torch.cuda.synchronize()
    for b in range(B):
        assert (y[b, n[b]:] == 5).all(), b
        q = {k: (v[b:b + 1, :n[b]] if k in ("x", "Bm", "Cm", "step", "z") else v) for k, v in p.items()}
        q["S0"] = p["S0"][b:b + 1]
        check(y[b:b + 1, :n[b]], state[b:b + 1], oracle(q), max(n[b], 1), S, "bf16")
    assert torch.equal(state[1], p["S0"][1])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_segments_equal_pieces(la, dt):
    # A sequence long enough to be cut into segments against the same sequence in two
    # calls through the state: both within the bounds of their own sums.
    p = problem(1, 2600, 8, 1, 64, 64, dt, 15, small=True)
    S_out = torch.empty(1, 8, 64, 64, device="cuda")
    y = la.la_selective_scan_fwd(**p, S_out=S_out)
    state, outs = p["S0"].clone(), []
    for a, b in ((0, 1001), (1001, 2600)):
        q = {k: (v[:, a:b] if k in ("x", "Bm", "Cm", "step", "z") else v) for k, v in p.items()}
        outs.append(la.la_selective_scan_fwd(**dict(q, S0=state), S_out=state))
    torch.cuda.synchronize()
    ref = oracle(p)
    check(y, S_out, ref, 2600, 64, dt)
    check(torch.cat(outs, 1), state, ref, 2600, 64, dt)


def test_two_calls_on_two_streams(la):
    # Two calls in flight at once, each with its own workspace, equal the calls alone.
    ps = [problem(1, 1500, 4, 1, 128, 64, "bf16", s) for s in (16, 17)]
    alone = [la.la_selective_scan_fwd(**p) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    outs = [la.la_selective_scan_fwd(**p, stream=s) for p, s in zip(ps, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, outs):
        assert torch.equal(a, b)


def test_shared_batch_inputs(la):
    # B and C expanded over the batch (stride 0) and a batch that is a slice of a larger one.
    p = problem(3, 70, 4, 1, 64, 64, "bf16", 18)
    p["Bm"], p["Cm"] = (p[k][:1].expand(3, -1, -1, -1) for k in ("Bm", "Cm"))
    S_out = torch.empty(3, 4, 64, 64, device="cuda")
    y = la.la_selective_scan_fwd(**p, S_out=S_out)
    torch.cuda.synchronize()
    check(y, S_out, oracle(p), 70, 64, "bf16")
    q = problem(4, 150, 2, 1, 128, 64, "bf16", 19)
    q = {k: (v[::2, 10:140] if k in ("x", "Bm", "Cm", "step", "z") else v[::2].contiguous() if k == "S0" else v)
         for k, v in q.items()}
    S_out = torch.empty(2, 2, 128, 64, device="cuda")
    y = la.la_selective_scan_fwd(**q, S_out=S_out)
    torch.cuda.synchronize()
    check(y, S_out, oracle(q), 130, 128, "bf16")
