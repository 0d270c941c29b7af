"""la_short_conv_fwd / _step against the float64 oracle (oracle/token_mixing.py).

Tolerances. A value is W multiply-adds in fp32 (at most 5 roundings) and a silu
(hardware exponential and division: a few 2^-22): at most 2^-20 of the sum of
magnitudes, and the silu's slope is at most 1.1. bf16 outputs add half a step
of the value. States are copies: equal bits.
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


def problem(B, N, C, W, dt, seed, lead=0, tail=8):
    g = torch.Generator().manual_seed(seed)
    buf = torch.randn(B, N, lead + C + tail, generator=g).to(DT[dt]).cuda()
    w = torch.randn(C, W, generator=g).to(DT[dt]).cuda()
    bias = torch.randn(C, generator=g).to(DT[dt]).cuda()
    state = torch.randn(B, W - 1, C, generator=g).to(DT[dt]).cuda()
    return buf[:, :, lead:lead + C], w, bias, state


def close(got, ref, x, w, bias, state, dt):
    got = to_f64(got)
    size = np.abs(w).max() * w.shape[1] * max(np.abs(x).max(initial=0), np.abs(state).max(initial=0)) \
        + np.abs(bias).max()
    tol = 2.0 ** -20 * size + (2.0 ** -8 * np.abs(ref) if dt == "bf16" else 0)
    assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()


SHAPES = [
    # B, N, C, W, lead
    (2, 37, 64, 4, 0),
    (1, 1, 8, 4, 0),          # fewer tokens than the state holds
    (3, 2, 24, 4, 8),
    (2, 100, 40, 3, 16),
    (2, 19, 36, 2, 0),        # whole pieces for fp32 only
    (2, 50, 33, 4, 0),        # one channel per thread
    (1, 21, 64, 3, 3),        # rows not 16-byte aligned
    (1, 3000, 16, 4, 0),
    (4, 16, 520, 2, 0),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_matches_oracle(la, shape, act, dt):
    B, N, C, W, lead = shape
    x, w, bias, state = problem(B, N, C, W, dt, N + C, lead)
    for b, s0 in ((bias, state), (None, None)):
        y, s1 = la.la_short_conv_fwd(x, w, b, act, state0=s0, return_state=True)
        torch.cuda.synchronize()
        b64 = to_f64(b) if b is not None else np.zeros(C)
        s64 = to_f64(s0) if s0 is not None else np.zeros((B, W - 1, C))
        ry, rs = tm.short_conv(to_f64(x), to_f64(w), b64, act, state=s64)
        close(y, ry, to_f64(x), to_f64(w), b64, s64, dt)
        assert np.array_equal(to_f64(s1), rs)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("C,lead", [(64, 0), (33, 0), (64, 1)])
def test_ragged_rows_are_neither_read_nor_written(la, dt, C, lead):
    B, N, W = 5, 40, 4
    x, w, bias, state = problem(B, N, C, W, dt, 3, lead)
    n = [40, 0, 1, 2, 17]
    for b in range(B):
        x[b, n[b]:] = float("nan")
    buf = torch.full((B, N, C + 8), 5.0, dtype=x.dtype, device="cuda")
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    y = buf[:, :, :C]
    y, s1 = la.la_short_conv_fwd(x, w, bias, True, lengths, state, y=y, return_state=True)
    torch.cuda.synchronize()
    ry, rs = tm.short_conv(to_f64(x), to_f64(w), to_f64(bias), True, n, to_f64(state))
    clean = np.nan_to_num(to_f64(x))
    for b in range(B):
        close(y[b, :n[b]], ry[b, :n[b]], clean, to_f64(w), to_f64(bias), to_f64(state), dt)
        assert (y[b, n[b]:] == 5).all()
    assert np.array_equal(to_f64(s1), rs) and (buf[:, :, C:] == 5).all()
    # Lengths outside 0..N are taken as the nearest bound.
    wild = torch.tensor([99, -7, 1, 2, 17], dtype=torch.int32, device="cuda")
    y2, s2 = la.la_short_conv_fwd(x, w, bias, True, wild, state, y=torch.full_like(x, 5.0), return_state=True)
    assert torch.equal(y2, y) and torch.equal(s2, s1)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("C,W,lead", [(64, 4, 0), (33, 3, 0), (40, 2, 5)])
def test_steps_continue_a_prompt(la, dt, C, W, lead):
    # A prompt, then tokens one by one, equals the prompt with the tokens appended: same
    # multiply-adds in the same order, so equal bits.
    x, w, bias, _ = problem(3, 20, C, W, dt, 11, lead)
    full, last = la.la_short_conv_fwd(x, w, bias, True, return_state=True)
    y, state = la.la_short_conv_fwd(x[:, :14], w, bias, True, return_state=True)
    assert torch.equal(y, full[:, :14])
    for t in range(14, 20):
        yt = la.la_short_conv_step(x[:, t], w, state, bias, True)
        assert torch.equal(yt, full[:, t])
    assert torch.equal(state, last)
    ry, _ = tm.short_conv(to_f64(x), to_f64(w), to_f64(bias), True)
    close(full, ry, to_f64(x), to_f64(w), to_f64(bias), np.zeros(1), dt)


def test_empty_prompt_keeps_the_state_and_streams_and_graphs(la):
    x, w, bias, state = problem(2, 9, 64, 4, "bf16", 12)
    y, s = la.la_short_conv_fwd(x[:, :0], w, bias, state0=state, return_state=True)
    assert y.shape == (2, 0, 64) and torch.equal(s, state)
    first = la.la_short_conv_fwd(x, w, bias, state0=state)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = la.la_short_conv_fwd(x, w, bias, state0=state, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    out = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.la_short_conv_fwd(x, w, bias, state0=state, y=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, other) and torch.equal(first, out)


def test_extreme_values(la):
    # silu far out: -> v above, -> 0 below; infinities and NaN stay in their channel's window.
    x = torch.zeros(1, 6, 16, device="cuda")
    x[0, 2] = torch.tensor([1e4, -1e4, 88, -88, 200, -200] + [0.0] * 10)
    x[0, 2, 8] = float("nan")
    w = torch.zeros(16, 2, device="cuda")
    w[:, 1] = 1
    y = la.la_short_conv_fwd(x, w)[0, 2].cpu()
    assert y[0] == 1e4 and y[4] == 200 and abs(y[2] - 88) < 1e-4
    assert abs(y[1]) < 1e-30 and abs(y[3]) < 1e-30 and abs(y[5]) < 1e-30
    assert y[8].isnan() and torch.isfinite(y[9:]).all()


@pytest.mark.parametrize("dt,C", [("bf16", 4096), ("f32", 2048)])
@pytest.mark.parametrize("W", [2, 4])
def test_long_prompts_equal_their_pieces(la, dt, C, W):
    # Enough work that a thread walks 64 tokens; pieces of 500 tokens, which it walks 8 or
    # fewer at a time, continued from the state: same multiply-adds in the same order, so
    # equal bits, with ragged ends inside a group of rows and on its borders.
    g = torch.Generator(device="cuda").manual_seed(C + W)
    B, N = 4, 6000
    x = torch.randn(B, N, C, generator=g, device="cuda").to(DT[dt])
    w = torch.randn(C, W, generator=g, device="cuda").to(DT[dt])
    n = torch.tensor([N, 5000, 4481, 63], dtype=torch.int32, device="cuda")
    y = torch.full_like(x, 5.0)
    y, last = la.la_short_conv_fwd(x, w, None, True, n, y=y, return_state=True)
    state = torch.zeros(B, W - 1, C, dtype=x.dtype, device="cuda")
    want = torch.full_like(x, 5.0)
    for t in range(0, N, 500):
        _, state = la.la_short_conv_fwd(x[:, t:t + 500], w, None, True, (n - t).clamp(0, 500).to(torch.int32),
                                        state, y=want[:, t:t + 500], return_state=True)
    assert torch.equal(y, want) and torch.equal(last, state)
