"""Float64 token-mixing operators — TEST INFRASTRUCTURE ONLY.

Only tests/ may import this module. It shares no code with the CUDA library.

norm_rope(_bwd): per-head RMS norm and position rotation of one tensor
[B, N, H, D] to head-major [B, H, N, D], and its gradients; short_conv: the
causal depthwise convolution; selective_scan: the recurrence
S_t = exp(d_t A) S_{t-1} + d_t B_t x_t^T, y_t = C_t^T S_t + D x_t token by token.
Pins: tests/test_oracle_token_mixing.py.
"""
import numpy as np


def _f64(*ts):
    return [None if t is None else np.asarray(t, dtype=np.float64) for t in ts]


def _pairs(R, interleaved):
    i = np.arange(R)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R)


def angles(pos, inv_freq, axis):
    """[B, N, R] angles of the rotated pairs (pos [B, N, axes] whole numbers)."""
    pos, inv_freq = np.asarray(pos), np.asarray(inv_freq, dtype=np.float64)
    return pos[:, :, np.asarray(axis, dtype=int)].astype(np.float64) * inv_freq


def _rotate(u, th, interleaved):
    """u [B, N, H, D], th [B, N, R]."""
    a, b = _pairs(th.shape[-1], interleaved)
    c, s = np.cos(th)[:, :, None], np.sin(th)[:, :, None]
    out = u.copy()
    out[..., a] = u[..., a] * c - u[..., b] * s
    out[..., b] = u[..., b] * c + u[..., a] * s
    return out


def norm_rope(x, w, pos, inv_freq, axis, norm=True, eps=1e-6, interleaved=False):
    x, w = _f64(x, w)
    u = x
    if norm:
        u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        u = u if w is None else u * w
    return np.ascontiguousarray(_rotate(u, angles(pos, inv_freq, axis), interleaved).transpose(0, 2, 1, 3))


def norm_rope_bwd(x, w, go, pos, inv_freq, axis, norm=True, eps=1e-6, interleaved=False):
    """(dx [B, N, H, D], dw [D] or None) from go = dL/dout [B, H, N, D]."""
    x, w, go = _f64(x, w, go)
    g = _rotate(go.transpose(0, 2, 1, 3), -angles(pos, inv_freq, axis), interleaved)
    if not norm:
        return g, None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    gw = g if w is None else g * w
    dx = r * gw - x * r ** 3 * (gw * x).mean(-1, keepdims=True)
    return dx, (g * r * x).sum((0, 1, 2))


def silu(v):
    return v * np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def short_conv(x, w, bias=None, act=True, lengths=None, state=None):
    """x [B, N, C], w [C, W], state [B, W - 1, C] (inputs before the first token).

    Returns (y [B, N, C] with zero rows past each length, new state)."""
    x, w, bias, state = _f64(x, w, bias, state)
    B, N, C = x.shape
    W = w.shape[1]
    y, out = np.zeros((B, N, C)), np.zeros((B, W - 1, C))
    for b in range(B):
        n = N if lengths is None else int(lengths[b])
        past = np.zeros((W - 1, C)) if state is None else state[b]
        seq = np.concatenate((past, x[b, :n]))
        for t in range(n):
            v = (seq[t:t + W] * w.T).sum(0) + (0 if bias is None else bias)
            y[b, t] = silu(v) if act else v
        out[b] = seq[n:n + W - 1]
    return y, out


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def selective_scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, use_softplus=True, lengths=None,
                   S0=None):
    """x, z [B, N, H, P], dt [B, N, H], A, D, dt_bias [H], Bm, Cm [B, N, G, S], S0 [B, H, S, P].

    Returns (y [B, N, H, P] with zero rows past each length, final state)."""
    x, dt, A, Bm, Cm, D, z, dt_bias, S0 = _f64(x, dt, A, Bm, Cm, D, z, dt_bias, S0)
    B, N, H, P = x.shape
    G, S = Bm.shape[2:]
    grp = np.arange(H) // (H // G)
    step = dt if dt_bias is None else dt + dt_bias
    step = softplus(step) if use_softplus else step
    y = np.zeros((B, N, H, P))
    state = np.zeros((B, H, S, P)) if S0 is None else S0.copy()
    for t in range(N):
        on = np.ones(B, bool) if lengths is None else t < np.asarray(lengths)
        if not on.any():
            break
        d = step[on, t]                                        # [b, H]
        s = np.exp(d * A)[..., None, None] * state[on]
        s = s + (d[..., None] * Bm[on, t][:, grp])[..., None] * x[on, t][:, :, None, :]
        state[on] = s
        y[on, t] = np.einsum("bhs,bhsp->bhp", Cm[on, t][:, grp], s)
        if D is not None:
            y[on, t] += D[:, None] * x[on, t]
        if z is not None:
            y[on, t] *= silu(z[on, t])
    return y, state
