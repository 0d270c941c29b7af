"""Float64 token-mixing operators — TEST INFRASTRUCTURE ONLY.

Only tests/ may import this module. It shares no code with the CUDA library.

norm_rope(_bwd): per-head RMS norm and position rotation of one tensor
[B, N, H, D] to head-major [B, H, N, D], and its gradients; short_conv: the
causal depthwise convolution; selective_scan: the recurrence
S_t = exp(d_t A) S_{t-1} + d_t B_t x_t^T, y_t = C_t^T S_t + D x_t token by token;
decay_attn(_bwd): the recurrence S_t = e^l S_{t-1} + k_t v_t^T of a head and its gradients;
group_norm(_bwd): the norm of channels-last rows with silu and gate, and its gradients.
Pins: tests/test_oracle_token_mixing.py, tests/test_oracle_decay_norm.py.
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


def decay_attn(q, k, v, decay, scale=1.0, lengths=None, S0=None):
    """(o [B, H, N, Dv], S [B, H, Dk, Dv]) of S_t = e^decay S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t, token by
    token. q, k [B, H, N, Dk], v [B, H, N, Dv], decay [H]; rows past `lengths` are zero."""
    q, k, v, decay, S0 = _f64(q, k, v, decay, S0)
    B, H, N, Dk = q.shape
    f = np.exp(decay)[:, None, None]
    o = np.zeros(v.shape)
    S = np.zeros((B, H, Dk, v.shape[3])) if S0 is None else S0.copy()
    for b in range(B):
        n = N if lengths is None else min(max(int(lengths[b]), 0), N)
        for t in range(n):
            S[b] = f * S[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
            o[b, :, t] = scale * np.einsum("hd,hde->he", q[b, :, t], S[b])
    return o, S


def decay_attn_bwd(q, k, v, do, decay, scale=1.0, lengths=None):
    """(dq, dk, dv) of sum(o do): with R_t = sum_{i >= t} e^{decay (i - t)} scale q_i do_i^T,
    dq_t = scale S_t do_t, dk_t = R_t v_t, dv_t = R_t^T k_t."""
    q, k, v, do, decay = _f64(q, k, v, do, decay)
    B, H, N, Dk = q.shape
    f = np.exp(decay)[:, None, None]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for b in range(B):
        n = N if lengths is None else min(max(int(lengths[b]), 0), N)
        S = np.zeros((H, Dk, v.shape[3]))
        R = np.zeros_like(S)
        for t in range(n):
            S = f * S + k[b, :, t, :, None] * v[b, :, t, None, :]
            dq[b, :, t] = scale * np.einsum("hde,he->hd", S, do[b, :, t])
        for t in range(n - 1, -1, -1):
            R = f * R + scale * q[b, :, t, :, None] * do[b, :, t, None, :]
            dk[b, :, t] = np.einsum("hde,he->hd", R, v[b, :, t])
            dv[b, :, t] = np.einsum("hde,hd->he", R, k[b, :, t])
    return dq, dk, dv


def _logistic(x):
    return 0.5 * (1 + np.tanh(0.5 * np.asarray(x, dtype=np.float64)))


def group_norm(x, groups, w=None, b=None, z=None, use_silu=False, eps=1e-5):
    """(y [B, N, C], stats [B, G, 2]) of y = act(xh w + b) silu(z), xh over N and the group's channels."""
    x, w, b, z = _f64(x, w, b, z)
    B, N, C = x.shape
    xg = x.reshape(B, N, groups, C // groups)
    mean = xg.mean((1, 3))
    r = 1 / np.sqrt(((xg - mean[:, None, :, None]) ** 2).mean((1, 3)) + eps)
    u = ((xg - mean[:, None, :, None]) * r[:, None, :, None]).reshape(B, N, C)
    u = u if w is None else u * w
    u = u if b is None else u + b
    y = silu(u) if use_silu else u
    return (y if z is None else y * silu(z)), np.stack((mean, r), -1)


def group_norm_bwd(x, groups, dy, w=None, b=None, z=None, use_silu=False, eps=1e-5):
    """(dx, dw, db, dz) of sum(y dy); dw and db as if there were weights, dz None without a gate."""
    x, dy, w, b, z = _f64(x, dy, w, b, z)
    B, N, C = x.shape
    w = np.ones(C) if w is None else w
    b = np.zeros(C) if b is None else b
    _, stats = group_norm(x, groups, eps=eps)
    wide = lambda t: np.repeat(t, C // groups, -1)[:, None]  # noqa: E731
    r = wide(stats[..., 1])
    xh = (x - wide(stats[..., 0])) * r
    u = xh * w + b
    su = _logistic(u)
    v, slope = (u * su, su + u * su * (1 - su)) if use_silu else (u, 1.0)
    dz = None
    if z is not None:
        sz = _logistic(z)
        dz = dy * v * (sz + z * sz * (1 - sz))
        dy = dy * z * sz
    h = dy * slope
    g = h * w
    over = lambda t: wide(t.reshape(B, N, groups, -1).mean((1, 3)))  # noqa: E731
    return r * (g - over(g) - xh * over(g * xh)), (h * xh).sum((0, 1)), h.sum((0, 1)), dz
