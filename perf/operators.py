"""Cases of the token-mixing operators around the linear-attention kernels.

Four operators, each with a plain form in elementary torch operations (32 bits,
64 where 32 lose what matters), the call a user makes of the library, and the
value of its definition in 64 bits:

  rope   per-head RMS norm of q and k and the position rotation in one pass,
         from the token-major projection to the head-major layout that the
         attention entries take; forward, backward, single tokens
  axes   the rotation with several position axes (rows and columns of an
         image; time, height and width of a video), forward and backward
  conv   the short causal depthwise convolution, for prompts and single tokens
  scan   the selective state space scan, for prompts and single tokens

A case is a dict of plain values; `op` names the operator and `form` its
direction ("fwd", "bwd" or "step").
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One generated token for each of 64 sequences: latency counts.
        {"name": "rope_tokens", "op": "rope", "form": "fwd", "dt": "bf16", "B": 64, "N": 1, "Hq": 8,
         "Hk": 8, "D": 64, "R": 32, "axes": 1, "inter": False, "far": 100000},
        # Queries and keys of the bidirectional workload (B = 16, H = 8, N = 8192, D = 128).
        {"name": "rope_bidir", "op": "rope", "form": "fwd", "dt": "bf16", "B": 16, "N": 8192, "Hq": 8,
         "Hk": 8, "D": 128, "R": 64, "axes": 1, "inter": False, "far": 0},
        # Training on sequences of odd length, shared key heads, part of the head rotated.
        {"name": "rope_train", "op": "rope", "form": "bwd", "dt": "bf16", "B": 4, "N": 8191, "Hq": 16,
         "Hk": 4, "D": 64, "R": 24, "axes": 1, "inter": True, "far": 0},
        # 32 x 32 images, two axes, fp32.
        {"name": "axes_images", "op": "axes", "form": "fwd", "dt": "f32", "B": 16, "N": 1024, "Hq": 8,
         "Hk": 8, "D": 64, "R": 32, "axes": 2, "inter": False, "far": 0},
        # A video of 16 frames of 24 x 24 patches, three axes, its training step.
        {"name": "axes_video", "op": "axes", "form": "bwd", "dt": "bf16", "B": 4, "N": 9216, "Hq": 12,
         "Hk": 12, "D": 128, "R": 64, "axes": 3, "inter": True, "far": 0},
        # Four prompts of 4096 tokens, the channels that the scan reads (x, B and C of 64 heads).
        {"name": "conv_prompt", "op": "conv", "form": "fwd", "dt": "bf16", "B": 4, "N": 4096,
         "C": 4352, "W": 4, "silu": True, "ragged": False, "state": False},
        # Ragged prompts that continue from a state, odd channel count, fp32.
        {"name": "conv_ragged", "op": "conv", "form": "fwd", "dt": "f32", "B": 7, "N": 999, "C": 1083,
         "W": 3, "silu": False, "ragged": True, "state": True},
        # One generated token for each of 256 sequences.
        {"name": "conv_tokens", "op": "conv", "form": "step", "dt": "bf16", "B": 256, "N": 1,
         "C": 2304, "W": 4, "silu": True, "ragged": False, "state": True},
        # Short ragged prompts in one batch, continuing from a state: a serving step.
        {"name": "scan_ragged", "op": "scan", "form": "fwd", "dt": "bf16", "B": 8, "N": 333, "H": 16,
         "P": 64, "S": 128, "G": 1, "ragged": True, "state": True, "gate": True},
        # One long document.
        {"name": "scan_long", "op": "scan", "form": "fwd", "dt": "bf16", "B": 1, "N": 65536, "H": 32,
         "P": 64, "S": 128, "G": 1, "ragged": False, "state": False, "gate": True},
        # fp32, two groups.
        {"name": "scan_f32", "op": "scan", "form": "fwd", "dt": "f32", "B": 2, "N": 4000, "H": 8,
         "P": 64, "S": 64, "G": 2, "ragged": False, "state": False, "gate": False},
        # One generated token for each of 128 sequences.
        {"name": "scan_tokens", "op": "scan", "form": "step", "dt": "bf16", "B": 128, "N": 1, "H": 32,
         "P": 64, "S": 128, "G": 1, "ragged": False, "state": True, "gate": True},
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "axes", "conv", "scan", "scan"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op in ("rope", "axes"):
        D = rng.choice([32, 64, 64, 96, 128])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 2, 3])
        N = _log_int(rng, 1, 32768)
        # At most 2^25 values of q and k in all.
        B = _log_int(rng, 1, max(1, min(64, (1 << 25) // (N * (Hq + Hk) * D))))
        return {"op": op, "form": rng.choice(["fwd", "bwd"]), "dt": dt, "B": B, "N": N, "Hq": Hq,
                "Hk": Hk, "D": D, "R": rng.choice([D // 2, D // 2, D // 4, 3 * D // 8]),
                "axes": 1 if op == "rope" else rng.choice([2, 3]), "inter": rng.random() < 0.5,
                "far": rng.choice([0, 0, 1000000]) if op == "rope" else 0}
    if op == "conv":
        C = _log_int(rng, 64, 6000)
        if rng.random() < 0.7:
            C = C // 8 * 8
        form = rng.choice(["fwd", "fwd", "step"])
        N = 1 if form == "step" else _log_int(rng, 1, 16384)
        B = _log_int(rng, 1, max(1, min(512, (1 << 25) // (N * C))))
        ragged = form == "fwd" and rng.random() < 0.5
        return {"op": op, "form": form, "dt": dt, "B": B, "N": N, "C": C, "W": rng.choice([2, 3, 4, 4]),
                "silu": rng.random() < 0.7, "ragged": ragged,
                "state": form == "step" or rng.random() < 0.5}
    G = rng.choice([1, 1, 2])
    H = G * rng.choice([1, 3, 4, 8, 16])
    P = rng.choice([32, 64, 64, 64, 128, 48, 20])
    S = rng.choice([16, 64, 128, 128, 80, 33])
    form = rng.choice(["fwd", "fwd", "step"])
    N = 1 if form == "step" else _log_int(rng, 1, 8192)
    B = _log_int(rng, 1, max(1, min(128, (1 << (24 if dt == "bf16" else 22)) // (N * H * P))))
    ragged = form == "fwd" and rng.random() < 0.5
    return {"op": op, "form": form, "dt": dt, "B": B, "N": N, "H": H, "P": P, "S": S, "G": G,
            "ragged": ragged, "state": form == "step" or rng.random() < 0.5,
            "gate": rng.random() < 0.6}


# ----------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) % (1 << 62))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)


def _lengths(case, g):
    """Lengths of a padded batch: one full, the others anywhere from none to full."""
    if not case["ragged"]:
        return None
    n = (_rand(g, case["B"]) * (case["N"] + 1)).to(torch.int32).clamp_(0, case["N"])
    n[0] = case["N"]
    return n


def _sections(R, axes):
    """Rotated pairs of each axis: equal shares, the first axes take the remainder."""
    return [R // axes + (1 if a < R % axes else 0) for a in range(axes)]


def _frequencies(case):
    """Angle per position (float64) and axis of each rotated pair: base 10000, each axis with its own run."""
    f, ax = [], []
    for a, n in enumerate(_sections(case["R"], case["axes"])):
        f += [10000.0 ** (-i / n) for i in range(n)]
        ax += [a] * n
    return torch.tensor(f, dtype=torch.float64), torch.tensor(ax, dtype=torch.int64)


def _positions(case, g):
    """[B, N, axes]: a running count from a start (tokens), or places on a grid (images, video)."""
    B, N, A = case["B"], case["N"], case["axes"]
    if A == 1:
        start = (_rand(g, B, 1) * case["far"]).to(torch.int64)
        p = (start + torch.arange(N, device="cuda")).unsqueeze(-1)
    else:
        w = max(1, int(round(math.sqrt(N if A == 2 else N / 16))))
        i = torch.arange(N, device="cuda")
        cols = [i // w, i % w] if A == 2 else [i // (w * w), i // w % w, i % w]
        p = torch.stack(cols, -1).expand(B, N, A)
    return p.to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    dt, op, B, N = _DT[case["dt"]], case["op"], case["B"], case["N"]
    st = {"case": case}
    if op in ("rope", "axes"):
        Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
        # q and k are column ranges of one projection [B, N, (Hq + 2 Hk) D] (q | k | v).
        proj = (_randn(g, B, N, (Hq + 2 * Hk) * D) * 1.5).to(dt)
        st["q"] = proj[:, :, : Hq * D].view(B, N, Hq, D)
        st["k"] = proj[:, :, Hq * D:(Hq + Hk) * D].view(B, N, Hk, D)
        st["pos"] = _positions(case, g)
        f, ax = _frequencies(case)
        st["inv_freq"], st["axis"] = f, ax
        st["inv_freq_dev"], st["axis_dev"] = f.cuda(), ax.cuda()
        norm = op == "rope"
        st["wq"] = (1 + 0.2 * _randn(g, D)).to(dt) if norm else None
        st["wk"] = (1 + 0.2 * _randn(g, D)).to(dt) if norm else None
        if case["form"] == "bwd":
            st["dqo"] = _randn(g, B, Hq, N, D).to(dt)
            st["dko"] = _randn(g, B, Hk, N, D).to(dt)
        return st
    st["lengths"] = _lengths(case, g)
    if op == "conv":
        C, W = case["C"], case["W"]
        # x is a column range of the input projection (gate | x | step sizes).
        pad = 64
        if case["form"] == "step":
            st["x"] = _randn(g, B, C + pad).to(dt)[:, pad // 2:pad // 2 + C]
        else:
            st["x"] = _randn(g, B, N, C + pad).to(dt)[:, :, pad // 2:pad // 2 + C]
            st["y"] = torch.zeros(B, N, C, device="cuda", dtype=dt)
        st["w"] = (_randn(g, C, W) * W ** -0.5).to(dt)
        st["bias"] = (0.1 * _randn(g, C)).to(dt)
        st["state"] = _randn(g, B, W - 1, C).to(dt) if case["state"] else None
        return st
    H, P, S, G = case["H"], case["P"], case["S"], case["G"]
    silu = lambda v: v * torch.sigmoid(v)  # noqa: E731
    # x, B and C are column ranges of the convolution's output; the gate and the step
    # sizes are column ranges of the input projection.
    conv = silu(_randn(g, B, N, H * P + 2 * G * S)).to(dt)
    proj = _randn(g, B, N, H * P + H).to(dt)
    x = conv[:, :, : H * P].view(B, N, H, P)
    Bm = conv[:, :, H * P: H * P + G * S].view(B, N, G, S)
    Cm = conv[:, :, H * P + G * S:].view(B, N, G, S)
    z = proj[:, :, : H * P].view(B, N, H, P) if case["gate"] else None
    step = proj[:, :, H * P:]
    if case["form"] == "step":
        x, Bm, Cm, step = x[:, 0], Bm[:, 0], Cm[:, 0], step[:, 0]
        z = z[:, 0] if z is not None else None
    else:
        st["y"] = torch.zeros(B, N, H, P, device="cuda", dtype=dt)
        st["S_out"] = torch.empty(B, H, S, P, device="cuda")
    st.update(x=x, Bm=Bm, Cm=Cm, z=z, step=step)
    st["A"] = -(1 + 15 * _rand(g, H))                                   # decay rates in [-16, -1]
    size = torch.exp(math.log(1e-3) + _rand(g, H) * math.log(100.0))    # step sizes about 1e-3 .. 1e-1
    st["dt_bias"] = size + torch.log(-torch.expm1(-size))               # softplus(dt_bias) = size
    st["D"] = 1 + 0.1 * _randn(g, H)
    st["S0"] = 0.2 * _randn(g, B, H, S, P) if case["state"] else None
    return st


# -------------------------------------------------------------- the plain forms

def _angles(pos, inv_freq, axis):
    """cos and sin [B, N, R] in float64: far positions need it."""
    th = pos.to(torch.float64)[:, :, axis] * inv_freq
    return torch.cos(th), torch.sin(th)


def _rotate(x, cos, sin, inter, back):
    """Rotates the pairs of the first 2 R features of x [B, N, H, D]: (2i, 2i + 1) or (i, i + R)."""
    R = cos.shape[-1]
    c, s = cos.unsqueeze(2), sin.unsqueeze(2)
    s = -s if back else s
    if inter:
        a, b = x[..., 0:2 * R:2], x[..., 1:2 * R:2]
    else:
        a, b = x[..., :R], x[..., R:2 * R]
    u, v = a * c - b * s, b * c + a * s
    rot = torch.stack((u, v), -1).flatten(-2) if inter else torch.cat((u, v), -1)
    return torch.cat((rot, x[..., 2 * R:]), -1)


_EPS = 1e-6


def _rope_plain(st):
    case = st["case"]
    cos, sin = (t.float() for t in _angles(st["pos"], st["inv_freq_dev"], st["axis_dev"]))
    dt = st["q"].dtype

    def forward(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * w.float()
        return _rotate(x, cos, sin, case["inter"], False).transpose(1, 2).to(dt).contiguous()

    def backward(x, w, go):
        g = _rotate(go.float().transpose(1, 2), cos, sin, case["inter"], True)
        if w is None:
            return g.to(dt).contiguous(), None
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
        xh, gw = x * r, g * w.float()
        dx = r * (gw - xh * (gw * xh).mean(-1, keepdim=True))
        return dx.to(dt).contiguous(), (g * xh).sum((0, 1, 2), dtype=torch.float64).float()

    if case["form"] == "fwd":
        return {"qo": forward(st["q"], st["wq"]), "ko": forward(st["k"], st["wk"])}
    dq, dwq = backward(st["q"], st["wq"], st["dqo"])
    dk, dwk = backward(st["k"], st["wk"], st["dko"])
    out = {"dq": dq, "dk": dk}
    if dwq is not None:
        out.update(dwq=dwq, dwk=dwk)
    return out


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _conv_plain(st):
    case = st["case"]
    x, w, W = st["x"], st["w"].float(), case["W"]
    if case["form"] == "step":
        full = torch.cat((st["state"].float(), x.float().unsqueeze(1)), 1)        # [B, W, C]
        y = (full * w.t()).sum(1) + st["bias"].float()
        st["state"].copy_(full[:, 1:])
        y = y * _sigmoid(y) if case["silu"] else y
        return {"y": y.to(x.dtype), "state": st["state"]}
    B, N, C = x.shape
    lengths = st["lengths"]
    before = st["state"].float() if st["state"] is not None else torch.zeros(B, W - 1, C, device=x.device)
    full = torch.cat((before, x.float()), 1)                                     # [B, W - 1 + N, C]
    y = st["bias"].float() + (full.unfold(1, W, 1) * w).sum(-1)
    y = y * _sigmoid(y) if case["silu"] else y
    n = lengths.long() if lengths is not None else torch.full((B,), N, device=x.device)
    if lengths is not None:
        y = torch.where((torch.arange(N, device=x.device) < n[:, None])[..., None], y, 0.0)
    at = (n[:, None] + torch.arange(W - 1, device=x.device))[..., None].expand(B, W - 1, C)
    return {"y": y.to(x.dtype), "state": full.gather(1, at).to(x.dtype)}


def _steps(st):
    """Step sizes softplus(step + bias) in 32 bits."""
    v = st["step"].float() + st["dt_bias"]
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _finish(y, x, st):
    y = y + st["D"][:, None] * x
    if st["z"] is not None:
        z = st["z"].float()
        y = y * z * _sigmoid(z)
    return y.to(st["x"].dtype)


def _scan_plain(st):
    case = st["case"]
    H, P, S, G = case["H"], case["P"], case["S"], case["G"]
    rep = H // G
    d = _steps(st)
    if case["form"] == "step":
        x, Bm, Cm = st["x"].float(), st["Bm"].float(), st["Cm"].float()
        Bh, Ch = (t.repeat_interleave(rep, 1) for t in (Bm, Cm))
        st["S0"].mul_(torch.exp(d * st["A"])[..., None, None])
        st["S0"].add_((d[..., None] * Bh)[..., None] * x[:, :, None, :])
        y = (Ch[..., None] * st["S0"]).sum(2)
        return {"y": _finish(y, x, st), "S": st["S0"]}
    x, Bm, Cm = st["x"].float(), st["Bm"].float(), st["Cm"].float()
    B, N = x.shape[:2]
    if st["lengths"] is not None:
        valid = torch.arange(N, device=x.device) < st["lengths"].long()[:, None]
        d = torch.where(valid[..., None], d, 0.0)
        x, Bm, Cm = (torch.where(valid[..., None, None], t, 0.0) for t in (x, Bm, Cm))
    # Chunks of L tokens: products within a chunk, one matrix over the chunks' states.
    L = 64
    nc = (N + L - 1) // L
    pad = nc * L - N

    def chunks(t):                                     # [B, N, K, ...] -> [B, K, nc, L, ...]
        t = torch.cat((t, t.new_zeros((B, pad) + tuple(t.shape[2:]))), 1)
        return t.view((B, nc, L) + tuple(t.shape[2:])).movedim(3, 1)

    xc, Bc, Cc, dc = chunks(x), chunks(Bm), chunks(Cm), chunks(d)
    a = dc.double() * st["A"].double()[:, None, None]
    cum = torch.cumsum(a, -1)                          # [B, H, nc, L], float64
    low = torch.ones(L, L, device=x.device, dtype=torch.bool).tril()
    dec = torch.exp((cum[..., :, None] - cum[..., None, :]).float().masked_fill(~low, -math.inf))
    scores = torch.matmul(Cc, Bc.transpose(-1, -2)).repeat_interleave(rep, 1)
    y = torch.matmul(scores * dec * dc[..., None, :], xc)
    del scores, dec
    wgt = torch.exp((cum[..., -1:] - cum).float()) * dc
    inc = torch.matmul(Bc.repeat_interleave(rep, 1).transpose(-1, -2), xc * wgt[..., None])
    T = torch.cumsum(cum[..., -1], -1)                 # [B, H, nc]
    T0 = torch.cat((torch.zeros_like(T[..., :1]), T), -1)
    keep = torch.arange(nc + 1, device=x.device)[:, None] > torch.arange(nc, device=x.device)
    M = torch.exp((T0[..., :, None] - T[..., None, :]).float().masked_fill(~keep, -math.inf))
    states = torch.matmul(M, inc.reshape(B, H, nc, S * P)).view(B, H, nc + 1, S, P)
    if st["S0"] is not None:
        states = states + torch.exp(T0.float())[..., None, None] * st["S0"].unsqueeze(2)
    y = y + torch.exp(cum.float())[..., None] * torch.matmul(Cc.repeat_interleave(rep, 1), states[:, :, :-1])
    y = y.movedim(1, 3).reshape(B, nc * L, H, P)[:, :N]
    y = _finish(y, x, st)
    if st["lengths"] is not None:
        y = torch.where(valid[..., None, None], y, torch.zeros_like(y))
    return {"y": y.contiguous(), "S": states[:, :, -1].contiguous()}


def run(state):
    st = state
    case = st["case"]
    op, form = case["op"], case["form"]
    if not own:
        return {"rope": _rope_plain, "axes": _rope_plain, "conv": _conv_plain, "scan": _scan_plain}[op](st)
    import linear_attention_elu_gb300 as la

    if op in ("rope", "axes"):
        if "table" not in st:                          # the program's table, made once
            st["table"] = la.la_rope_table(st["inv_freq"], st["axis"], device=st["q"].device)
        how = dict(wq=st["wq"], wk=st["wk"], norm=op == "rope", eps=_EPS, interleaved=case["inter"])
        if form == "fwd":
            qo, ko = la.la_qk_norm_rope_fwd(st["q"], st["k"], st["pos"], st["table"], **how)
            return {"qo": qo, "ko": ko}
        if "ws" not in st:                             # the program's workspace, made once
            st["ws"] = la.qk_norm_rope_workspace(case["B"], case["N"], case["Hq"], case["Hk"], case["D"],
                                                 device=st["q"].device)
        dq, dk, dwq, dwk = la.la_qk_norm_rope_bwd(st["q"], st["k"], st["dqo"], st["dko"], st["pos"],
                                                  st["table"], ws=st["ws"], **how)
        out = {"dq": dq, "dk": dk}
        if dwq is not None:
            out.update(dwq=dwq, dwk=dwk)
        return out
    if op == "conv":
        if form == "step":
            y = la.la_short_conv_step(st["x"], st["w"], st["state"], bias=st["bias"], silu=case["silu"])
            return {"y": y, "state": st["state"]}
        y, s = la.la_short_conv_fwd(st["x"], st["w"], bias=st["bias"], silu=case["silu"],
                                    lengths=st["lengths"], state0=st["state"], y=st["y"],
                                    return_state=True)
        return {"y": y, "state": s}
    if form == "step":
        y = la.la_selective_scan_step(st["x"], st["step"], st["A"], st["Bm"], st["Cm"], st["S0"], D=st["D"],
                                      z=st["z"], dt_bias=st["dt_bias"])
        return {"y": y, "S": st["S0"]}
    if "ws" not in st:                                 # the program's workspace, made once
        st["ws"] = la.workspace(la.LA_OP_SELECTIVE_SCAN, case["B"], case["H"], case["N"], case["S"], case["P"],
                                st["x"].dtype, st["x"].device)
    y = la.la_selective_scan_fwd(st["x"], st["step"], st["A"], st["Bm"], st["Cm"], D=st["D"], z=st["z"],
                                 dt_bias=st["dt_bias"], lengths=st["lengths"], S0=st["S0"], S_out=st["S_out"],
                                 y=st["y"], ws=st["ws"])
    return {"y": y, "S": st["S_out"]}


# ------------------------------------------------------------------- the work

def work(case):
    e = 2 if case["dt"] == "bf16" else 4
    B, N, op, form = case["B"], case["N"], case["op"], case["form"]
    if op in ("rope", "axes"):
        v = B * N * (case["Hq"] + case["Hk"]) * case["D"]
        # Read and write once; the backward also reads the outputs' gradients (without the
        # norm it needs no inputs).
        passes = 2 if form == "fwd" or op == "axes" else 3
        return {"bytes": v * e * passes + B * N * case["axes"] * 4, "flops": v * (7 if form == "fwd" else 14)}
    if op == "conv":
        v, C, W = B * N * case["C"], case["C"], case["W"]
        s = B * (W - 1) * C
        states = 2 if form == "step" or case["state"] else 1
        return {"bytes": e * (2 * v + states * s + C * (W + 1)), "flops": v * (2 * W + 4)}
    H, P, S, G = case["H"], case["P"], case["S"], case["G"]
    tok = e * (2 * H * P + 2 * G * S + H + (H * P if case["gate"] else 0))
    states = 2 if form == "step" or case["state"] else 1
    return {"bytes": B * N * tok + states * 4 * B * H * S * P, "flops": 5 * B * N * H * S * P}


# -------------------------------------------------- the definitions in 64 bits

def _exact_rope(st):
    case = st["case"]
    B, N, A = st["pos"].shape
    R, D = case["R"], case["D"]
    # The rotation of each pair as a complex factor.
    th = torch.zeros(B, N, R, dtype=torch.float64, device="cuda")
    for i in range(R):
        th[:, :, i] = st["pos"][:, :, int(st["axis"][i])].double() * float(st["inv_freq"][i])
    turn = torch.polar(torch.ones_like(th), th)

    def spin(x, turn):
        x = x.clone()
        if case["inter"]:
            ia, ib = torch.arange(0, 2 * R, 2), torch.arange(1, 2 * R, 2)
        else:
            ia, ib = torch.arange(R), torch.arange(R, 2 * R)
        w = torch.complex(x[..., ia].contiguous(), x[..., ib].contiguous()) * turn.unsqueeze(2)
        x[..., ia], x[..., ib] = w.real, w.imag
        return x

    outs = {}
    for n in ("q", "k"):
        x = st[n].double()
        w = st["w" + n].double() if st["w" + n] is not None else None
        ms = (x.square().sum(-1, keepdim=True) / D + _EPS) if w is not None else None
        if case["form"] == "fwd":
            v = x / ms.sqrt() * w if w is not None else x
            outs[n + "o"] = spin(v, turn).permute(0, 2, 1, 3).contiguous()
            continue
        g = spin(st["d" + n + "o"].double().permute(0, 2, 1, 3), turn.conj())
        if w is None:
            outs["d" + n] = g
            continue
        # d/dx of sum g w x / sqrt(ms): quotient rule, with d ms / dx = 2 x / D.
        dot = (g * w * x).sum(-1, keepdim=True)
        outs["d" + n] = g * w / ms.sqrt() - x * dot / (D * ms * ms.sqrt())
        outs["dw" + n] = (g * x / ms.sqrt()).sum((0, 1, 2))
    return outs


def _exact_conv(st):
    case = st["case"]
    W = case["W"]
    x = st["x"].double()
    x = x.unsqueeze(1) if case["form"] == "step" else x
    B, N, C = x.shape
    hist = st["state"].double() if st["state"] is not None else x.new_zeros(B, W - 1, C)
    w, bias = st["w"].double(), st["bias"].double()
    y, state = x.new_zeros(B, N, C), x.new_zeros(B, W - 1, C)
    for b in range(B):
        n = int(st["lengths"][b]) if st["lengths"] is not None else N
        seq = torch.cat((hist[b], x[b, :n]))
        acc = bias.expand(n, C).clone()
        for k in range(W):
            acc += w[:, k] * seq[k:k + n]
        y[b, :n] = acc / (1 + torch.exp(-acc)) if case["silu"] else acc
        state[b] = seq[n:n + W - 1]
    return {"y": y[:, 0] if case["form"] == "step" else y, "state": state}


def _exact_scan(st):
    # The recurrence, token by token.
    case = st["case"]
    one = case["form"] == "step"
    lift = (lambda t: t.double().unsqueeze(1)) if one else (lambda t: t.double())
    x, Bm, Cm, step = lift(st["x"]), lift(st["Bm"]), lift(st["Cm"]), lift(st["step"])
    B, N, H, P = x.shape
    S, rep = case["S"], case["H"] // case["G"]
    d = torch.nn.functional.softplus(step + st["dt_bias"].double(), threshold=100.0)
    decay = torch.exp(d * st["A"].double())
    state = st["S0"].double() if st["S0"] is not None else x.new_zeros(B, H, S, P)
    y = torch.empty_like(x)
    n = st["lengths"].long() if st["lengths"] is not None else torch.full((B,), N, device=x.device)
    head = torch.arange(H, device=x.device) // rep
    for t in range(N):
        Bt, Ct = Bm[:, t, head], Cm[:, t, head]
        new = decay[:, t, :, None, None] * state
        new.addcmul_((d[:, t, :, None] * Bt).unsqueeze(-1), x[:, t].unsqueeze(2))
        state = new if st["lengths"] is None else torch.where((t < n)[:, None, None, None], new, state)
        y[:, t] = torch.matmul(Ct.unsqueeze(2), state).squeeze(2)
    y = y + st["D"].double()[:, None] * x
    if st["z"] is not None:
        z = lift(st["z"])
        y = y * z / (1 + torch.exp(-z))
    if st["lengths"] is not None:
        y[torch.arange(N, device=x.device) >= n[:, None]] = 0
    return {"y": y[:, 0] if one else y, "S": state}


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "axes": _exact_rope, "conv": _exact_conv, "scan": _exact_scan}[case["op"]](st)
