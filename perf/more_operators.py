"""Cases of linear attention with a decay for each head, and of the group norm behind it.

Two operators, each with a plain form in elementary torch operations (32 bits,
64 where 32 lose what matters), the call a user makes of the library, and the
value of its definition in 64 bits:

  decay  causal linear attention whose state decays by a factor of its head per
         token: prompts, their backward pass, single tokens
  norm   group norm over channels-last rows with a silu and a gate: statistics over
         all tokens of a sample (images) or over one token (the heads of an attention
         output), forward and backward

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
        # One generated token for each of 16 sequences: latency counts.
        {"name": "decay_tokens", "op": "decay", "form": "step", "dt": "bf16", "B": 16, "N": 1, "H": 8,
         "Dk": 64, "Dv": 64, "layout": "tok", "ragged": False, "state": True, "slopes": "wide"},
        # One generated token for each of 64 sequences with wide heads.
        {"name": "decay_tokens_wide", "op": "decay", "form": "step", "dt": "bf16", "B": 64, "N": 1, "H": 32,
         "Dk": 128, "Dv": 128, "layout": "tok", "ragged": False, "state": True, "slopes": "narrow"},
        # Short ragged prompts in one batch, continuing from a state: a serving step.
        {"name": "decay_ragged", "op": "decay", "form": "fwd", "dt": "bf16", "B": 8, "N": 333, "H": 16,
         "Dk": 64, "Dv": 64, "layout": "tok", "ragged": True, "state": True, "slopes": "wide"},
        # One long document.
        {"name": "decay_long", "op": "decay", "form": "fwd", "dt": "bf16", "B": 1, "N": 65536, "H": 16,
         "Dk": 64, "Dv": 64, "layout": "head", "ragged": False, "state": False, "slopes": "narrow"},
        # fp32, a value width of its own.
        {"name": "decay_f32", "op": "decay", "form": "fwd", "dt": "f32", "B": 2, "N": 4000, "H": 8,
         "Dk": 64, "Dv": 96, "layout": "head", "ragged": False, "state": False, "slopes": "wide"},
        # A training step's backward pass.
        {"name": "decay_train", "op": "decay", "form": "bwd", "dt": "bf16", "B": 8, "N": 4096, "H": 8,
         "Dk": 64, "Dv": 64, "layout": "head", "ragged": False, "state": False, "slopes": "narrow"},
        # The same for wide heads and an odd length, on the projection's own layout.
        {"name": "decay_train_wide", "op": "decay", "form": "bwd", "dt": "bf16", "B": 4, "N": 2047, "H": 8,
         "Dk": 128, "Dv": 128, "layout": "tok", "ragged": False, "state": False, "slopes": "wide"},
        # Heads of single generated tokens, gated: latency counts.
        {"name": "norm_tokens", "op": "norm", "form": "fwd", "dt": "bf16", "B": 64, "N": 1, "C": 512,
         "G": 8, "silu": False, "gate": True},
        # Heads of whole prompts (B = 16, N = 8192 tokens, H = 8, D = 128), gated.
        {"name": "norm_heads", "op": "norm", "form": "fwd", "dt": "bf16", "B": 131072, "N": 1, "C": 1024,
         "G": 8, "silu": False, "gate": True},
        # Their training step, an odd number of tokens.
        {"name": "norm_heads_train", "op": "norm", "form": "bwd", "dt": "bf16", "B": 32765, "N": 1, "C": 512,
         "G": 8, "silu": False, "gate": True},
        # 64 x 64 images, groups of 10 channels.
        {"name": "norm_images", "op": "norm", "form": "fwd", "dt": "bf16", "B": 16, "N": 4096, "C": 320,
         "G": 32, "silu": True, "gate": False},
        # 32 x 32 images, their training step, fp32.
        {"name": "norm_images_train", "op": "norm", "form": "bwd", "dt": "f32", "B": 16, "N": 1024, "C": 256,
         "G": 16, "silu": True, "gate": False},
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dt = rng.choice(["bf16", "bf16", "f32"])
    if rng.random() < 0.5:
        Dk = rng.choice([64, 64, 128, 32, 80, 33])
        Dv = rng.choice([Dk, Dk, 64, 128, 48, 20])
        H = rng.choice([1, 3, 4, 8, 16])
        form = rng.choice(["fwd", "fwd", "bwd", "bwd", "step"])
        N = 1 if form == "step" else _log_int(rng, 1, 8192)
        B = _log_int(rng, 1, max(1, min(128, (1 << (20 if dt == "bf16" else 19)) // (N * H * (4 if form == "bwd" else 1)))))
        return {"op": "decay", "form": form, "dt": dt, "B": B, "N": N, "H": H, "Dk": Dk, "Dv": Dv,
                "layout": rng.choice(["head", "tok"]), "ragged": form != "step" and rng.random() < 0.3,
                "state": form == "step" or (form == "fwd" and rng.random() < 0.5),
                "slopes": rng.choice(["narrow", "wide"])}
    form = rng.choice(["fwd", "bwd"])
    if rng.random() < 0.5:
        # The heads of single tokens.
        G = rng.choice([1, 4, 8, 12])
        C = G * rng.choice([64, 128, 64, 32, 96, 33])
        N = 1
        B = _log_int(rng, 1, (1 << 25) // C)
    else:
        G = rng.choice([8, 16, 32, 32])
        C = G * rng.choice([4, 8, 10, 16, 20, 7])
        N = _log_int(rng, 16, 9216)
        B = _log_int(rng, 1, max(1, min(64, (1 << 24) // (N * C))))
    return {"op": "norm", "form": form, "dt": dt, "B": B, "N": N, "C": C, "G": G,
            "silu": rng.random() < 0.6, "gate": rng.random() < 0.5}


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


def _log_decay(case, g):
    """Per head: factors 1 - 2^-5 .. 1 - 2^-12 (narrow), or e^-1 .. e^-2^-8 as slopes fall over the heads (wide)."""
    H = case["H"]
    if case["slopes"] == "narrow":
        return torch.log1p(-torch.exp2(-5 - 7 * _rand(g, H)))
    return -torch.exp2(-8 * _rand(g, H))


def _heads(t, case, D):
    """[B, N, H D] as [B, H, N, D]: the view, or laid out that way."""
    t = t.unflatten(-1, (case["H"], D)).transpose(1, 2)
    return t if case["layout"] == "tok" else t.contiguous()


def prepare(case, seed):
    g = _gen(seed)
    dt, op, B, N = _DT[case["dt"]], case["op"], case["B"], case["N"]
    st = {"case": case}
    if op == "decay":
        H, Dk, Dv = case["H"], case["Dk"], case["Dv"]
        # q, k and v are column ranges of one projection (q | k | v) of the tokens.
        proj = _randn(g, B, N, H * (2 * Dk + Dv)).to(dt)
        cut = (H * Dk, 2 * H * Dk)
        st["q"], st["k"], st["v"] = (_heads(t, case, D) for t, D in
                                     ((proj[..., :cut[0]], Dk), (proj[..., cut[0]:cut[1]], Dk), (proj[..., cut[1]:], Dv)))
        st["decay"] = _log_decay(case, g)
        st["scale"] = Dk ** -0.5
        st["S0"] = _randn(g, B, H, Dk, Dv) if case["state"] else None
        st["lengths"] = _lengths(case, g)
        if case["form"] == "step":
            st["q"], st["k"], st["v"] = (st[n][:, :, 0] for n in "qkv")
        elif case["form"] == "fwd":
            st["o"] = _heads(torch.zeros(B, N, H * Dv, device="cuda", dtype=dt), case, Dv)
            st["S_out"] = torch.empty(B, H, Dk, Dv, device="cuda") if case["state"] else None
        else:
            st["do"] = _heads(_randn(g, B, N, H * Dv).to(dt), case, Dv)
            grad = torch.zeros_like(proj)
            st["dq"], st["dk"], st["dv"] = (_heads(t, case, D) for t, D in
                                            ((grad[..., :cut[0]], Dk), (grad[..., cut[0]:cut[1]], Dk), (grad[..., cut[1]:], Dv)))
        return st
    C, G = case["C"], case["G"]
    # Activations with a mean and a size of each channel.
    st["x"] = (_randn(g, B, N, C) * (0.5 + _rand(g, C)) + 0.5 * _randn(g, C)).to(dt)
    st["w"], st["b"] = (1 + 0.2 * _randn(g, C)).to(dt), (0.1 * _randn(g, C)).to(dt)
    # The gate is a column range of the input projection.
    st["z"] = _randn(g, B, N, C + 64).to(dt)[..., 64:] if case["gate"] else None
    if case["form"] == "bwd":
        st["dy"] = _randn(g, B, N, C).to(dt)
        # What the forward pass leaves for the backward one: mean and inverse deviation.
        xg = st["x"].double().view(B, N, G, C // G)
        mean = xg.mean((1, 3))
        var = (xg - mean[:, None, :, None]).square().mean((1, 3))
        st["stats"] = torch.stack((mean, torch.rsqrt(var + _EPS)), -1).float()
    return st


# -------------------------------------------------------------- the plain forms

_EPS = 1e-5
_CHUNK = 64


def _valid(case, st, n):
    """[B, 1, n, 1]: the tokens that a sequence has."""
    return (torch.arange(n, device="cuda") < st["lengths"].long()[:, None])[:, None, :, None]


def _attend(a, b, c, log_decay, S0, n):
    """sum_{j <= i} e^{l (i - j)} (a_i . b_j) c_j with the state S0 before the first token: chunks of tokens, products
    within a chunk, one matrix over the chunks' states. a, b, c [B, H, N, D] in 32 bits, n [B] tokens of each sequence;
    returns the sums and the states after them."""
    B, H, N, D = a.shape
    E, L = c.shape[-1], _CHUNK
    nc = max(1, (N + L - 1) // L)
    pad = nc * L - N
    ac, bc, cc = (torch.cat((t, t.new_zeros(B, H, pad, t.shape[-1])), 2).view(B, H, nc, L, t.shape[-1]) for t in (a, b, c))
    l = log_decay.double()
    i = torch.arange(L, device=a.device, dtype=torch.float64)
    gap = i[:, None] - i
    dec = torch.exp(l[:, None, None] * gap.clamp(min=0)).masked_fill(gap < 0, 0.0).float()          # [H, L, L]
    y = torch.matmul(torch.matmul(ac, bc.transpose(-1, -2)) * dec[:, None], cc)
    inc = torch.matmul(bc.transpose(-1, -2), cc * torch.exp(l[:, None] * (L - 1 - i)).float()[:, None, :, None])
    t = torch.arange(nc, device=a.device, dtype=torch.float64)
    gap = t[:, None] - t - 1
    M = torch.exp(l[:, None, None] * L * gap.clamp(min=0)).masked_fill(gap < 0, 0.0).float()        # [H, nc, nc]
    states = torch.matmul(M, inc.view(B, H, nc, D * E)).view(B, H, nc, D, E)
    if S0 is not None:
        states = states + torch.exp(l[:, None] * L * t).float()[:, :, None, None] * S0.unsqueeze(2)
    y = y + torch.exp(l[:, None] * (i + 1)).float()[:, None, :, None] * torch.matmul(ac, states)
    # The state after n tokens: from the chunk that holds the last one.
    at = ((n - 1).clamp(min=0) // L).view(B, 1, 1, 1, 1)
    rest = (n.view(B) - at.view(B) * L).double()
    back = rest[:, None] - 1 - i                                                                      # [B, L]
    w = torch.exp(l[None, :, None] * back[:, None].clamp(min=0)).masked_fill((back < 0)[:, None], 0.0).float()
    take = lambda t: t.gather(2, at.expand(B, H, 1, t.shape[3], t.shape[4])).squeeze(2)  # noqa: E731
    S = torch.matmul(take(bc).transpose(-1, -2), take(cc) * w[..., None])
    S = S + torch.exp(l * rest[:, None]).float()[..., None, None] * take(states)
    return y.reshape(B, H, nc * L, E)[:, :, :N], S


def _decay_plain(st):
    case = st["case"]
    dt, scale, l = st["q"].dtype, st["scale"], st["decay"]
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    if case["form"] == "step":
        st["S0"].mul_(torch.exp(l)[:, None, None])
        st["S0"].add_(k[..., None] * v[:, :, None, :])
        return {"o": (scale * (q[..., None] * st["S0"]).sum(2)).to(dt), "S": st["S0"]}
    N = case["N"]
    n = st["lengths"].long() if st["lengths"] is not None else torch.full((case["B"],), N, device="cuda")
    if case["form"] == "fwd":
        o, S = _attend(q, k, v, l, st["S0"], n)
        o = scale * o
        if st["lengths"] is not None:
            o = torch.where(_valid(case, st, N), o, 0.0)
        return {"o": o.to(dt), "S": S} if case["state"] else {"o": o.to(dt)}
    g = st["do"].float()
    if st["lengths"] is not None:
        keep = _valid(case, st, N)
        q, k, v, g = (torch.where(keep, t, 0.0) for t in (q, k, v, g))
    # The gradient of each input is a sum of the same form: of earlier tokens for q, of later ones for k and v.
    back = lambda a, b, c: _attend(a.flip(2), b.flip(2), c.flip(2), l, None, n)[0].flip(2)  # noqa: E731
    dq = _attend(g, v, k, l, None, n)[0]
    dk = back(v, g, q)
    dv = back(k, q, g)
    if st["lengths"] is not None:
        dq, dk, dv = (torch.where(keep, t, 0.0) for t in (dq, dk, dv))
    return {"dq": (scale * dq).to(dt), "dk": (scale * dk).to(dt), "dv": (scale * dv).to(dt)}


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _norm_plain(st):
    case = st["case"]
    B, N, C, G = case["B"], case["N"], case["C"], case["G"]
    dt = st["x"].dtype
    x = st["x"].float().view(B, N, G, C // G)
    w, b = st["w"].float().view(G, -1), st["b"].float().view(G, -1)
    z = st["z"].float().view(B, N, G, C // G) if st["z"] is not None else None
    if case["form"] == "fwd":
        mean = x.mean((1, 3), keepdim=True)
        d = x - mean
        rstd = 1 / torch.sqrt((d * d).mean((1, 3), keepdim=True) + _EPS)
        u = d * rstd * w + b
        y = u * _sigmoid(u) if case["silu"] else u
        if z is not None:
            y = y * z * _sigmoid(z)
        return {"y": y.view(B, N, C).to(dt), "stats": torch.stack((mean.view(B, G), rstd.view(B, G)), -1)}
    mean, rstd = (t.view(B, 1, G, 1) for t in st["stats"].unbind(-1))
    xh = (x - mean) * rstd
    u = xh * w + b
    g = st["dy"].float().view(B, N, G, C // G)
    out = {}
    if z is not None:
        s = _sigmoid(z)
        a = u * _sigmoid(u) if case["silu"] else u
        out["dz"] = (g * a * s * (1 + z * (1 - s))).view(B, N, C).to(dt)
        g = g * z * s
    if case["silu"]:
        s = _sigmoid(u)
        g = g * s * (1 + u * (1 - s))
    out["dw"] = (g * xh).sum((0, 1), dtype=torch.float64).float().view(C)
    out["db"] = g.sum((0, 1), dtype=torch.float64).float().view(C)
    g = g * w
    dx = rstd * (g - g.mean((1, 3), keepdim=True) - xh * (g * xh).mean((1, 3), keepdim=True))
    out["dx"] = dx.view(B, N, C).to(dt)
    return out


def run(state):
    st = state
    case = st["case"]
    form = case["form"]
    if not own:
        return _decay_plain(st) if case["op"] == "decay" else _norm_plain(st)
    import linear_attention_elu_gb300 as la

    if case["op"] == "norm":
        if "ws" not in st:                             # the program's workspace, made once
            st["ws"] = la.group_norm_workspace(case["B"], case["N"], case["C"], case["G"], device=st["x"].device)
        how = dict(w=st["w"], b=st["b"], z=st["z"], silu=case["silu"], ws=st["ws"])
        if form == "fwd":
            y, stats = la.la_group_norm_fwd(st["x"], case["G"], eps=_EPS, return_stats=True, **how)
            return {"y": y, "stats": stats}
        dx, dw, db, dz = la.la_group_norm_bwd(st["x"], case["G"], st["dy"], st["stats"], **how)
        out = {"dx": dx, "dw": dw, "db": db}
        if dz is not None:
            out["dz"] = dz
        return out
    if form == "step":
        o = la.la_decay_attn_step(st["q"], st["k"], st["v"], st["decay"], st["S0"], scale=st["scale"])
        return {"o": o, "S": st["S0"]}
    op = la.LA_OP_DECAY_ATTN if form == "fwd" else la.LA_OP_DECAY_ATTN_BWD
    if "ws" not in st:                                 # the program's workspace, made once
        st["ws"] = la.workspace(op, case["B"], case["H"], case["N"], case["Dk"], case["Dv"], st["q"].dtype, st["q"].device)
    how = dict(scale=st["scale"], lengths=st["lengths"], ws=st["ws"])
    if form == "fwd":
        o = la.la_decay_attn_fwd(st["q"], st["k"], st["v"], st["decay"], S0=st["S0"], S_out=st["S_out"], o=st["o"], **how)
        return {"o": o, "S": st["S_out"]} if case["state"] else {"o": o}
    dq, dk, dv = la.la_decay_attn_bwd(st["q"], st["k"], st["v"], st["do"], st["decay"], dq=st["dq"], dk=st["dk"],
                                      dv=st["dv"], **how)
    return {"dq": dq, "dk": dk, "dv": dv}


# ------------------------------------------------------------------- the work

def work(case):
    e = 2 if case["dt"] == "bf16" else 4
    B, N, form = case["B"], case["N"], case["form"]
    if case["op"] == "decay":
        H, Dk, Dv = case["H"], case["Dk"], case["Dv"]
        # q, k, v in and o out; backward q, k, v and o's gradient in, three gradients out. States once each way.
        row = 2 * Dk + 2 * Dv if form != "bwd" else 4 * Dk + 3 * Dv
        states = 2 if case["state"] else 0
        return {"bytes": B * N * H * row * e + states * 4 * B * H * Dk * Dv + 4 * H,
                "flops": (15 if form == "bwd" else 5) * B * N * H * Dk * Dv}
    v = B * N * case["C"]
    # x in, y out, the gate; backward x and y's gradient in, x's out, the gate in and its gradient out.
    passes = (2 + case["gate"]) if form == "fwd" else (3 + 2 * case["gate"])
    return {"bytes": v * e * passes + 8 * B * case["G"] + 2 * e * case["C"] + (8 * case["C"] if form == "bwd" else 0),
            "flops": v * (12 if form == "fwd" else 24)}


# -------------------------------------------------- the definitions in 64 bits

def _exact_decay(st):
    # The recurrence, token by token.
    case = st["case"]
    f = torch.exp(st["decay"].double())[:, None, None]
    scale = st["scale"]
    if case["form"] == "step":
        S = f * st["S0"].double() + torch.einsum("bhd,bhe->bhde", st["k"].double(), st["v"].double())
        return {"o": scale * torch.einsum("bhd,bhde->bhe", st["q"].double(), S), "S": S}
    B, N, H, Dk, Dv = (case[n] for n in ("B", "N", "H", "Dk", "Dv"))
    n = st["lengths"].tolist() if st["lengths"] is not None else [N] * B
    q, k, v = (st[t].double().permute(2, 0, 1, 3).contiguous() for t in "qkv")

    def sweep(a, b, c, order, S):
        """y_t = a_t^T S with S decayed and b_t c_t^T added, over the tokens in the given order."""
        y = c.new_zeros(N, B, H, c.shape[-1])
        alive = torch.tensor(n, device=a.device)
        for t in order:
            new = torch.baddbmm((f * S).flatten(0, 1), b[t].flatten(0, 1).unsqueeze(2), c[t].flatten(0, 1).unsqueeze(1)).view(S.shape)
            if st["lengths"] is not None:
                new = torch.where((t < alive)[:, None, None, None], new, S)
            S = new
            y[t] = torch.matmul(a[t].unsqueeze(2), S).squeeze(2)
        for i, m in enumerate(n):
            y[m:, i] = 0
        return scale * y.permute(1, 2, 0, 3), S

    if case["form"] == "fwd":
        S = st["S0"].double() if st["S0"] is not None else q.new_zeros(B, H, Dk, Dv)
        o, S = sweep(q, k, v, range(N), S)
        return {"o": o, "S": S} if case["state"] else {"o": o}
    g = st["do"].double().permute(2, 0, 1, 3).contiguous()
    zero = lambda d, e: q.new_zeros(B, H, d, e)  # noqa: E731
    return {"dq": sweep(g, v, k, range(N), zero(Dv, Dk))[0],
            "dk": sweep(v, g, q, range(N - 1, -1, -1), zero(Dv, Dk))[0],
            "dv": sweep(k, q, g, range(N - 1, -1, -1), zero(Dk, Dv))[0]}


def _exact_norm(st):
    # Group by group.
    case = st["case"]
    B, N, C, G = case["B"], case["N"], case["C"], case["G"]
    D = C // G
    logistic = lambda t: torch.special.expit(t)  # noqa: E731
    out = {n: [] for n in ("y", "stats", "dx", "dz", "dw", "db")}
    for g in range(G):
        cols = slice(g * D, (g + 1) * D)
        x, w, b = st["x"][..., cols].double(), st["w"][cols].double(), st["b"][cols].double()
        z = st["z"][..., cols].double() if st["z"] is not None else None
        if case["form"] == "fwd":
            var, mean = torch.var_mean(x, (1, 2), correction=0, keepdim=True)
            rstd = (var + _EPS) ** -0.5
            u = (x - mean) * rstd * w + b
            y = u * logistic(u) if case["silu"] else u
            out["y"].append(y * z * logistic(z) if z is not None else y)
            out["stats"].append(torch.cat((mean.view(B, 1), rstd.view(B, 1)), 1))
            continue
        mean, rstd = (st["stats"][:, g, i].double().view(B, 1, 1) for i in (0, 1))
        xh = (x - mean) * rstd
        u = xh * w + b
        gate = z * logistic(z) if z is not None else 1.0
        dy = st["dy"][..., cols].double()
        act = u * logistic(u) if case["silu"] else u
        slope = logistic(u) + act * (1 - logistic(u)) if case["silu"] else 1.0
        if z is not None:
            out["dz"].append(dy * act * (logistic(z) + gate * (1 - logistic(z))))
        du = dy * gate * slope
        out["dw"].append((du * xh).sum((0, 1)))
        out["db"].append(du.sum((0, 1)))
        dxh = du * w
        m = N * D
        out["dx"].append(rstd / m * (m * dxh - dxh.sum((1, 2), keepdim=True) - xh * (dxh * xh).sum((1, 2), keepdim=True)))
    join = {"stats": lambda t: torch.stack(t, 1), "dw": torch.cat, "db": torch.cat}
    return {n: join.get(n, lambda t: torch.cat(t, -1))(t) for n, t in out.items() if t}


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_decay(st) if case["op"] == "decay" else _exact_norm(st)
