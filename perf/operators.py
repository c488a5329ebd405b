"""The gated delta rule (whole sequences, their gradients, single decode tokens) and the norm of queries and keys
with the position rotation in the same pass: what is measured, in plain torch and through the framework.

The gated delta rule keeps a matrix state S per head. For a token with decay a = exp(g) and write strength beta:
    u = beta (v - a S^T k),  S <- a S + k u^T,  o = scale S^T q
q and k may have fewer heads than v (each key head serves H / Hk neighbouring value heads).
"""
import math

import torch

own = False

CHUNK = 64
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


# ---- cases ---------------------------------------------------------------------------------------------------------

def delta(name, op, B, Hk, H, T, dk, dv, io, state=True):
    return {"name": name, "op": op, "B": B, "Hk": Hk, "H": H, "T": T, "dk": dk, "dv": dv, "io": io, "state": state}


def norm(name, op, B, Hq, Hk, T, D, io, kind, layout, rot, heads_last, start):
    return {"name": name, "op": op, "B": B, "Hq": Hq, "Hk": Hk, "T": T, "D": D, "io": io, "norm": kind,
            "layout": layout, "rot": rot, "heads_last": heads_last, "start": start}


def listed():
    return [
        # training and prefill at the framework's headline shape
        delta("forward headline", "forward", 8, 16, 16, 4096, 64, 64, "bf16"),
        # the framework's fp32 shape, a ragged length
        delta("forward fp32", "forward", 4, 8, 8, 2047, 64, 64, "f32"),
        # one long document, wide heads
        delta("forward long", "forward", 1, 16, 16, 65536, 128, 128, "bf16"),
        # a few new tokens of a short conversation, shared key heads: latency
        delta("forward short", "forward", 1, 4, 8, 37, 32, 64, "bf16"),
        # gradients of the headline shape
        delta("backward headline", "backward", 8, 16, 16, 4096, 64, 64, "bf16"),
        # gradients in fp32, shared key heads, ragged length, rectangular heads
        delta("backward fp32", "backward", 2, 4, 8, 1023, 64, 128, "f32"),
        # decoding: a large batch, and a single request
        delta("step batch", "step", 256, 16, 16, 1, 64, 64, "bf16"),
        delta("step single", "step", 1, 16, 32, 1, 128, 128, "bf16"),
        # queries and keys of the headline shape, straight out of a projection
        norm("norm headline", "norm", 8, 16, 16, 4096, 64, "bf16", "l2", "half", 64, True, 0),
        # decoding far into a long context, part of the head rotated
        norm("norm decode", "norm", 256, 16, 4, 1, 128, "bf16", "rms", "interleaved", 64, True, 1000000),
        # gradients of the first, and in fp32 with neighbouring pairs at a ragged length
        norm("norm grad headline", "norm_grad", 8, 16, 16, 4096, 64, "bf16", "rms", "half", 64, True, 0),
        norm("norm grad fp32", "norm_grad", 2, 8, 8, 1023, 128, "f32", "rms", "interleaved", 32, False, 5000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "backward", "step", "norm", "norm_grad"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_grad"):
        D = rng.choice([16, 32, 64, 128])
        Hk = rng.choice([1, 2, 4, 8, 16])
        Hq = Hk * rng.choice([1, 2, 4])
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(2, min(16384, 67000000 // (B * (Hq + Hk) * D))))
        rot = rng.choice([D, D, D // 2, D // 4])
        return {"op": op, "B": B, "Hq": Hq, "Hk": Hk, "T": T, "D": D, "io": io, "norm": rng.choice(["rms", "l2"]),
                "layout": rng.choice(["half", "interleaved"]), "rot": rot, "heads_last": rng.random() < 0.5,
                "start": rng.choice([0, _log(rng, 1, 4000000)])}
    dk, dv = rng.choice([16, 32, 64, 64, 128, 128]), rng.choice([16, 32, 64, 64, 128, 128])
    Hk = rng.choice([1, 2, 4, 8, 16])
    H = Hk * rng.choice([1, 1, 2, 4])
    if op == "step":
        B, T = _log(rng, 1, max(2, min(512, 33000000 // (H * dk * dv)))), 1
    else:
        B = _log(rng, 1, 16)
        tokens = (33000000 if op == "backward" else 67000000) // (B * H * max(dk, dv))
        T = _log(rng, 1, max(2, min(16384, tokens)))
    state = rng.random() < 0.7
    if op == "backward" and not state:
        T = max(T, 2)  # a single token without a state has no gradient for its decay
    return {"op": op, "B": B, "Hk": Hk, "H": H, "T": T, "dk": dk, "dv": dv, "io": io, "state": state}


def work(c):
    z = 2 if c["io"] == "bf16" else 4
    if c["op"] in ("norm", "norm_grad"):
        n = c["B"] * (c["Hq"] + c["Hk"]) * c["T"] * c["D"]
        if c["op"] == "norm":
            return {"bytes": 2 * n * z, "flops": 8 * n}
        return {"bytes": 3 * n * z, "flops": 20 * n}
    B, Hk, H, T, dk, dv = (c[x] for x in ("B", "Hk", "H", "T", "dk", "dv"))
    keys, values, gates, state = 2 * B * Hk * T * dk, B * H * T * dv, 2 * B * H * T, B * H * dk * dv
    if c["op"] == "backward":
        return {"bytes": (2 * keys + 3 * values + 2 * gates) * z + (16 if c["state"] else 4) * state,
                "flops": 22 * B * H * T * dk * dv}
    return {"bytes": (keys + 2 * values + gates) * z + (8 if c["state"] else 4) * state,
            "flops": 7 * B * H * T * dk * dv}


# ---- inputs --------------------------------------------------------------------------------------------------------

def prepare(c, seed):
    r = torch.Generator(device=DEV).manual_seed(seed)
    dt = DT[c["io"]]

    def randn(*shape):
        return torch.randn(*shape, generator=r, device=DEV)

    if c["op"] in ("norm", "norm_grad"):
        B, T, D = c["B"], c["T"], c["D"]

        def heads(h):  # a projection's [B, T, H, D] seen as [B, H, T, D], or that layout itself
            if c["heads_last"]:
                return randn(B, T, h, D).to(dt).transpose(1, 2)
            return randn(B, h, T, D).to(dt)

        s = {"case": c, "q": heads(c["Hq"]), "k": heads(c["Hk"])}
        s["wq"], s["wk"] = 1 + 0.1 * randn(D), 1 + 0.1 * randn(D)
        half = c["rot"] // 2
        s["freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(DEV)
        first = c["start"] + torch.randint(0, 8, (B, 1), generator=r, device=DEV)
        s["pos"] = first + torch.arange(T, device=DEV)  # every sequence at a place of its own
        if c["op"] == "norm_grad":
            s["gq"], s["gk"] = randn(B, c["Hq"], T, D).to(dt), randn(B, c["Hk"], T, D).to(dt)
        return s
    B, Hk, H, T, dk, dv = (c[x] for x in ("B", "Hk", "H", "T", "dk", "dv"))

    def unit(x):  # queries and keys come normalised
        return (x * x.square().sum(-1, keepdim=True).add(1e-6).rsqrt()).to(dt)

    s = {"case": c, "q": unit(randn(B, Hk, T, dk)), "k": unit(randn(B, Hk, T, dk) + 0.5 * randn(B, Hk, 1, dk)),
         "v": randn(B, H, T, dv).to(dt)}
    # heads forget at rates of their own, from a few tokens to thousands
    rate = torch.exp(-7 * torch.rand(B, H, 1, generator=r, device=DEV))
    s["g"] = (-rate * torch.nn.functional.softplus(randn(B, H, T))).to(dt)
    s["beta"] = torch.sigmoid(randn(B, H, T)).to(dt)
    s["state"] = 0.3 * randn(B, H, dk, dv) if c["state"] or c["op"] == "step" else None
    s["scale"] = dk ** -0.5
    if c["op"] == "step":
        for n in ("q", "k", "v", "g", "beta"):
            s[n] = s[n][:, :, 0].contiguous()
    if c["op"] == "backward":
        s["go"] = randn(B, H, T, dv).to(dt)
        s["gstate"] = 0.3 * randn(B, H, dk, dv) if c["state"] else None
    return s


# ---- the plain forms -----------------------------------------------------------------------------------------------

def _chunks(x, n):
    """[B, H, T, ...] in fp32, padded with zeros to whole chunks: [B, H, n, CHUNK, ...]."""
    x = x.float()
    T = x.shape[2]
    if n * CHUNK > T:
        x = torch.cat([x, x.new_zeros(*x.shape[:2], n * CHUNK - T, *x.shape[3:])], 2)
    return x.reshape(*x.shape[:2], n, CHUNK, *x.shape[3:])


def _tokens(x, T, dt):
    return x.reshape(*x.shape[:2], -1, *x.shape[4:])[:, :, :T].to(dt)


def _inside(s):
    """What each chunk needs of itself, for all chunks at once."""
    c = s["case"]
    n = -(-c["T"] // CHUNK)
    rep = c["H"] // c["Hk"]
    q, k, v = (_chunks(s[x].repeat_interleave(rep, 1) if x != "v" else s[x], n) for x in ("q", "k", "v"))
    b = _chunks(s["beta"], n)[..., None]
    cum = _chunks(s["g"], n).double().cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    D = (cum[..., :, None] - cum[..., None, :]).float().masked_fill_(~low, -math.inf).exp_()
    G = cum.float().exp()[..., None]                              # decay since the chunk's start
    E = (cum[..., -1:] - cum).float().exp()[..., None]            # decay until its end
    A = (b * D * (k @ k.mT)).tril(-1)
    M = torch.zeros_like(A)                                       # (I + A)^-1, row by row
    M.diagonal(dim1=-2, dim2=-1).fill_(1)
    for i in range(1, CHUNK):
        M[..., i:i + 1, :i] = -(A[..., i:i + 1, :i] @ M[..., :i, :i])
    P = D * (q @ k.mT)
    return n, q, k, v, b, D, G, E, M, P


def _states(n, k, v, b, G, E, M, S):
    """The states before every chunk, the chunks' updates u, and the last state."""
    W, V = M @ (b * G * k), M @ (b * v)
    kE, g_end = (E * k).mT, G[..., -1:, :]
    states, U = [], []
    for i in range(n):
        states.append(S)
        u = V[:, :, i] - W[:, :, i] @ S
        U.append(u)
        S = g_end[:, :, i] * S + kE[:, :, i] @ u
    return torch.stack(states, 2), torch.stack(U, 2), S


def _start(s):
    c = s["case"]
    if s["state"] is not None:
        return s["state"]
    return torch.zeros(c["B"], c["H"], c["dk"], c["dv"], device=DEV)


def _forward(s):
    c = s["case"]
    n, q, k, v, b, D, G, E, M, P = _inside(s)
    S, U, last = _states(n, k, v, b, G, E, M, _start(s))
    o = s["scale"] * (G * (q @ S) + P @ U)
    return _tokens(o, c["T"], s["v"].dtype), last


def _backward(s):
    c = s["case"]
    T, dt = c["T"], s["v"].dtype
    n, q, k, v, b, D, G, E, M, P = _inside(s)
    S, U, last = _states(n, k, v, b, G, E, M, _start(s))
    do = s["scale"] * _chunks(s["go"], n)
    Z = s["gstate"] if s["gstate"] is not None else torch.zeros_like(last)
    inner, qG, kb, kE, g_end, Mt = P.mT @ do, (G * q).mT, (b * G * k).mT, E * k, G[..., -1:, :], M.mT
    Zs, dRs, ends = [None] * n, [None] * n, [None] * n
    after = last
    for i in reversed(range(n)):
        Zs[i] = Z
        ends[i] = (Z * after).sum((-2, -1))
        after = S[:, :, i]
        dR = Mt[:, :, i] @ (inner[:, :, i] + kE[:, :, i] @ Z)
        dRs[i] = dR
        Z = g_end[:, :, i] * Z + qG[:, :, i] @ do[:, :, i] - kb[:, :, i] @ dR
    Zc, dR, end = torch.stack(Zs, 2), torch.stack(dRs, 2), torch.stack(ends, 2)
    dP = D * (do @ U.mT).tril()
    dA = D * (-(dR @ U.mT)).tril(-1)
    dq = G * (do @ S.mT) + dP @ k
    X = dA @ k - G * (dR @ S.mT)
    Y = E * (U @ Zc.mT) + dP.mT @ q + (b * dA).mT @ k
    dk = b * X + Y
    kX = (k * X).sum(-1)
    line = ((q * dq).sum(-1) + b[..., 0] * kX - (k * Y).sum(-1)).double()
    dg = line.flip(-1).cumsum(-1).flip(-1) + end[..., None]
    db = (dR * v).sum(-1) + kX
    rep = c["H"] // c["Hk"]

    def shared(x):
        x = x.reshape(*x.shape[:2], -1, x.shape[-1])[:, :, :T]
        return x.reshape(x.shape[0], c["Hk"], rep, T, -1).sum(2).to(dt)

    out = {"gq": shared(dq), "gk": shared(dk), "gv": _tokens(b * dR, T, dt), "gg": _tokens(dg, T, dt),
           "gbeta": _tokens(db, T, dt)}
    if s["state"] is not None:
        out["gstate0"] = Z
    return out


def _step(s):
    c = s["case"]
    rep = c["H"] // c["Hk"]
    q, k = (s[x].float().repeat_interleave(rep, 1)[..., None] for x in ("q", "k"))
    v, S = s["v"].float(), s["state"]
    S = s["g"].float().exp()[..., None, None] * S
    u = s["beta"].float()[..., None] * (v - (S * k).sum(-2))
    S = S + k * u[..., None, :]
    s["state"].copy_(S)
    return (s["scale"] * (S * q).sum(-2)).to(s["v"].dtype), s["state"]


def _pairs(x, half, layout):
    if layout == "half":
        return x[..., :half], x[..., half:2 * half]
    return x[..., :2 * half:2], x[..., 1:2 * half:2]


def _joined(a, b, rest, layout):
    turned = torch.cat([a, b], -1) if layout == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _angles(s):
    a = s["pos"].double()[:, None, :, None] * s["freq"].double()
    return a.cos().float(), a.sin().float()


def _rotated(x, cos, sin, half, layout):
    a, b = _pairs(x, half, layout)
    return _joined(a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:], layout)


def _size(c, x):
    m = x.square().sum(-1, keepdim=True) if c["norm"] == "l2" else x.square().mean(-1, keepdim=True)
    return (m + 1e-6).rsqrt()


def _norm(s):
    c = s["case"]
    cos, sin = _angles(s)
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        dt, x = x.dtype, x.float()
        y = _rotated(x * _size(c, x) * w, cos, sin, c["rot"] // 2, c["layout"])
        out.append(y.to(dt).contiguous())
    return out


def _norm_grad(s):
    c = s["case"]
    cos, sin = _angles(s)
    out = {}
    for name, x, w, g in (("q", s["q"], s["wq"], s["gq"]), ("k", s["k"], s["wk"], s["gk"])):
        dt, x = x.dtype, x.float()
        g = _rotated(g.float(), cos, -sin, c["rot"] // 2, c["layout"])  # the rotation's transpose
        r = _size(c, x)
        xr, gw = x * r, g * w
        out["g%s_weight" % name] = (g * xr).sum((0, 1, 2), dtype=torch.float64).float()
        dot = (gw * xr).sum(-1, keepdim=True)
        out["g" + name] = (r * (gw - xr * (dot / (1 if c["norm"] == "l2" else c["D"])))).to(dt)
    return out


# ---- one pass ------------------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"forward": _forward, "backward": _backward, "step": _step, "norm": _norm, "norm_grad": _norm_grad}[op](s)
    from bayesian_filtering_linear_gb300 import kla
    c = s["case"]
    if op == "forward":
        return kla.delta_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], scale=s["scale"])
    if op == "backward":
        return kla.delta_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], go=s["go"],
                                  gstateT=s["gstate"], scale=s["scale"], state_grad=s["state"] is not None)
    if op == "step":
        return kla.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], scale=s["scale"]), s["state"]
    how = {"norm": c["norm"], "layout": c["layout"], "eps": 1e-6}
    if op == "norm":
        return list(kla.norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["freq"], s["pos"], **how))
    return kla.norm_rope_backward(s["q"], s["k"], s["wq"], s["wk"], s["freq"], s["pos"], gyq=s["gq"], gyk=s["gk"],
                                  **how)


# ---- in 64 bits, token by token ------------------------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    d = {n: x.double() for n, x in s.items() if isinstance(x, torch.Tensor)}
    if c["op"] in ("norm", "norm_grad"):
        return _exact_norm(c, d)
    B, Hk, H, T, dk, dv = (c[x] for x in ("B", "Hk", "H", "T", "dk", "dv"))
    if c["op"] == "step":
        for n in ("q", "k", "v", "g", "beta"):
            d[n] = d[n].unsqueeze(2)
    keep = c["op"] == "backward"
    if keep and 8.0 * B * H * T * dk * dv > 6e10:
        return None
    heads = torch.arange(H, device=DEV) // (H // Hk)
    by_token = {n: d[n][:, heads].movedim(2, 0).contiguous() for n in ("q", "k")}
    q, k = by_token["q"], by_token["k"]
    v, a, b = (d[n].movedim(2, 0).contiguous() for n in ("v", "g", "beta"))
    a = a.exp()
    S = d["state"].clone() if "state" in d else torch.zeros(B, H, dk, dv, dtype=torch.float64, device=DEV)
    o = torch.empty(T, B, H, dv, dtype=torch.float64, device=DEV)
    missed = torch.empty_like(o)                                   # v - a S^T k
    before = torch.empty(T, B, H, dk, dv, dtype=torch.float64, device=DEV) if keep else None
    for t in range(T):
        if keep:
            before[t] = S
        S = S * a[t][..., None, None]
        missed[t] = v[t] - torch.matmul(k[t].unsqueeze(-2), S).squeeze(-2)
        S = S + k[t].unsqueeze(-1) * (b[t].unsqueeze(-1) * missed[t]).unsqueeze(-2)
        o[t] = torch.matmul(q[t].unsqueeze(-2), S).squeeze(-2) * s["scale"]
    if c["op"] == "step":
        return o[0], S
    if not keep:
        return o.movedim(0, 2), S
    go = d["go"].movedim(2, 0) * s["scale"]
    Z = d["gstate"].clone() if "gstate" in d else torch.zeros_like(S)
    gq, gk, gv, gg, gb = (torch.empty_like(x) for x in (q, k, v, a, b))
    after = S
    for t in reversed(range(T)):
        u = b[t].unsqueeze(-1) * missed[t]
        gq[t] = torch.matmul(after, go[t].unsqueeze(-1)).squeeze(-1)
        Z = Z + q[t].unsqueeze(-1) * go[t].unsqueeze(-2)
        gu = torch.matmul(k[t].unsqueeze(-2), Z).squeeze(-2)
        gb[t] = (gu * missed[t]).sum(-1)
        gv[t] = b[t].unsqueeze(-1) * gu
        gk[t] = torch.matmul(Z, u.unsqueeze(-1)).squeeze(-1) - a[t][..., None] * torch.matmul(before[t], gv[t].unsqueeze(-1)).squeeze(-1)
        Z = Z - k[t].unsqueeze(-1) * gv[t].unsqueeze(-2)
        Z = Z * a[t][..., None, None]
        gg[t] = (Z * before[t]).sum((-2, -1))
        after = before[t]
    by_key = [x.movedim(0, 2).reshape(B, Hk, H // Hk, T, dk).sum(2) for x in (gq, gk)]
    out = {"gq": by_key[0], "gk": by_key[1], "gv": gv.movedim(0, 2), "gg": gg.movedim(0, 2), "gbeta": gb.movedim(0, 2)}
    if "state" in d:
        out["gstate0"] = Z
    return out


def _exact_norm(c, d):
    """Each pair as a complex number, turned by exp(i angle)."""
    half, D = c["rot"] // 2, c["D"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), d["pos"][:, None, :, None] * d["freq"])

    def rotate(x, turn):
        y = x.clone()
        if c["layout"] == "half":
            z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
            y[..., :half], y[..., half:2 * half] = z.real, z.imag
        else:
            z = torch.view_as_complex(x[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * turn
            y[..., :2 * half] = torch.view_as_real(z).flatten(-2)
        return y

    out = {}
    for n in ("q", "k"):
        x, w = d[n], d["w" + n]
        size = ((x * x).sum(-1, keepdim=True) / (1 if c["norm"] == "l2" else D) + 1e-6).sqrt()
        if c["op"] == "norm":
            out[n] = rotate(w * (x / size), turn)
            continue
        g = rotate(d["g" + n], turn.conj())
        out["g%s_weight" % n] = (g * (x / size)).flatten(0, 2).sum(0)
        g = g * w
        out["g" + n] = g / size - x * ((g * x).sum(-1, keepdim=True) / size ** 3 / (1 if c["norm"] == "l2" else D))
    return [out["q"], out["k"]] if c["op"] == "norm" else out
