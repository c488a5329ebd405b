"""The gated linear recurrence (whole sequences, a training step, single decode tokens) and the layer norm with the
residual sum before it (and its gradients): what is measured, in plain torch and through the framework.

The recurrence keeps one number per channel:
    h_t = a_t h_{t-1} + s(a_t) sigmoid(i_t) x_t,  y_t = h_t
with the decay a = exp(g) ("log"), sigmoid(g) ("sigmoid") or exp(-rate sigmoid(g)) ("rate", one rate per channel), and
the scale s = 1 ("none"), sqrt(1 - a^2) ("sqrt") or 1 - a ("complement"); without i its factor is left out.

The layer norm: total = x + residual, rounded to the type it is kept in; y = (total - mean) / sqrt(var + eps) w + b.
"""
import math

import torch

own = False

CHUNK = 64
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


# ---- cases ---------------------------------------------------------------------------------------------------------

def rec(name, op, B, H, T, D, io, decay="rate", scale="sqrt", gate=True, heads_last=True, state=True):
    return {"name": name, "op": op, "B": B, "H": H, "T": T, "D": D, "io": io, "decay": decay, "scale": scale,
            "gate": gate, "heads_last": heads_last, "state": state}


def norm(name, op, rows, D, io, residual=True, affine=True):
    return {"name": name, "op": op, "rows": rows, "D": D, "io": io, "residual": residual, "affine": affine}


def listed():
    return [
        # prefill at the framework's headline shape, all gates, straight out of the projections
        rec("scan headline", "scan", 8, 16, 4096, 64, "bf16"),
        # the framework's fp32 shape at a ragged length: a plain log decay, inputs in the mixers' own layout
        rec("scan fp32", "scan", 4, 8, 2047, 64, "f32", "log", "none", gate=False, heads_last=False),
        # one long document, wide heads
        rec("scan long", "scan", 1, 16, 65536, 128, "bf16", "sigmoid", "complement", gate=False),
        # a few new tokens of a short conversation: latency
        rec("scan short", "scan", 1, 8, 37, 64, "bf16"),
        # a training step (forward and gradients) at the headline shape
        rec("train headline", "train", 8, 16, 4096, 64, "bf16"),
        # the same in fp32 at a ragged length
        rec("train fp32", "train", 2, 8, 1023, 128, "f32", "sigmoid", "sqrt", heads_last=False),
        # decoding: a large batch, and a single request
        rec("step batch", "step", 256, 16, 1, 64, "bf16"),
        rec("step single", "step", 1, 32, 1, 128, "bf16", "log", "sqrt"),
        # the norm before a mixer at the headline shape, with the residual sum
        norm("norm headline", "norm", 8 * 4096, 16 * 64, "bf16"),
        # the same for one decode token of a large batch
        norm("norm decode", "norm", 256, 16 * 64, "bf16"),
        # gradients at the headline shape
        norm("norm grad headline", "norm_grad", 8 * 4096, 16 * 64, "bf16"),
        # gradients in fp32: ragged rows of an odd width
        norm("norm grad fp32", "norm_grad", 4 * 2047, 8 * 64 + 5, "f32", residual=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "train", "train", "step", "norm", "norm_grad"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_grad"):
        D = _log(rng, 16, 8192)
        if rng.random() < 0.7:
            D = (D + 7) // 8 * 8
        rows = _log(rng, 1, max(2, min(65536, 33000000 // D)))
        return {"op": op, "rows": rows, "D": D, "io": io, "residual": rng.random() < 0.6, "affine": rng.random() < 0.9}
    D = rng.choice([16, 32, 64, 64, 128, 128, 24, 200])
    H = rng.choice([1, 2, 4, 8, 16])
    if op == "step":
        B, T = _log(rng, 1, 1024), 1
    else:
        B = _log(rng, 1, 32)
        T = _log(rng, 1, max(2, min(65536, (16000000 if op == "train" else 67000000) // (B * H * D))))
    state = rng.random() < 0.7
    if op == "train" and not state:
        T = max(T, 2)  # a single token without a state has no gradient for its decay
    return {"op": op, "B": B, "H": H, "T": T, "D": D, "io": io, "decay": rng.choice(["rate", "rate", "log", "sigmoid"]),
            "scale": rng.choice(["sqrt", "sqrt", "none", "complement"]), "gate": rng.random() < 0.7,
            "heads_last": rng.random() < 0.6, "state": state}


def work(c):
    z = 2 if c["io"] == "bf16" else 4
    if c["op"] in ("norm", "norm_grad"):
        n = c["rows"] * c["D"]
        streams = (4 if c["residual"] else 2) if c["op"] == "norm" else (4 if c["residual"] else 3)
        return {"bytes": streams * n * z + 8 * c["D"] * c["affine"], "flops": (8 if c["op"] == "norm" else 16) * n}
    channels = c["B"] * c["H"] * c["D"]
    n = channels * c["T"]
    rates = 4 * c["H"] * c["D"] if c["decay"] == "rate" else 0
    if c["op"] == "train":  # inputs and gy read once, y and the gradients written once
        return {"bytes": ((8 if c["gate"] else 6) * n) * z + (16 if c["state"] else 4) * channels + 2 * rates,
                "flops": 60 * n}
    return {"bytes": (4 if c["gate"] else 3) * n * z + (8 if c["state"] or c["op"] == "step" else 4) * channels + rates,
            "flops": 20 * n}


# ---- inputs --------------------------------------------------------------------------------------------------------

def prepare(c, seed):
    r = torch.Generator(device=DEV).manual_seed(seed)
    dt = DT[c["io"]]

    def randn(*shape):
        return torch.randn(*shape, generator=r, device=DEV)

    if c["op"] in ("norm", "norm_grad"):
        n, D = c["rows"], c["D"]
        # a residual stream has a few channels that are much larger than the others
        loud = 1 + 8 * (torch.rand(D, generator=r, device=DEV) < 0.02)
        s = {"case": c, "x": (randn(n, D) * loud + 0.1 * randn(n, 1)).to(dt)}
        s["weight"] = 1 + 0.1 * randn(D) if c["affine"] else None
        s["bias"] = 0.1 * randn(D) if c["affine"] else None
        if c["op"] == "norm":
            s["residual"] = randn(n, D).to(dt) if c["residual"] else None
        else:
            s["gy"] = randn(n, D).to(dt)
            s["gtotal"] = randn(n, D).to(dt) if c["residual"] else None
        return s
    B, H, T, D = (c[x] for x in ("B", "H", "T", "D"))

    def rows():  # a projection's [B, T, H, D] seen as [B, H, T, D], or that layout itself
        return randn(B, T, H, D).transpose(1, 2) if c["heads_last"] else randn(B, H, T, D)

    s = {"case": c, "x": rows().to(dt), "rate": None}
    if c["decay"] == "rate":  # decays of 0.9 to 0.999 where the gate is half open
        a = 0.9 + 0.099 * torch.rand(H, D, generator=r, device=DEV)
        s["rate"] = -2 * a.log()
        s["g"] = rows().to(dt)
    elif c["decay"] == "sigmoid":
        s["g"] = (2 + rows()).to(dt)
    else:  # channels forget at rates of their own, from a few tokens to a thousand
        rate = torch.exp(-7 * torch.rand(B, H, 1, D, generator=r, device=DEV))
        s["g"] = (-rate * torch.nn.functional.softplus(rows())).to(dt)
    s["i"] = rows().to(dt) if c["gate"] else None
    s["state"] = randn(B, H, D) if c["state"] or c["op"] == "step" else None
    if c["op"] == "step":
        for n in ("x", "g", "i"):
            s[n] = None if s[n] is None else s[n][:, :, 0].contiguous()
    if c["op"] == "train":
        s["gy"] = rows().to(dt)
        s["gstate"] = randn(B, H, D) if c["state"] else None
    return s


# ---- the plain forms -----------------------------------------------------------------------------------------------

def _gates(s):
    """log a, a, the scale s(a), its derivative by log a, sigmoid(i) and the factor of x."""
    c = s["case"]
    g = s["g"].float()
    if c["decay"] == "rate":
        rate = s["rate"][:, None] if g.dim() == 4 else s["rate"]
        la = -rate * torch.sigmoid(g)
    elif c["decay"] == "sigmoid":
        la = -torch.log1p(torch.exp(-g))
    else:
        la = g
    a = 1 + torch.expm1(la)  # nearest to the decay where it is near 1, and a long sequence multiplies thousands
    if c["scale"] == "sqrt":
        size = torch.sqrt(-torch.expm1(2 * la))
        by_log = -a * a / size
    elif c["scale"] == "complement":
        size, by_log = -torch.expm1(la), -a
    else:
        size, by_log = torch.ones_like(a), torch.zeros_like(a)
    open_ = torch.sigmoid(s["i"].float()) if s["i"] is not None else None
    return la, a, size, by_log, open_, size if open_ is None else size * open_


def _doubling(a, b):
    """Prefixes of h <- a h + b along dim -2: the products of a and h from a start of zero."""
    T, n = a.shape[-2], 1
    while n < T:
        b = torch.cat([b[..., :n, :], b[..., n:, :] + a[..., n:, :] * b[..., :-n, :]], -2)
        a = torch.cat([a[..., :n, :], a[..., n:, :] * a[..., :-n, :]], -2)
        n *= 2
    return a, b


def _scan(a, b, h0):
    """h_t = a_t h_{t-1} + b_t along dim 2 of [B, H, T, D]: prefixes inside chunks, then over the chunks."""
    B, H, T, D = a.shape
    n = -(-T // CHUNK)
    pad = n * CHUNK - T
    if pad:
        a = torch.cat([a, a.new_ones(B, H, pad, D)], 2)
        b = torch.cat([b, b.new_zeros(B, H, pad, D)], 2)
    A, S = _doubling(a.reshape(B, H, n, CHUNK, D), b.reshape(B, H, n, CHUNK, D))
    wholeA, wholeS = _doubling(A[..., -1, :], S[..., -1, :])
    ends = wholeA * h0[:, :, None] + wholeS
    starts = torch.cat([h0[:, :, None], ends[:, :, :-1]], 2)
    return (A * starts[..., None, :] + S).reshape(B, H, n * CHUNK, D)[:, :, :T]


def _start(s):
    c = s["case"]
    return s["state"] if s["state"] is not None else torch.zeros(c["B"], c["H"], c["D"], device=DEV)


def _like(x, like):
    """x in the type and the memory order of `like`."""
    return torch.empty_like(like).copy_(x)


def _forward(s):
    la, a, size, by_log, open_, f = _gates(s)
    h = _scan(a, f * s["x"].float(), _start(s))
    return _like(h, s["x"]), h[:, :, -1].contiguous()


def _train(s):
    c = s["case"]
    x, h0 = s["x"].float(), _start(s)
    la, a, size, by_log, open_, f = _gates(s)
    h = _scan(a, f * x, h0)
    out = {"y": _like(h, s["x"]), "hT": h[:, :, -1].contiguous()}
    # G_t = gy_t + a_{t+1} G_{t+1}, with the last state's gradient behind the last token
    end = s["gstate"] if s["gstate"] is not None else torch.zeros_like(h0)
    gy = s["gy"].float()
    after = torch.cat([a[:, :, 1:], torch.ones_like(a[:, :, :1])], 2)
    G = _scan(after.flip(2), gy.flip(2), end).flip(2)
    before = torch.cat([h0[:, :, None], h[:, :, :-1]], 2)
    in_ = x if open_ is None else open_ * x
    by_a = G * (a * before + by_log * in_)
    if c["decay"] == "rate":
        sg = torch.sigmoid(s["g"].float())
        out["grate"] = -(by_a * sg).sum((0, 2), dtype=torch.float64).float()
        by_a = by_a * (-s["rate"][:, None] * sg * (1 - sg))
    elif c["decay"] == "sigmoid":
        by_a = by_a * torch.sigmoid(-s["g"].float())
    out["gg"] = _like(by_a, s["g"])
    out["gx"] = _like(G * f, s["x"])
    if open_ is not None:
        out["gi"] = _like(G * f * x * torch.sigmoid(-s["i"].float()), s["i"])
    if s["state"] is not None:
        out["gh0"] = G[:, :, 0] * a[:, :, 0]
    return out


def _step(s):
    la, a, size, by_log, open_, f = _gates(s)
    h = a * s["state"] + f * s["x"].float()
    s["state"].copy_(h)
    return h.to(s["x"].dtype), s["state"]


def _standard(x):
    x = x - x.mean(-1, keepdim=True)
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return x * r, r


def _norm(s):
    x, dt, total = s["x"].float(), s["x"].dtype, None
    if s["residual"] is not None:
        total = (x + s["residual"].float()).to(dt)
        x = total.float()
    y = _standard(x)[0]
    if s["weight"] is not None:
        y = y * s["weight"] + s["bias"]
    return [y.to(dt)] if total is None else [y.to(dt), total]


def _norm_grad(s):
    n, r = _standard(s["x"].float())
    g, out = s["gy"].float(), {}
    if s["weight"] is not None:
        out["gweight"] = (g * n).sum(0, dtype=torch.float64).float()
        out["gbias"] = g.sum(0, dtype=torch.float64).float()
        g = g * s["weight"]
    gx = r * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    if s["gtotal"] is not None:
        gx = gx + s["gtotal"].float()
    out["gx"] = gx.to(s["x"].dtype)
    return out


# ---- one pass ------------------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"scan": _forward, "train": _train, "step": _step, "norm": _norm, "norm_grad": _norm_grad}[op](s)
    from bayesian_filtering_linear_gb300 import kla
    c = s["case"]
    if op == "norm":
        y, total = kla.layer_norm(s["x"], s["weight"], s["bias"], s["residual"], eps=EPS)
        return [y] if total is None else [y, total]
    if op == "norm_grad":
        return kla.layer_norm_backward(s["x"], s["weight"], gy=s["gy"], gtotal=s["gtotal"], eps=EPS)
    how = {"decay": c["decay"], "scale": c["scale"]}
    if op == "step":
        return kla.recurrence_step(s["x"], s["g"], s["i"], s["rate"], s["state"], **how), s["state"]
    if op == "scan":
        return kla.recurrence_forward(s["x"], s["g"], s["i"], s["rate"], s["state"], **how)
    y, hT, kept = kla.recurrence_forward(s["x"], s["g"], s["i"], s["rate"], s["state"], checkpoints=True, **how)
    out = kla.recurrence_backward(s["x"], s["g"], s["i"], s["rate"], s["state"], gy=s["gy"], ghT=s["gstate"],
                                  checkpoints=kept, state_grad=s["state"] is not None, **how)
    return {"y": y, "hT": hT, **out}


# ---- in 64 bits, token by token ------------------------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    d = {n: x.double() for n, x in s.items() if isinstance(x, torch.Tensor)}
    if c["op"] in ("norm", "norm_grad"):
        return _exact_norm(c, s["x"].dtype, d)
    if c["op"] == "step":
        for n in ("x", "g", "i"):
            if n in d:
                d[n] = d[n].unsqueeze(2)
    B, H, T, D = d["x"].shape
    if c["op"] == "train" and 8.0 * B * H * T * D > 2e10:
        return None
    by_token = {n: d[n].movedim(2, 0).contiguous() for n in ("x", "g", "i", "gy") if n in d}
    x, g = by_token["x"], by_token["g"]
    sg = 1 / (1 + torch.exp(-g))
    loga = {"log": lambda: g, "sigmoid": lambda: -torch.logaddexp(torch.zeros_like(g), -g),
            "rate": lambda: -d["rate"] * sg}[c["decay"]]()
    a, less = torch.exp(loga), -torch.expm1(loga)                  # a, and 1 - a
    size = {"none": lambda: torch.ones_like(a), "complement": lambda: less,
            "sqrt": lambda: torch.sqrt(less * (1 + a))}[c["scale"]]()
    gate = 1 / (1 + torch.exp(-by_token["i"])) if "i" in by_token else torch.ones_like(a)
    h = d["state"].clone() if "state" in d else torch.zeros(B, H, D, dtype=torch.float64, device=DEV)
    first, b = h, size * gate * x
    y = torch.empty_like(x)
    for t in range(T):
        h = torch.addcmul(b[t], a[t], h)
        y[t] = h
    if c["op"] == "step":
        return y[0], h
    if c["op"] == "scan":
        return y.movedim(0, 2), h
    Z = d["gstate"] if "gstate" in d else torch.zeros_like(h)
    G = torch.empty_like(x)
    for t in reversed(range(T)):
        G[t] = Z + by_token["gy"][t]
        Z = a[t] * G[t]
    last = torch.cat([first[None], y[:-1]])
    dsize = {"none": lambda: torch.zeros_like(a), "complement": lambda: -torch.ones_like(a),
             "sqrt": lambda: -a / size}[c["scale"]]()
    ga = G * (last + dsize * gate * x)                             # by the decay itself
    out = {"y": y.movedim(0, 2), "hT": h, "gx": (G * size * gate).movedim(0, 2)}
    if c["decay"] == "log":
        gg = ga * a
    elif c["decay"] == "sigmoid":
        gg = ga * a * less
    else:
        gg = ga * a * -d["rate"] * sg * (1 - sg)
        out["grate"] = (ga * a * -sg).sum((0, 1))
    out["gg"] = gg.movedim(0, 2)
    if "i" in by_token:
        out["gi"] = (G * size * x * gate * (1 - gate)).movedim(0, 2)
    if "state" in d:
        out["gh0"] = Z
    return out


def _exact_norm(c, dt, d):
    x, total = d["x"], None
    if c["op"] == "norm" and c["residual"]:
        total = x + d["residual"]
        x = total.to(dt).double()
    D = x.shape[-1]
    mean = x.sum(-1, keepdim=True) / D
    r = 1 / torch.sqrt(((x - mean) ** 2).sum(-1, keepdim=True) / D + EPS)
    n = (x - mean) * r
    if c["op"] == "norm":
        y = n * d["weight"] + d["bias"] if c["affine"] else n
        return [y] if total is None else [y, total]
    out, g = {}, d["gy"]
    if c["affine"]:
        out["gweight"], out["gbias"] = torch.einsum("nd,nd->d", g, n), g.sum(0)
        g = g * d["weight"]
    # dn/dx = r (1 - 1/D - n n^T / D), symmetric
    gx = r * (g - (g.sum(-1, keepdim=True) + n * torch.einsum("nd,nd->n", g, n)[:, None]) / D)
    out["gx"] = gx + d["gtotal"] if "gtotal" in d else gx
    return out
