"""The gated linear recurrence against the fp64 oracle, which also gives the
bound that arithmetic in 24 bits keeps (see there). bf16 outputs are off by half
a step more, 2^-8 of the value and of the bound."""
import itertools

import numpy as np
import pytest
import torch

from bayesian_filtering_linear_gb300 import kla
from oracle import recurrence as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
KINDS = list(itertools.product(["log", "sigmoid", "rate"], ["none", "sqrt", "complement"]))


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(got, want, err, io, what):
    got = f64(got)
    tol = err + (2.0 ** -8 * (np.abs(want) + err) if io == "bf16" else 0) + 1e-36
    off = np.abs(got - want)
    assert (off <= tol).all(), f"{what}: {np.nanmax(off / tol):.3g} of the bound (largest {np.abs(want).max():.3g})"


def make(B, H, T, D, io, decay="log", gate=True, state=True, heads_last=False, seed=0):
    r = torch.Generator().manual_seed(seed + T)

    def rows():
        x = torch.randn(B, T, H, D, generator=r) if heads_last else torch.randn(B, H, T, D, generator=r)
        return x, (lambda z: z.to(DT[io]).to(DEV).transpose(1, 2) if heads_last else z.to(DT[io]).to(DEV))

    x, put = rows()
    x = put(x)
    g, put = rows()
    if decay == "log":  # from a token's memory to a thousand tokens'
        g = -torch.exp(-7 * torch.rand(D, generator=r)) * torch.nn.functional.softplus(g)
    g = put(g + (2 if decay == "sigmoid" else 0))
    i = put(rows()[0]) if gate else None
    rate = (-2 * torch.log(0.9 + 0.099 * torch.rand(H, D, generator=r))).to(DEV) if decay == "rate" else None
    h0 = torch.randn(B, H, D, generator=r).to(DEV) if state else None
    gy = put(rows()[0])
    ghT = torch.randn(B, H, D, generator=r).to(DEV) if state else None
    return x, g, i, rate, h0, gy, ghT


def check(B, H, T, D, io, decay="log", scale="none", **kw):
    x, g, i, rate, h0, gy, ghT = make(B, H, T, D, io, decay, **kw)
    how = {"decay": decay, "scale": scale}
    y, hT, kept = kla.recurrence_forward(x, g, i, rate, h0, checkpoints=True, **how)
    d = kla.recurrence_backward(x, g, i, rate, h0, gy=gy, ghT=ghT, checkpoints=kept, **how)
    again = kla.recurrence_backward(x, g, i, rate, h0, gy=gy, ghT=ghT, **how)
    args = [f64(t) for t in (x, g, i, rate, h0)]
    f = R.forward(*args, **how)
    near(y, f["y"], f["y_err"], io, "y")
    near(hT, f["hT"], f["hT_err"], "f32", "hT")
    want = R.backward(*args, f64(gy), f64(ghT), **how)
    for n, t in d.items():
        near(t, want[n], want[n + "_err"], "f32" if n in ("grate", "gh0") else io, n)
        assert torch.equal(t, again[n]), n
    assert set(d) == {n for n in want if not n.endswith("_err")}
    assert y.stride() == x.stride() and d["gx"].stride() == x.stride()


@pytest.mark.parametrize("decay,scale", KINDS)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [True, False])
def test_kinds(decay, scale, io, gate):
    check(2, 3, 77, 24, io, decay, scale, gate=gate)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 63, 64, 65, 127, 129, 511, 513, 1031])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_lengths(T, io):
    check(1, 2, T, 32, io, "rate", "sqrt", heads_last=True, seed=T)


@pytest.mark.parametrize("B,H,T,D", [(1, 1, 100, 8), (3, 1, 40, 8), (1, 5, 200, 200), (2, 4, 300, 128), (7, 3, 65, 40)])
@pytest.mark.parametrize("state", [True, False])
def test_shapes(B, H, T, D, state):
    check(B, H, T, D, "bf16", "sigmoid", "complement", state=state)
    check(B, H, T, D, "f32", "log", "sqrt", gate=False, state=state, heads_last=True)


@pytest.mark.parametrize("channels", [64 * k for k in (12, 30, 60, 80, 110, 160, 230)])
def test_clusters_of_every_size(channels):
    """From eight blocks along a sequence to one, by the number of channels."""
    check(channels // 64, 2, 700, 32, "bf16", "rate", "sqrt", heads_last=True, seed=channels)


@pytest.mark.parametrize("channels,T", [(64, 1100), (64 * 12, 1025), (64 * 18, 1400), (64 * 30, 800)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_clusters_above_eight(channels, T, io):
    check(1, channels // 64, T, 64, io, "log", "sqrt", gate=False)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_many_channels(io):
    check(40, 16, 131, 64, io, "log", "sqrt", gate=False)


def test_thousands_of_decays_do_not_drift():
    """Decays of 1 - 2^-13, the same for every token, from a state of one and from random inputs: the error stays that of
    random roundings, sqrt(memory) steps of 2^-24, sixteen for the worst channel (one float of a decay: up to memory)."""
    T, D = 16384, 64
    g = torch.full((1, 1, T, D), -2.0 ** -13, device=DEV) * (1 + 0.3 * torch.rand(D, device=DEV))
    x = torch.randn(1, 1, T, D, device=DEV)
    h0 = torch.ones(1, 1, D, device=DEV)
    for v in (x, torch.zeros_like(x)):
        y, hT = kla.recurrence_forward(v, g, None, None, h0)
        f = R.forward(f64(v), f64(g), h0=f64(h0))
        top = np.abs(f["y"]).max(2)
        assert (np.abs(f64(hT) - f["hT"]) <= 16 * np.sqrt(2.0 ** 13) * 2.0 ** -24 * top).all()


def test_pieces_and_single_tokens_are_one_sequence():
    x, g, i, rate, h0, _, _ = make(2, 3, 150, 40, "f32", "rate")
    how = {"decay": "rate", "scale": "sqrt"}
    f = R.forward(*[f64(t) for t in (x, g, i, rate, h0)], **how)
    h, got = h0, []
    for a, b in ((0, 64), (64, 71), (71, 130), (130, 150)):
        y, h = kla.recurrence_forward(x[:, :, a:b], g[:, :, a:b], i[:, :, a:b], rate, h, **how)
        got.append(y)
    near(torch.cat(got, 2), f["y"], f["y_err"], "f32", "pieces")
    state, got = h0.clone(), []
    for t in range(150):
        got.append(kla.recurrence_step(*(z[:, :, t].contiguous() for z in (x, g, i)), rate, state, **how))
    near(torch.stack(got, 2), f["y"], f["y_err"], "f32", "steps")
    near(state, f["hT"], f["hT_err"], "f32", "state")


@pytest.mark.parametrize("decay,scale", KINDS)
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,D", [(1, 1, 8), (3, 2, 40), (64, 16, 64)])
def test_step(decay, scale, io, B, H, D):
    x, g, i, rate, h0, _, _ = make(B, H, 1, D, io, decay, seed=D)
    how = {"decay": decay, "scale": scale}
    f = R.forward(*[f64(t) for t in (x, g, i, rate, h0)], **how)
    state = h0.clone()
    y = kla.recurrence_step(*(t[:, :, 0].contiguous() for t in (x, g, i)), rate, state, **how)
    near(y, f["y"][:, :, 0], f["y_err"][:, :, 0], io, "y")
    near(state, f["hT"], f["hT_err"], "f32", "state")


def test_packed_sequences_by_resets():
    """g = -inf begins a sequence: forward and backward are those of the sequences alone."""
    x, g, i, _, _, gy, _ = make(1, 2, 200, 16, "f32", state=False)
    starts = [0, 5, 64, 65, 130, 200]
    g[:, :, starts[:-1]] = -float("inf")
    for scale in ("none", "sqrt", "complement"):
        y, hT = kla.recurrence_forward(x, g, i, scale=scale)
        d = kla.recurrence_backward(x, g, i, gy=gy, scale=scale)
        for a, b in zip(starts, starts[1:]):
            part = [t[:, :, a:b] for t in (x, g, i)]
            f = R.forward(*[f64(t) for t in part], scale=scale)
            near(y[:, :, a:b], f["y"], f["y_err"], "f32", "y")
            want = R.backward(*[f64(t) for t in part], gy=f64(gy[:, :, a:b]), scale=scale)
            for n in ("gx", "gg", "gi"):
                near(d[n][:, :, a:b], want[n], want[n + "_err"], "f32", n)
        near(hT, f["hT"], f["hT_err"], "f32", "hT")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_decays_of_one_and_far_gates(io):
    """a = 1 (g = 0): nothing is written under sqrt and complement; gates far out stay finite, forward and backward."""
    x, g, i, _, h0, gy, ghT = make(1, 2, 90, 16, io)
    g[:, :, 10:20] = 0
    i[:, :, 30:40] = 300.0
    i[:, :, 40:50] = -300.0
    for scale in ("none", "sqrt", "complement"):
        f = R.forward(*[f64(t) for t in (x, g, i)], h0=f64(h0), scale=scale)
        y, hT = kla.recurrence_forward(x, g, i, None, h0, scale=scale)
        near(y, f["y"], f["y_err"], io, "y")
        d = kla.recurrence_backward(x, g, i, None, h0, gy=gy, ghT=ghT, scale=scale)
        want = R.backward(*[f64(t) for t in (x, g, i)], h0=f64(h0), gy=f64(gy), ghT=f64(ghT), scale=scale)
        for n in ("gx", "gg", "gi", "gh0"):
            near(d[n], want[n], want[n + "_err"], "f32" if n == "gh0" else io, n)
    for decay, rate in (("sigmoid", None), ("rate", torch.full((2, 16), 0.05, device=DEV))):
        far = g.clone()
        far[:, :, ::3], far[:, :, 1::3], far[:, :, 2::3] = 200.0, -200.0, 0.5
        for scale in ("none", "sqrt", "complement"):
            y, hT = kla.recurrence_forward(x, far, i, rate, h0, decay=decay, scale=scale)
            d = kla.recurrence_backward(x, far, i, rate, h0, gy=gy, ghT=ghT, decay=decay, scale=scale)
            assert all(bool(t.isfinite().all()) for t in (y, hT, *d.values()))


def test_what_is_no_number_stays_in_its_channel():
    x, g, i, rate, h0, gy, ghT = make(2, 2, 200, 64, "bf16", "rate")
    how = {"decay": "rate", "scale": "sqrt"}
    y, hT = kla.recurrence_forward(x, g, i, rate, h0, **how)
    d = kla.recurrence_backward(x, g, i, rate, h0, gy=gy, ghT=ghT, **how)
    x2, i2, gy2 = x.clone(), i.clone(), gy.clone()
    x2[0, 1, 70, 5], i2[1, 0, 100, 6], gy2[0, 0, 150, 7] = float("nan"), float("nan"), float("inf")
    y2, hT2 = kla.recurrence_forward(x2, g, i2, rate, h0, **how)
    d2 = kla.recurrence_backward(x2, g, i2, rate, h0, gy=gy2, ghT=ghT, **how)
    hit = torch.zeros(2, 2, 64, dtype=torch.bool, device=DEV)
    hit[0, 1, 5] = hit[1, 0, 6] = True
    keep = ~hit[:, :, None].expand_as(y)
    assert torch.equal(y[keep], y2[keep]) and torch.equal(hT[~hit], hT2[~hit])
    assert bool(y2[0, 1, 70:, 5].isnan().all()) and torch.equal(y2[0, 1, :70, 5], y[0, 1, :70, 5])
    hit[0, 0, 7] = True
    keep = ~hit[:, :, None].expand_as(y)
    for n in ("gx", "gg", "gi"):
        assert torch.equal(d[n][keep], d2[n][keep]), n
    assert torch.equal(d["gh0"][~hit], d2["gh0"][~hit])
    channels = ~hit.any(0)
    assert torch.equal(d["grate"][channels], d2["grate"][channels])


def test_strided_views():
    """Slices of one projection, inputs seen several times, gradients of any layout: the bits of contiguous copies."""
    B, T, H, D = 2, 90, 3, 32
    p = torch.randn(B, T, 4 * H * D, device=DEV, dtype=torch.bfloat16)
    x, g, i, gy = (t.unflatten(-1, (H, D)).transpose(1, 2) for t in p.split(H * D, -1))
    g = -g.abs()
    one = p[:, :, :D].unsqueeze(1).expand(B, H, T, D)  # one head seen as three
    for args in ((x, g, i), (x, g, one), (one, g, None)):
        a = kla.recurrence_forward(*args, scale="sqrt")
        b = kla.recurrence_forward(*(None if t is None else t.contiguous() for t in args), scale="sqrt")
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        da = kla.recurrence_backward(*args, gy=gy, scale="sqrt")
        db = kla.recurrence_backward(*(None if t is None else t.contiguous() for t in args), gy=gy.contiguous(), scale="sqrt")
        assert all(torch.equal(da[n], db[n]) for n in db)
    assert kla.recurrence_forward(x, g)[0].transpose(1, 2).is_contiguous()
    out = torch.zeros(B, T, 2 * H * D, device=DEV, dtype=torch.bfloat16)  # into a part of a wider tensor
    y = out[..., H * D:].unflatten(-1, (H, D)).transpose(1, 2)
    kla.recurrence_forward(x, g, i, y=y)
    assert torch.equal(y, kla.recurrence_forward(x, g, i)[0]) and float(out[..., :H * D].abs().max()) == 0


def test_offsets_beyond_32_bits():
    """Tokens 2^30 elements apart."""
    big = torch.empty(3 << 30, dtype=torch.bfloat16, device=DEV)
    far = torch.as_strided(big, (1, 1, 3, 64), (0, 0, 1 << 30, 1))
    far.copy_(torch.randn(1, 1, 3, 64, device=DEV))
    g = -torch.rand(1, 1, 3, 64, device=DEV).bfloat16()
    want = kla.recurrence_forward(far.contiguous(), g)[0]
    assert torch.equal(kla.recurrence_forward(far, g)[0], want)
    y = torch.as_strided(torch.empty(3 << 30, dtype=torch.bfloat16, device=DEV), (1, 1, 3, 64), (0, 0, 1 << 30, 1))
    kla.recurrence_forward(far, g, y=y)
    assert torch.equal(y, want)
    d = kla.recurrence_backward(far, g, gy=y)
    e = kla.recurrence_backward(far.contiguous(), g, gy=want)
    assert all(torch.equal(d[n], e[n]) for n in e)


def test_state_in_place_buffers_and_empty():
    x, g, i, _, h0, _, _ = make(2, 3, 70, 16, "f32")
    y, hT, kept = kla.recurrence_forward(x, g, i, None, h0, checkpoints=True)
    assert torch.equal(kept[0], h0) and kept.shape == (2, 2, 3, 16)
    h, out, buf = h0.clone(), torch.empty_like(y), torch.empty_like(kept)
    got = kla.recurrence_forward(x, g, i, None, h, y=out, hT=h, checkpoints=buf)
    assert got[0] is out and got[1] is h and torch.equal(out, y) and torch.equal(h, hT) and torch.equal(buf, kept)
    assert kla.recurrence_forward(x, g, final_state=False)[1] is None
    none = x[:, :, :0]
    y, hT = kla.recurrence_forward(none, none, none, None, h0)
    assert y.shape == none.shape and torch.equal(hT, h0)
    rate = torch.ones(3, 16, device=DEV)
    d = kla.recurrence_backward(none, none, none, rate, h0, ghT=hT, decay="rate")
    assert torch.equal(d["gh0"], hT) and float(d["grate"].abs().max()) == 0
    none = x[:0]
    y, hT = kla.recurrence_forward(none, none)
    d = kla.recurrence_backward(none, none, None, rate, decay="rate")
    assert y.numel() == hT.numel() == 0 and float(d["grate"].abs().max()) == 0


def test_gradients_without_some_inputs():
    x, g, i, rate, h0, gy, ghT = make(1, 2, 100, 32, "f32", "rate")
    how = {"decay": "rate", "scale": "sqrt"}
    for a, b in ((gy, None), (None, ghT), (None, None)):
        want = R.backward(*[f64(t) for t in (x, g, i, rate, h0)], f64(a), f64(b), **how)
        d = kla.recurrence_backward(x, g, i, rate, h0, gy=a, ghT=b, **how)
        for n in d:
            near(d[n], want[n], want[n + "_err"], "f32", n)


def test_autograd_graph_and_streams():
    x, g, i, rate, h0, gy, ghT = make(2, 4, 300, 64, "bf16", "rate", heads_last=True)
    how = {"decay": "rate", "scale": "sqrt"}
    want = kla.recurrence_forward(x, g, i, rate, h0, **how)
    grads = kla.recurrence_backward(x, g, i, rate, h0, gy=gy, ghT=ghT, **how)
    leaves = [t.detach().requires_grad_() for t in (x, g, i, rate, h0)]
    y, hT = kla.gated_recurrence(*leaves, **how)
    torch.autograd.backward([y, hT], [gy, ghT])
    for t, n in zip(leaves, ("gx", "gg", "gi", "grate", "gh0")):
        assert torch.equal(t.grad, grads[n]), n
    z = x.detach().requires_grad_()
    kla.gated_recurrence(z, g, i, rate, h0, **how)[1].sum().backward()  # through the last state alone
    only = kla.recurrence_backward(x, g, i, rate, h0, ghT=torch.ones_like(ghT), **how)
    assert torch.equal(z.grad, only["gx"])
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs, replayed at the same time
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = kla.recurrence_forward(x, g, i, rate, h0, checkpoints=True, **how)
            back = kla.recurrence_backward(x, g, i, rate, h0, gy=gy, ghT=ghT, checkpoints=out[2], **how)
            alone = kla.recurrence_backward(x, g, i, rate, h0, gy=gy, ghT=ghT, **how)
        graphs.append((graph, out, back, alone))
    side = torch.cuda.Stream()
    for _ in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    for _, out, back, alone in graphs:
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        assert all(torch.equal(back[n], grads[n]) and torch.equal(alone[n], grads[n]) for n in grads)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    got = kla.recurrence_backward(x, g, i, rate, h0, gy=gy, ghT=ghT, stream=side, **how)
    taken = [torch.full((1 << b,), -1, dtype=torch.int8, device=DEV) for b in range(9, 24) for _ in range(2)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(got[n], grads[n]) for n in grads) and all(bool((t == -1).all()) for t in taken)


def test_refusals_of_the_binding():
    x, g, i, rate, h0, _, _ = make(1, 2, 10, 16, "f32", "rate")
    for f, error in ((lambda: kla.recurrence_forward(x, g, i, rate), ValueError),            # a rate that the decay does not take
                     (lambda: kla.recurrence_forward(x, g, i, None, decay="rate"), TypeError),
                     (lambda: kla.recurrence_forward(x, g, decay="linear"), ValueError),
                     (lambda: kla.recurrence_forward(x, g, scale="both"), ValueError),
                     (lambda: kla.recurrence_forward(x, g.bfloat16()), TypeError),
                     (lambda: kla.recurrence_forward(x, g[:, :, 1:]), ValueError),
                     (lambda: kla.recurrence_forward(x.transpose(2, 3), g.transpose(2, 3)), ValueError),
                     (lambda: kla.recurrence_forward(x, g, h0=h0.bfloat16()), TypeError),
                     (lambda: kla.recurrence_forward(x, g, h0=h0[:, :1]), ValueError),
                     (lambda: kla.recurrence_forward(x, g, y=x), kla.KlaError),
                     (lambda: kla.recurrence_forward(x.half(), g.half()), TypeError),
                     (lambda: kla.recurrence_forward(x[..., :4], g[..., :4]), kla.KlaError),
                     (lambda: kla.recurrence_forward(x[..., 2:10], g[..., 2:10]), kla.KlaError),   # off 16 bytes
                     (lambda: kla.recurrence_step(x[:, :, 0], g[:, :, 0], None, None, h0), ValueError),  # not contiguous
                     (lambda: kla.recurrence_backward(x, g, checkpoints=h0), ValueError),
                     (lambda: kla.recurrence_backward(x, g, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)),
                      kla.KlaError),
                     (lambda: kla.recurrence_backward(x, g, workspace=torch.empty(1 << 20, dtype=torch.uint8)), ValueError)):
        with pytest.raises(error):
            f()
    torch.cuda.synchronize()
