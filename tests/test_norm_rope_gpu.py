"""The norm of queries and keys with the rotation, against the fp64 oracle.

Tolerances: the sum of squares and the row's product with gy are sums of D fp32
terms (√D · 2^-24 of the value, sixteen for the worst element), the angle is
known to a few 2^-24 of a turn (2π · 4 · 2^-24 of the row's largest entry), and
a weight's gradient adds a sum over all rows in quadrature. bf16 outputs are off
by half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

from bayesian_filtering_linear_gb300 import kla
from oracle import norm_rope as N

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(x):
    return x.detach().double().cpu().numpy()


def near(got, want, io, D, what, terms=0):
    top = np.abs(want).max(-1, keepdims=True) if terms == 0 else np.abs(want).max()
    tol = (16 * np.sqrt(D + terms) + 8 * np.pi) * 2.0 ** -24 * (1.5 * top + 1e-6 * np.abs(want).max())
    err = np.abs(f64(got) - want)
    if io == "bf16":
        err = err - 2.0 ** -8 * np.abs(want)
    assert (err <= tol + 1e-30).all(), f"{what}: {(err - tol).max():.3g} over (largest {np.abs(want).max():.3g})"


def run(B, Hq, Hk, T, D, io, norm="rms", layout="half", rot=None, weights=True, heads_last=False, start=0, eps=1e-6,
        rot_scale=1.0, positions=True, seed=0):
    r = torch.Generator().manual_seed(seed)
    rot = D if rot is None else rot

    def rows(h):
        x = torch.randn(B, T, h, D, generator=r) if heads_last else torch.randn(B, h, T, D, generator=r)
        x = x.to(DT[io]).to(DEV)
        return x.transpose(1, 2) if heads_last else x

    q, k = rows(Hq), rows(Hk)
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=r)).to(DEV) for _ in range(2)) if weights else (None, None)
    freq = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(rot // 2, 1))).float().to(DEV) if rot else None
    pos = start + torch.arange(T) + 3 * torch.arange(B)[:, None]
    kw = {"norm": norm, "layout": layout, "eps": eps, "rot_scale": rot_scale}
    if positions:
        kw["positions"] = pos.to(DEV)
    else:
        pos = (start + torch.arange(T)).expand(B, T)
        kw["offset"] = start
    gyq, gyk = (torch.randn(B, h, T, D, generator=r).to(DT[io]).to(DEV) for h in (Hq, Hk))
    yq, yk = kla.norm_rope(q, k, wq, wk, freq, **kw)
    g = kla.norm_rope_backward(q, k, wq, wk, freq, gyq=gyq, gyk=gyk, **kw)
    f = np.zeros(0) if freq is None else f64(freq)
    for n, x, w, y, gy in (("q", q, wq, yq, gyq), ("k", k, wk, yk, gyk)):
        w64 = np.ones(D) if w is None else f64(w)
        how = (pos.numpy(), f, norm, layout, eps, rot_scale)
        near(y, N.forward(f64(x), w64, *how), io, D, "y" + n)
        gx, gw = N.backward(f64(x), w64, f64(gy), *how)
        near(g["g" + n], gx, io, D, "g" + n)
        if w is not None:
            near(g[f"g{n}_weight"], gw, "f32", D, f"g{n}_weight", terms=B * T * x.shape[1])
        assert y.is_contiguous() and g["g" + n].shape == x.shape
    return q, k, wq, wk, freq, kw, gyq, gyk, yq, yk, g


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("part", [0, 2, 6, "quarter", "half", "all"])
def test_sizes_layouts_and_parts(io, D, layout, part):
    rot = {"quarter": D // 4, "half": D // 2, "all": D}.get(part, part)
    run(2, 3, 1, 5, D, io, layout=layout, rot=rot, seed=D)


@pytest.mark.parametrize("norm", ["none", "rms", "l2"])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("weights", [True, False])
def test_norms_and_weights(norm, io, weights):
    run(1, 4, 2, 67, 64, io, norm=norm, weights=weights, heads_last=True, rot_scale=1.25)


@pytest.mark.parametrize("B,Hq,Hk,T", [(1, 1, 1, 1), (33, 16, 4, 1), (1, 2, 2, 1027), (3, 5, 3, 100)])
def test_shapes(B, Hq, Hk, T):
    run(B, Hq, Hk, T, 64, "bf16", heads_last=True)
    run(B, Hq, Hk, T, 32, "f32", positions=False, start=11)


@pytest.mark.parametrize("start", [-1000, 1 << 20, 1000003, (1 << 31) - 7, (1 << 33) + 12345])
def test_far_positions_are_as_exact_as_near_ones(start):
    run(1, 2, 1, 9, 64, "f32", start=start)
    run(1, 2, 1, 9, 64, "f32", start=start, positions=False, layout="interleaved")


def test_rows_of_zeros_and_tiny_and_large_rows():
    q = torch.zeros(1, 1, 4, 64, device=DEV)
    q[0, 0, 1] = 1e-12
    q[0, 0, 2] = 1e15
    q[0, 0, 3, 5] = 1
    y, none = kla.norm_rope(q, norm="l2")
    assert none is None and bool(y.isfinite().all()) and float(y[0, 0, 0].abs().max()) == 0
    assert torch.allclose(y[0, 0, 2], torch.full((64,), 0.125, device=DEV))
    g = kla.norm_rope_backward(q, gyq=torch.ones_like(q), norm="l2")["gq"]
    assert bool(g.isfinite().all()) and torch.allclose(g[0, 0, 0], torch.full((64,), 1e3, device=DEV))


def test_strided_views_of_one_projection():
    """q and k as slices of a fused projection: rows far apart, in place."""
    x = torch.randn(2, 7, (4 + 2 + 2) * 64, device=DEV, dtype=torch.bfloat16)
    q = x[..., :256].unflatten(-1, (4, 64)).transpose(1, 2)
    k = x[..., 256:384].unflatten(-1, (2, 64)).transpose(1, 2)
    f, s = kla.rope_frequencies(64, device=DEV)
    a = kla.norm_rope(q, k, None, None, f, rot_scale=s)
    b = kla.norm_rope(q.contiguous(), k.contiguous(), None, None, f)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    gy = torch.randn_like(a[0])
    ga = kla.norm_rope_backward(q, k, None, None, f, gyq=gy)
    gb = kla.norm_rope_backward(q.contiguous(), k.contiguous(), None, None, f, gyq=gy)
    assert torch.equal(ga["gq"], gb["gq"]) and float(ga["gk"].abs().max()) == 0
    assert ga["gq"].transpose(1, 2).is_contiguous()
    same = k[:, :1].expand(2, 3, 7, 64)  # one head seen as three
    assert torch.equal(kla.norm_rope(same, None, None, None, f)[0][:, 2], a[1][:, 0])
    with pytest.raises(kla.KlaError):
        kla.norm_rope(x[..., 4:68].unflatten(-1, (1, 64)).transpose(1, 2))  # off 16 bytes
    with pytest.raises(ValueError):
        kla.norm_rope(q.transpose(2, 3))


def test_empty():
    f, _ = kla.rope_frequencies(64, device=DEV)
    q = torch.empty(2, 3, 0, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    assert kla.norm_rope(q, q, w, w, f)[0].shape == q.shape
    g = kla.norm_rope_backward(q, q, w, w, f)
    assert float(g["gq_weight"].abs().max()) == 0 and float(g["gk_weight"].abs().max()) == 0


def test_one_row_that_is_no_number_stays_alone():
    x = torch.randn(1, 2, 8, 64, device=DEV)
    a = kla.norm_rope(x)[0]
    x[0, 1, 3, 0] = float("inf")
    b = kla.norm_rope(x)[0]
    keep = torch.ones(2, 8, dtype=torch.bool, device=DEV)
    keep[1, 3] = False
    assert torch.equal(a[0][keep], b[0][keep]) and not bool(b[0, 1, 3].isfinite().all())


def test_autograd_repeats_and_graph():
    q, k, wq, wk, f, kw, gyq, gyk, yq, yk, g = run(2, 4, 2, 300, 64, "bf16", heads_last=True)
    leaves = [x.detach().requires_grad_() for x in (q, k, wq, wk)]
    a, b = kla.qk_norm_rope(*leaves, f, **kw)
    torch.autograd.backward([a, b], [gyq, gyk])
    for x, n in zip(leaves, ("gq", "gk", "gq_weight", "gk_weight")):
        assert torch.equal(x.grad, g[n]), n
    torch.cuda.synchronize()
    ws = torch.empty(kla.LIB.kla_norm_rope_backward_workspace_size(2, 4, 2, 300, 64), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kla.norm_rope(q, k, wq, wk, f, **kw)
        back = kla.norm_rope_backward(q, k, wq, wk, f, gyq=gyq, gyk=gyk, workspace=ws, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], yq) and torch.equal(out[1], yk)
    assert all(torch.equal(back[n], g[n]) for n in g)
