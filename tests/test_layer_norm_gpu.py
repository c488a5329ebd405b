"""The layer norm with the residual sum against the fp64 oracle, which also gives
the bound that arithmetic in 24 bits keeps (see there). bf16 outputs are off by
half a step more, 2^-8 of the value and of the bound."""
import numpy as np
import pytest
import torch

from bayesian_filtering_linear_gb300 import kla
from oracle import layer_norm as N

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(got, want, err, io, what):
    tol = err + (2.0 ** -8 * (np.abs(want) + err) if io == "bf16" else 0) + 1e-36
    off = np.abs(f64(got) - want)
    assert (off <= tol).all(), f"{what}: {np.nanmax(off / tol):.3g} of the bound (largest {np.abs(want).max():.3g})"


def make(rows, D, io, seed=0, offset=0.0):
    r = torch.Generator().manual_seed(seed + D)
    x, res, gy, gt = (torch.randn(rows, D, generator=r).to(DT[io]).to(DEV) for _ in range(4))
    x = (x.float() * (1 + 8 * (torch.rand(D, generator=r) < 0.05).to(DEV)) + offset).to(DT[io])
    w, b = ((k + 0.3 * torch.randn(D, generator=r)).to(DEV) for k in (1, 0))
    return x, res, gy, gt, w, b


def check(rows, D, io, weight=True, bias=True, residual=True, **kw):
    x, res, gy, gt, w, b = make(rows, D, io, **kw)
    w, b, res, gt = w if weight else None, b if bias else None, res if residual else None, gt if residual else None
    y, total = kla.layer_norm(x, w, b, res)
    if residual:
        assert torch.equal(total, (x.float() + res.float()).to(x.dtype))
    else:
        assert total is None
        total = x
    want, err = N.forward(f64(total), f64(w), f64(b))
    near(y, want, err, io, "y")
    d = kla.layer_norm_backward(total, w, gy=gy, gtotal=gt, param_grads=True)
    e = N.backward(f64(total), f64(w), f64(gy), f64(gt))
    near(d["gx"], e["gx"], e["gx_err"], io, "gx")
    near(d["gweight"], e["gweight"], e["gweight_err"], "f32", "gweight")
    near(d["gbias"], e["gbias"], e["gbias_err"], "f32", "gbias")
    again = kla.layer_norm_backward(total, w, gy=gy, gtotal=gt, param_grads=False)
    assert set(again) == {"gx"} and torch.equal(again["gx"], d["gx"])


WIDTHS = [1, 2, 7, 8, 16, 63, 64, 65, 72, 128, 136, 256, 264, 500, 512, 520, 1000, 1024, 1025, 1032, 2000, 2048, 2056,
          4096, 4100, 4104, 5001, 8184, 8191, 8192]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_widths(D, io):
    check(9, D, io)


@pytest.mark.parametrize("rows", [1, 2, 3, 33, 1000, 5003])
@pytest.mark.parametrize("D", [24, 200, 517, 1024])
def test_rows(rows, D):
    check(rows, D, "bf16", seed=rows)
    check(rows, D, "f32", seed=rows, residual=False)


@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("residual", [True, False])
def test_parts(weight, bias, residual):
    check(50, 320, "bf16", weight, bias, residual)
    check(50, 33, "f32", weight, bias, residual)


def test_rows_far_from_zero():
    """A mean a thousand times the spread: as exact as the sums allow."""
    check(40, 512, "f32", offset=1000.0, residual=False)
    check(40, 512, "f32", offset=-30.0)


def test_constant_and_tiny_rows():
    x = torch.full((3, 96), 5.0, device=DEV)
    x[1] = 0
    w, b = torch.ones(96, device=DEV), torch.full((96,), 0.25, device=DEV)
    y, _ = kla.layer_norm(x, w, b)
    assert float((y[1] - 0.25).abs().max()) == 0 and float((y - 0.25).abs().max()) < 1e-3
    d = kla.layer_norm_backward(x, w, gy=torch.randn_like(x))
    assert bool(d["gx"].isfinite().all())
    one = torch.randn(5, 1, device=DEV)
    assert float(kla.layer_norm(one)[0].abs().max()) == 0


def test_a_row_that_is_no_number_stays_alone():
    x, res, gy, gt, w, b = make(70, 200, "bf16")
    y, total = kla.layer_norm(x, w, b, res)
    gx = kla.layer_norm_backward(total, w, gy=gy, gtotal=gt)["gx"]
    x[3, 5], x[60, 199] = float("inf"), float("nan")
    y2, total2 = kla.layer_norm(x, w, b, res)
    gx2 = kla.layer_norm_backward(total2, w, gy=gy, gtotal=gt)["gx"]
    keep = torch.ones(70, dtype=torch.bool, device=DEV)
    keep[[3, 60]] = False
    assert torch.equal(y[keep], y2[keep]) and torch.equal(gx[keep], gx2[keep])
    assert not bool(y2[~keep].isfinite().any())


def test_strided_rows_shapes_and_in_place():
    x, res, gy, gt, w, b = make(24, 136, "bf16")
    want, total = kla.layer_norm(x, w, b, res)
    grads = kla.layer_norm_backward(total, w, gy=gy, gtotal=gt)
    wide = torch.randn(24, 5, 136, device=DEV).bfloat16()
    wide[:, 2] = x
    a, t = kla.layer_norm(wide[:, 2], w, b, res)  # every fifth row
    assert torch.equal(a, want) and torch.equal(t, total)
    odd = torch.randn(24, 137, device=DEV).bfloat16()
    odd[:, 1:] = x
    a, t = kla.layer_norm(odd[:, 1:], w, b, res)  # rows off 16 bytes: element by element, the sums in another order
    assert torch.equal(t, total) and float((a.float() - want.float()).abs().max()) <= 2.0 ** -7 * float(want.abs().max())
    same = res[:1].expand(24, 136)
    assert torch.equal(kla.layer_norm(x, w, b, same)[0], kla.layer_norm(x, w, b, same.contiguous())[0])
    deep = [z.view(2, 3, 4, 136) for z in (x, res, gy, gt)]
    a, t = kla.layer_norm(deep[0], w, b, deep[1])
    assert a.shape == deep[0].shape and torch.equal(a.view(24, 136), want)
    d = kla.layer_norm_backward(t, w, gy=deep[2], gtotal=deep[3])
    assert d["gx"].shape == deep[0].shape and all(torch.equal(d[n].flatten(), grads[n].flatten()) for n in grads)
    assert torch.equal(kla.layer_norm(x[0], w, b, res[0])[0], want[0])
    with pytest.raises(ValueError):
        kla.layer_norm(deep[0].transpose(1, 2), w, b)
    u, v = x.clone(), res.clone()
    a, t = kla.layer_norm(u, w, b, v, y=u, total=v)
    assert a is u and t is v and torch.equal(u, want) and torch.equal(v, total)
    u, v = x.clone(), res.clone()
    kla.layer_norm(u, w, b, v, y=v, total=u)
    assert torch.equal(v, want) and torch.equal(u, total)
    with pytest.raises(kla.KlaError):
        kla.layer_norm(wide[:12].view(60, 136)[1:37], w, b, y=wide.view(120, 136)[:36])
    with pytest.raises(kla.KlaError):
        kla.layer_norm(x, w, b, res, y=u, total=u)


def test_empty():
    x = torch.empty(0, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    y, total = kla.layer_norm(x, w, w, x)
    assert y.shape == total.shape == x.shape
    d = kla.layer_norm_backward(x, w, gy=x)
    assert d["gx"].shape == x.shape and float(d["gweight"].abs().max()) == 0 and float(d["gbias"].abs().max()) == 0


def test_offsets_beyond_32_bits():
    far = torch.as_strided(torch.empty(3 << 30, dtype=torch.bfloat16, device=DEV), (3, 64), (1 << 30, 1))
    far.copy_(torch.randn(3, 64, device=DEV))
    near_ = far.contiguous()
    assert torch.equal(kla.layer_norm(far)[0], kla.layer_norm(near_)[0])
    a, b = (kla.layer_norm_backward(t, gy=t, gtotal=t)["gx"] for t in (far, near_))
    assert torch.equal(a, b)


def test_autograd_graph_and_streams():
    x, res, gy, gt, w, b = make(300, 256, "bf16")
    want, total = kla.layer_norm(x, w, b, res)
    grads = kla.layer_norm_backward(total, w, gy=gy, gtotal=gt)
    leaves = [t.detach().requires_grad_() for t in (x, w, b, res)]
    y, t = kla.add_layer_norm(*leaves)
    torch.autograd.backward([y, t], [gy, gt])
    for z, n in zip(leaves, ("gx", "gweight", "gbias", "gx")):
        assert torch.equal(z.grad, grads[n]), n
    leaves[0].grad.zero_()
    assert torch.equal(leaves[3].grad, grads["gx"])  # not one tensor for both
    only = x.detach().requires_grad_()
    kla.add_layer_norm(only, w, b)[0].backward(gy)
    assert torch.equal(only.grad, kla.layer_norm_backward(x, w, gy=gy)["gx"])
    just_total = x.detach().requires_grad_()
    kla.add_layer_norm(just_total, w, b, res)[1].backward(gt)
    assert torch.equal(just_total.grad, gt)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = kla.layer_norm(x, w, b, res)
            back = kla.layer_norm_backward(out[1], w, gy=gy, gtotal=gt)
        graphs.append((graph, out, back))
    side = torch.cuda.Stream()
    for _ in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    for _, out, back in graphs:
        assert torch.equal(out[0], want) and all(torch.equal(back[n], grads[n]) for n in grads)
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    got = kla.layer_norm_backward(total, w, gy=gy, gtotal=gt, stream=side)
    taken = [torch.full((1 << b,), -1, dtype=torch.int8, device=DEV) for b in range(9, 24) for _ in range(2)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(got[n], grads[n]) for n in grads) and all(bool((t == -1).all()) for t in taken)


def test_refusals_of_the_binding():
    x, res, gy, gt, w, b = make(8, 64, "f32")
    for f, error in ((lambda: kla.layer_norm(x, w[:32]), ValueError), (lambda: kla.layer_norm(x, w.bfloat16()), TypeError),
                     (lambda: kla.layer_norm(x, w, b, res[:4]), ValueError), (lambda: kla.layer_norm(x.half()), TypeError),
                     (lambda: kla.layer_norm(x, w, b, res.bfloat16()), TypeError),
                     (lambda: kla.layer_norm(x, w, b, total=x), ValueError), (lambda: kla.layer_norm(x, eps=-1.0), kla.KlaError),
                     (lambda: kla.layer_norm(x.cpu()), ValueError), (lambda: kla.layer_norm(x[:, :0]), ValueError),
                     (lambda: kla.layer_norm(torch.zeros(2, 8200, device=DEV)), kla.KlaError),
                     (lambda: kla.layer_norm(x.t()), ValueError),
                     (lambda: kla.layer_norm_backward(x, w, gy=gy[:4]), ValueError),
                     (lambda: kla.layer_norm_backward(x, w, gy=gy, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)),
                      kla.KlaError),
                     (lambda: kla.layer_norm_backward(x, w, gy=gy, workspace=torch.empty(1 << 22, dtype=torch.uint8)), ValueError)):
        with pytest.raises(error):
            f()
    torch.cuda.synchronize()
