"""The layer norm at the widths around which the kernels share a row out differently, where rows begin on 16 bytes, on
four and on neither."""
import pytest
import torch
from test_layer_norm_gpu import DEV, check

from bayesian_filtering_linear_gb300 import kla

pytestmark = pytest.mark.gpu
AROUND = [32, 64, 128, 256, 384, 512, 640, 768, 1024, 2048, 4096]
WIDTHS = sorted({w + d for w in AROUND for d in (-1, 0, 1)} | {2 * w + d for w in AROUND for d in (-2, 2)} - {8194})


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_widths(D, io):
    check(21, D, io, residual=D % 4 < 2)


@pytest.mark.parametrize("D", [50, 446, 1030, 4098])
def test_many_rows(D):
    check(2500, D, "bf16")


@pytest.mark.parametrize("first,gap", [(0, 8), (2, 2), (1, 2), (2, 3), (4, 4)])
def test_rows_that_begin_anywhere(first, gap):
    """Views of columns: the bytes that rows begin on choose the pieces, the results stay."""
    D, rows = 128, 37
    r = torch.Generator().manual_seed(1)
    wide = [torch.randn(rows, D + first + gap, generator=r).to(torch.bfloat16).to(DEV) for _ in range(4)]
    x, res, gy, gt = (t[:, first:first + D] for t in wide)
    w = torch.rand(D, generator=r).to(DEV)
    y, total = kla.layer_norm(x, w, w, res)
    d = kla.layer_norm_backward(x, w, gy=gy, gtotal=gt, param_grads=True)
    y1, total1 = kla.layer_norm(x.contiguous(), w, w, res.contiguous())
    d1 = kla.layer_norm_backward(x.contiguous(), w, gy=gy.contiguous(), gtotal=gt.contiguous(), param_grads=True)
    assert torch.equal(total, total1)
    # the sums' order depends on the pieces: a step of bf16 apart at most; a sum over 37 rows of |g n| < 16, of which
    # each is off by the order of the sums of 128 in n, under 26 units of 2^-24 of it
    torch.testing.assert_close(y.float(), y1.float(), rtol=2.0 ** -7, atol=1e-5)
    torch.testing.assert_close(d["gx"].float(), d1["gx"].float(), rtol=2.0 ** -7, atol=1e-4)
    for n in ("gweight", "gbias"):
        torch.testing.assert_close(d[n], d1[n], rtol=0, atol=128 * 128 * 2.0 ** -24)
