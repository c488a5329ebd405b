"""A caller's workspace is written to by the kernels as it is, so one that is not
contiguous memory of the inputs' device is turned down."""
from types import SimpleNamespace

import pytest
import torch

from bayesian_filtering_linear_gb300 import kla

DEV = "cuda:0"


class Elsewhere(torch.Tensor):
    """A tensor that says it is on a CUDA device."""

    @staticmethod
    def __new__(cls, x, index):
        y = x.as_subclass(cls)
        y.index = index
        return y

    def get_device(self):
        return self.index


def test_bytes_of_a_workspace():
    x = torch.zeros(6, 4, dtype=torch.float32)
    assert kla._space(None, 0) == 0 and kla._space(Elsewhere(x, 0), 0) == 96
    for bad, error in ((x, ValueError), (Elsewhere(x, 1), ValueError), (Elsewhere(x[:, ::2], 0), ValueError),
                       (Elsewhere(x.t(), 0), ValueError), (SimpleNamespace(numel=lambda: 1), TypeError)):
        with pytest.raises(error):
            kla._space(bad, 0)


def calls():
    r = lambda *s: torch.rand(*s, device=DEV)
    x, g, n = [r(1, 2, 600, 16) for _ in range(6)], r(1, 2, 600), r(2, 3, 5, 64)
    w = torch.ones(64, device=DEV)
    return {"forward": lambda ws: kla.forward(*x, strategy="chunked", workspace=ws),
            "backward": lambda ws: kla.backward(*x, gy=x[0], workspace=ws),
            "conv_backward": lambda ws: kla.conv_backward(x[0], r(2, 16, 4), gy=x[0], workspace=ws),
            "delta_forward": lambda ws: kla.delta_forward(*x[:3], -g, g, workspace=ws),
            "delta_backward": lambda ws: kla.delta_backward(*x[:3], -g, g, go=x[0], workspace=ws),
            "norm_rope_backward": lambda ws: kla.norm_rope_backward(n, n, w, w, gyq=n, gyk=n, workspace=ws)}


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["forward", "backward", "conv_backward", "delta_forward", "delta_backward",
                                  "norm_rope_backward"])
def test_every_call_refuses(name):
    call = calls()[name]
    big = 1 << 26
    call(torch.empty(big, dtype=torch.uint8, device=DEV))
    for bad in (torch.empty(big, dtype=torch.uint8), torch.empty(2 * big, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError):
            call(bad)
    with pytest.raises(kla.KlaError):
        call(torch.empty(16, dtype=torch.uint8, device=DEV))  # too small
    torch.cuda.synchronize()
