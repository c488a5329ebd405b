"""Threads whose layer norm gradients share a kernel at different widths, and so ask for different amounts of shared memory:
every call succeeds, with the results of the same calls one after the other."""
import threading

import pytest
import torch

from bayesian_filtering_linear_gb300 import kla

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype,widths", [(torch.bfloat16, [520, 768, 1024, 640]), (torch.float32, [516, 768, 1024, 640]),
                                          (torch.float32, [260, 384, 512, 300])])
def test_widths_of_one_kernel(dtype, widths):
    r = torch.Generator(device=DEV).manual_seed(0)
    io = kla.BF16 if dtype == torch.bfloat16 else kla.F32
    work = []
    for D in widths * 2:
        x, gy = (torch.randn(3, D, generator=r, device=DEV).to(dtype) for _ in range(2))
        gx, gw, gb = torch.empty_like(x), torch.empty(D, device=DEV), torch.empty(D, device=DEV)
        space = torch.empty(kla.LIB.kla_layer_norm_backward_workspace_size(3, D), dtype=torch.uint8, device=DEV)
        work.append((D, x, gy, gx, gw, gb, space, torch.cuda.Stream(), kla.layer_norm_backward(x, gy=gy, param_grads=True)))
    torch.cuda.synchronize()
    ready, bad = threading.Barrier(len(work)), []

    def run(D, x, gy, gx, gw, gb, space, stream, _):
        args = (x.data_ptr(), None, gy.data_ptr(), None, gx.data_ptr(), gw.data_ptr(), gb.data_ptr(), 3, D, D, D, 0, io, 1e-5,
                space.data_ptr(), space.numel(), stream.cuda_stream)
        ready.wait()
        for _ in range(4000):
            st = kla.LIB.kla_layer_norm_backward(*args)
            if st != kla.OK:
                bad.append((D, st))
                break

    threads = [threading.Thread(target=run, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, bad
    for D, x, gy, gx, gw, gb, space, stream, want in work:
        assert torch.equal(gx, want["gx"]) and torch.equal(gw, want["gweight"]) and torch.equal(gb, want["gbias"]), D
