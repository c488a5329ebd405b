"""Threads whose scans and gradients share a kernel at different widths, and so ask for different amounts of shared memory:
every call succeeds, with the results of the same calls one after the other."""
import ctypes
import threading

import pytest
import torch

from bayesian_filtering_linear_gb300 import kla
from bayesian_filtering_linear_gb300.inputs import make_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B, H, T = 8, 16, 70
CALLS = 1500


def tensors(dk, dv, dtype, chunk_len):
    drawn = make_inputs(B, H, T, dk, dv, io="bf16" if dtype == torch.bfloat16 else "f32", seed=dk + dv, device=DEV)
    x = [drawn[n] for n in ("q", "k", "v", "lam_v", "a", "pbar")]
    gy = torch.randn(B, H, T, dv, device=DEV).to(dtype)
    io = kla.BF16 if dtype == torch.bfloat16 else kla.F32
    how = {} if chunk_len == 0 else {"strategy": "chunked", "chunk_len": chunk_len}
    y, lamT, etaT = kla.forward(*x, **how)
    g = kla.backward(*x, gy=gy, state_grads=False)
    torch.cuda.synchronize()
    opt = kla.options(**how)
    info = kla.PlanInfo()
    assert kla.LIB.kla_plan(B, H, T, dk, dv, io, ctypes.byref(opt), ctypes.byref(info)) == kla.OK
    ws = torch.empty(max(int(info.workspace_bytes), 16), dtype=torch.uint8, device=DEV)
    bws = torch.empty(kla.LIB.kla_backward_workspace_size(B, H, T, dk, dv), dtype=torch.uint8, device=DEV)
    out = [torch.empty_like(t) for t in (y, lamT, etaT)]
    back = {n: torch.empty_like(t) for n, t in g.items()}
    p, none = (lambda t: ctypes.c_void_p(t.data_ptr())), None
    stream = torch.cuda.Stream()
    s = ctypes.c_void_p(stream.cuda_stream)
    forward = [*map(p, x), none, none, *map(p, out), B, H, T, dk, dv, io, p(ws), ws.numel(), ctypes.byref(opt), s]
    backward = [*map(p, x), none, none, p(gy), none, none, *(p(back[n]) for n in ("gq", "gk", "gv", "glam_v", "ga", "gpbar")),
                none, none, B, H, T, dk, dv, io, 0, p(bws), bws.numel(), s]
    keep = (x, gy, ws, bws, opt, stream)
    return forward, backward, out, back, (y, lamT, etaT), g, keep


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,widths", [(128, [16, 32, 128]), (16, [16, 32, 64]), (64, [16, 32, 64])])
@pytest.mark.parametrize("chunk_len", [0, 32])
def test_widths_of_one_kernel(dtype, dk, widths, chunk_len):
    work = [tensors(dk, dv, dtype, chunk_len) for dv in widths * 2]
    ready, bad = threading.Barrier(len(work)), []

    def run(forward, backward, *_):
        ready.wait()
        for _ in range(CALLS):
            st = kla.LIB.kla_forward(*forward), kla.LIB.kla_backward(*backward)
            if st != (kla.OK, kla.OK):
                bad.append(st)
                break

    threads = [threading.Thread(target=run, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, bad
    for _, _, out, back, want, g, _ in work:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        # sums by atomics, whose order varies: of 128 terms, 2^-24 of the sum of their sizes each, which may be 2^5 times the
        # sum; in bf16 half a step of either result
        for n in back:
            off = (back[n].double() - g[n].double()).norm() / g[n].double().norm()
            assert float(off) <= (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -12), n
