"""What the delta rule's chunked kernels leave when a wait runs out: outputs that
came of it are no numbers, whichever threads of a block noticed.

No wait is made to run out: tests/host/delta_waits.cu builds the kernels so that
every wait ends as ever, but counts as run out for chosen threads."""
import ctypes
import os
import subprocess

import pytest
import torch

from bayesian_filtering_linear_gb300 import build, kla
from test_delta_gpu import DEV, problem, to_dev

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
# the chain's threads in bf16: eight warps keep the state, four bring K and W, one issues the products
CHAIN = {"a state's thread": (37, 38), "the feeding warps": (256, 384), "one feeding thread": (300, 301),
         "the issuing warp": (384, 416)}


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("waits") / "delta_waits.so")
    subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-shared", "-o", out,
                    os.path.join(HERE, "host", "delta_waits.cu")], check=True)
    lib = ctypes.CDLL(out)
    lib.delta_waits_bytes.restype = ctypes.c_size_t
    return lib


def run(lib, p, backward, stage=0, threads=(0, 0), sms=1):
    B, Hk, T, dk = p["k"].shape
    H, dv = p["v"].shape[1], p["v"].shape[-1]
    new = lambda n: torch.zeros_like(p[n])
    space = torch.zeros(lib.delta_waits_bytes(B, Hk, H, T, dk, dv), dtype=torch.uint8, device=DEV)
    if backward:
        out = {"gq": new("q"), "gk": new("k"), "gv": new("v"), "gg": new("g"), "gbeta": new("beta"), "gstate0": new("state0")}
        outs = [None, None, p["v"], *out.values()]
    else:
        out = {"o": new("v"), "stateT": new("state0")}
        outs = [*out.values(), *[None] * 7]
    ptr = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())
    torch.cuda.synchronize()
    rc = lib.delta_waits(*(ptr(p[n]) for n in ("q", "k", "v", "g", "beta", "state0")), *map(ptr, outs), B, Hk, H, T, dk, dv,
                         ptr(space), sms, stage, *threads)
    assert rc == 0
    return out


def nan(x):
    return bool(x.isnan().all())


# sms: with one SM blocks of 64 columns run, with many those of 32
@pytest.mark.parametrize("sms", [1, 1000])
@pytest.mark.parametrize("Hk,H,dk,dv", [(2, 2, 64, 64), (1, 2, 32, 128), (1, 1, 64, 16)])
def test_outputs_are_marked(lib, Hk, H, dk, dv, sms):
    p = to_dev(problem(1, Hk, H, 150, dk, dv, "bf16", seed=3))
    args = [p[n] for n in ("q", "k", "v", "g", "beta", "state0")]
    clean = run(lib, p, False, sms=sms)
    o, last = kla.delta_forward(*args, scale=1.0)
    assert float((clean["o"].float() - o.float()).abs().max()) <= 2.0 ** -7 * float(o.float().abs().max())
    assert bool(clean["stateT"].isfinite().all())
    grads = run(lib, p, True, sms=sms)
    assert all(bool(x.isfinite().all()) for x in grads.values())
    for threads in ((37, 38), (255, 256)):
        got = run(lib, p, False, 0, threads, sms)
        assert nan(got["o"]) and nan(got["stateT"]), ("prepare", threads)
        got = run(lib, p, False, 2, threads, sms)
        assert nan(got["o"]) and torch.equal(got["stateT"], clean["stateT"]), ("output", threads)
        got = run(lib, p, True, 0, threads, sms)
        assert all(map(nan, got.values())), ("prepare", threads)
        got = run(lib, p, True, 2, threads, sms)
        for n in ("gstate0", "gv"):  # made of what the chain left alone
            assert torch.equal(got.pop(n), grads[n]), n
        assert all(map(nan, got.values())), ("gradients", threads)
    for name, threads in CHAIN.items():
        got = run(lib, p, False, 1, threads, sms)
        assert nan(got["o"]) and nan(got["stateT"]), (name, {n: int(x.isnan().sum()) for n, x in got.items()})
        got = run(lib, p, True, 1, threads, sms)
        assert all(map(nan, got.values())), (name, {n: int(x.isnan().sum()) for n, x in got.items()})
