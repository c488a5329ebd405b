"""The recurrence and the layer norm where nothing was called before: the first calls of a process inside a captured
graph, and many threads at once with streams of their own."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from bayesian_filtering_linear_gb300 import kla

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST = """
import torch
from bayesian_filtering_linear_gb300 import kla
x, g, i, gy = (torch.randn(1, 2, 300, 64, device="cuda") for _ in range(4))
rate, w = torch.rand(2, 64, device="cuda"), torch.ones(64, device="cuda")
def step():
    n, total = kla.layer_norm(x, w, w, gy)
    y, hT, kept = kla.recurrence_forward(n, g, i, rate, decay="rate", scale="sqrt", checkpoints=True)
    d = kla.recurrence_backward(n, g, i, rate, gy=gy, decay="rate", scale="sqrt", checkpoints=kept)
    e = kla.layer_norm_backward(total, w, gy=d["gx"], gtotal=gy)
    return [y, hT, *d.values(), *e.values()]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
print("same")
"""


def test_first_calls_are_captured():
    out = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "same" in out.stdout, out.stderr[-2000:]


def test_many_threads():
    """Eight threads, each with its own stream, shapes and kinds: the results of the same calls one after the other."""
    kinds = [("log", "none"), ("log", "sqrt"), ("sigmoid", "complement"), ("rate", "sqrt")] * 2
    work = []
    for n, (decay, scale) in enumerate(kinds):
        r = torch.Generator(device=DEV).manual_seed(n)
        x, g, i, gy = (torch.randn(1 + n % 3, 2, 150 + 40 * n, 64, generator=r, device=DEV) for _ in range(4))
        rate = torch.rand(2, 64, generator=r, device=DEV) if decay == "rate" else None
        work.append((x, -g.abs() if decay == "log" else g, i, rate, gy, {"decay": decay, "scale": scale}))

    def call(x, g, i, rate, gy, how):
        y, hT = kla.recurrence_forward(x, g, i, rate, **how)
        d = kla.recurrence_backward(x, g, i, rate, gy=gy, **how)
        n, total = kla.layer_norm(y, None, None, gy)
        return [y, hT, *d.values(), n, kla.layer_norm_backward(total, gy=gy, param_grads=True)["gweight"]]

    want = [call(*a) for a in work]
    torch.cuda.synchronize()
    got, errors = [None] * len(work), []

    def run(n):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got[n] = call(*work[n])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(n,)) for n in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert all(torch.equal(a, b) for u, v in zip(got, want) for a, b in zip(u, v))
