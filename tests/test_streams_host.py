"""Calls with ``stream=``: everything that such a call allocates is allocated
under that stream, and what it returns is kept for the caller's stream too."""
import contextlib
import inspect
from types import SimpleNamespace

import pytest
import torch

from bayesian_filtering_linear_gb300 import kla

CALLS = sorted(n for n, f in vars(kla).items() if inspect.isfunction(f) and not n.startswith("_")
               and "stream" in inspect.signature(f).parameters)


@pytest.fixture
def streams(monkeypatch):
    """Streams 0 (current) and 7 of a device that need not be there; `entered` lists what torch.cuda.stream was given."""
    entered = []

    @contextlib.contextmanager
    def enter(s):
        entered.append(s)
        yield

    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "caller")
    monkeypatch.setattr(kla, "_raw_stream", lambda index: 0)
    make = lambda handle: SimpleNamespace(cuda_stream=handle, device=SimpleNamespace(index=0, type="cuda"))
    return make(0), make(7), entered


def test_the_calls_are_known():
    assert {"forward", "backward", "step", "conv", "conv_backward", "shard_map", "shard_start", "forward_context_parallel",
            "delta_forward", "delta_backward", "delta_step", "norm_rope", "norm_rope_backward"} <= set(CALLS)


@pytest.mark.parametrize("name", CALLS)
def test_allocations_are_made_under_the_given_stream(name, streams):
    """(The calls get no arguments and fail, but inside the stream.)"""
    current, other, entered = streams
    f = getattr(kla, name)
    for s, want in ((None, []), (current, []), (other, [other])):
        entered.clear()
        with pytest.raises(TypeError):
            f(**({} if s is None else {"stream": s}))
        assert entered == want


def test_results_are_kept_for_the_callers_stream(streams):
    current, other, _ = streams
    kept = []

    class Tensor:
        def record_stream(self, s):
            kept.append((self, s))

    x, y = Tensor(), Tensor()
    for out in ((x, None, y), {"a": x, "b": y}):
        kept.clear()
        f = kla._on_stream(lambda stream=None: out)
        assert f(stream=other) is out and kept == [(x, "caller"), (y, "caller")]
        kept.clear()
        assert f() is out and f(stream=current) is out and not kept
    assert kla._on_stream(lambda stream=None: x)(stream=other) is x and kept == [(x, "caller")]
