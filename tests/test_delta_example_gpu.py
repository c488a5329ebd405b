"""The README's delta rule example runs as written; the example model trains through the convolution, the norm with rotation and
the delta rule, and decodes one token at a time to the same logits."""
import importlib.util
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_example_runs():
    text = open(os.path.join(ROOT, "README.md")).read()
    block = [b for b in re.findall(r"```python\n(.*?)```", text, flags=re.S) if "delta_forward" in b]
    scope = {}
    exec(compile(block[0], "README.md", "exec"), scope)
    torch.cuda.synchronize()
    assert scope["o"].shape == (2, 8, 1000, 128) and bool(scope["o"].isfinite().all())
    assert bool(scope["o_t"].isfinite().all()) and bool(scope["state"].isfinite().all())


def test_example_learns_and_decodes():
    path = os.path.join(ROOT, "examples", "delta_mixer.py")
    spec = importlib.util.spec_from_file_location("delta_mixer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    said = []
    loss, right, apart = example.main(steps=300, say=said.append)
    first = float(said[0].split()[-1])
    assert first > 3.0 and loss < 0.5 * first, said
    assert apart < 1e-4  # fp32 throughout: sums in another order
