"""Frequencies scaled by bands: pairs that turn at least ``beta_fast`` times over
the original length are kept, those that turn at most ``beta_slow`` times are
divided by the factor, and only the pairs between are blended, also where one end
of the blend lies before the first pair or past the last."""
import math

import pytest
import torch

from bayesian_filtering_linear_gb300 import kla


def turns_of(rot, base, length):
    return length * base ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2)) / (2 * math.pi)


@pytest.mark.parametrize("rot,base,length", [(64, 10000.0, 4096), (128, 10000.0, 131072), (32, 10000.0, 65536),
                                             (128, 500000.0, 8192), (64, 10000.0, 150), (16, 100.0, 32768),
                                             (64, 10000.0, 3)])
@pytest.mark.parametrize("factor", [4.0, 8.0])
def test_bands_keep_divide_and_blend_where_they_say(rot, base, length, factor):
    got, _ = kla.rope_frequencies(rot, base, scaling="bands", factor=factor, original_length=length)
    full, turns = kla.rope_frequencies(rot, base)[0], turns_of(rot, base, length)
    share = (full / got).double()                                # 1: kept, factor: divided
    eps = 1e-6 * factor
    kept, divided = turns >= 32.0, turns <= 1.0
    assert bool((share[kept] - 1 <= eps).all())
    assert bool((share[divided] >= factor - eps).all())
    between = ~kept & ~divided
    assert bool((share[between] >= 1 - eps).all()) and bool((share[between] <= factor + eps).all())
    # not a pair before the one where the blend ends is divided in full, nor one after its start kept
    ends = [rot // 2 * math.log(length / (2 * math.pi * t)) / math.log(base) for t in (32.0, 1.0)]
    i = torch.arange(rot // 2)
    inside = (i > math.floor(ends[0])) & (i < math.ceil(ends[1]))
    assert bool((share[inside] > 1 + eps).all()) and bool((share[inside] < factor - eps).all())
    assert bool((share[1:] >= share[:-1] - eps).all())


def test_a_last_pair_that_still_turns_is_not_divided_in_full():
    """rot_dim 128, base 10000, 131072 positions: the last pair turns 2.4 times."""
    got, _ = kla.rope_frequencies(128, scaling="bands", factor=4.0, original_length=131072)
    full = kla.rope_frequencies(128)[0]
    assert float(turns_of(128, 10000.0, 131072)[-1]) > 2.4
    lo, hi = (64 * math.log(131072 / (2 * math.pi * t)) / math.log(10000.0) for t in (32.0, 1.0))
    slow = (torch.arange(64) - math.floor(lo)).clamp_min(0) / (math.ceil(hi) - math.floor(lo))
    assert torch.allclose(got, full * (1 - slow) + full / 4.0 * slow, rtol=1e-6)
    assert float(full[-1] / got[-1]) < 3.0
