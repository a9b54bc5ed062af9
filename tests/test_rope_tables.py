"""The rotary tables (hs.rope_frequencies, hs.rope_turns) against their definitions
(no GPU)."""
import math

import pytest
import torch

from sparse_top_kv_gb300 import hs


@pytest.mark.parametrize("rot,base,length,factor,slow,fast", [
    (128, 10000.0, 4096, 8.0, 1.0, 32.0), (64, 10000.0, 2048, 4.0, 1.0, 32.0),
    (128, 1e6, 32768, 4.0, 1.0, 32.0), (64, 10000.0, 4096, 40.0, 1.0, 32.0),
    (96, 500000.0, 8192, 2.0, 2.0, 20.0), (2, 10000.0, 100, 2.0, 1.0, 32.0),
    (16, 10000.0, 7, 3.0, 1.0, 32.0)])
def test_yarn_goes_over_by_pairs(rot, base, length, factor, slow, fast):
    inv, scale = hs.rope_frequencies(rot, base, scaling="yarn", factor=factor, original_len=length,
                                     slow_turns=slow, fast_turns=fast)
    # Pair i of frequency base^(-2 i / rot) turns length base^(-2 i / rot) / 2 pi times.
    # The outermost pairs that have to change and that have not to, one pair outwards
    # where the border lies between two.
    at = [rot * math.log(length / (2 * math.pi * n)) / (2 * math.log(base)) for n in (fast, slow)]
    low, high = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
    for i, f in enumerate(inv.tolist()):
        w = base ** (-2.0 * i / rot)
        if high > low:
            part = min(1.0, max(0.0, (i - low) / (high - low)))
        else:
            part = 0.0 if i <= low else 1.0
        # A dozen roundings of 2^-53 each.
        assert abs(f - ((1 - part) * w + part * w / factor)) <= 1e-14 * w
    assert abs(scale - (0.1 * math.log(factor) + 1)) <= 1e-14
    assert inv.dtype == torch.float64


def test_yarn_refusals():
    ok = dict(rot=64, scaling="yarn", factor=4.0, original_len=4096)
    hs.rope_frequencies(**ok)
    for bad in (dict(original_len=0), dict(original_len=None), dict(slow_turns=0.0),
                dict(slow_turns=32.0), dict(base=1.0), dict(base=0.5)):
        with pytest.raises(ValueError):
            hs.rope_frequencies(**{**ok, **bad})
    assert hs.rope_frequencies(**{**ok, "rot": 0})[0].numel() == 0
