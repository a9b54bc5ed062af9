"""The rotary tables (hs.rope_frequencies, hs.rope_turns) against their definitions
(no GPU)."""
import math
from fractions import Fraction

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


PI = Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620899,
              10 ** 80)


@pytest.mark.parametrize("inv", [
    hs.rope_frequencies(128)[0], hs.rope_frequencies(64, 1e6)[0],
    hs.rope_frequencies(64, scaling="linear", factor=32.0)[0],
    torch.tensor([0.0, 1.0, -1.0, 3.0, 4.0, 6.0, 7.0, 100.0, 1e-300, 5e-324, 1e15, -0.3]),
    torch.tensor([0.1, 2.5], dtype=torch.float32), torch.zeros(0)])
def test_turns_are_rounded_at_64_bits(inv):
    """Every entry is the nearest to its frequency's, so that the product with a
    position, modulo whole turns, is off by half a unit of 2^-64 a position."""
    table = hs.rope_turns(inv, "cpu")
    assert table.dtype == torch.int64 and table.shape == inv.shape
    for f, t in zip(inv.double().tolist(), table.tolist()):
        exact = Fraction(f) / (2 * PI) * 2 ** 64
        off = (t - exact) % 2 ** 64  # whole turns do not count
        assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + abs(exact) / 10 ** 60
        for p in (1, 12345, 2 ** 30, 2 ** 31 - 1):
            turns = Fraction(p * t, 2 ** 64) - Fraction(f) * p / (2 * PI)
            off = turns % 1
            assert min(off, 1 - off) <= Fraction(p, 2 ** 65) + p * abs(Fraction(f)) / 10 ** 60


def test_turns_refuse_what_has_none():
    for f in (math.inf, math.nan):
        with pytest.raises(ValueError):
            hs.rope_turns(torch.tensor([1.0, f]), "cpu")
