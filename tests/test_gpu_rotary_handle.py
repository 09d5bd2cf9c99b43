"""The frequencies that a rotary handle holds, for stretched contexts."""
import math
from fractions import Fraction

import pytest

torch = pytest.importorskip("torch")

from .prompt_reference import TURN  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dk():
    import sparse_attention_indexer_stable_gb300 as dk
    return dk


@pytest.mark.parametrize("kw", [
    dict(dim=128, factor=4.0, original=4096), dict(dim=64, factor=40.0, original=4096),
    dict(dim=96, base=500000.0, factor=8.0, original=8192, slow=1.0, fast=4.0, magnitude=1.0),
    dict(dim=128, factor=1.5, original=1000, slow=0.0, fast=0.5)])
def test_the_blend_between_kept_and_divided_frequencies(dk, kw):
    """By wavelengths: one of `original / fast` tokens or less is kept, one of
    `original / slow` or more is stretched by the factor, and in between the
    frequency moves linearly with the turns over the original length."""
    rope = dk.Rotary(**kw)
    slow, fast = kw.get("slow", 1.0), kw.get("fast", 32.0)
    blended = 0
    for i, got in enumerate(rope.frequencies):
        length = 2.0 * math.pi * kw.get("base", 10000.0) ** (2.0 * i / kw["dim"])
        turns = kw["original"] / length
        if turns >= fast:
            want = 2.0 * math.pi / length
        elif turns <= slow:
            want = 2.0 * math.pi / (length * kw["factor"])
        else:
            blended += 1
            share = (turns - slow) / (fast - slow)
            want = 2.0 * math.pi * (share / length + (1.0 - share) / (length * kw["factor"]))
        # the power's exponent is rounded by 2^-53, which comes out times ln base (13),
        # and a blend's share in the frequency times the factor (40): 2^-44; twice
        assert got == pytest.approx(want, rel=2.0 ** -42)
    assert blended
    assert rope.magnitude == pytest.approx(kw.get("magnitude", 0.1 * math.log(kw["factor"]) + 1))


@pytest.mark.parametrize("kw", [dict(), dict(factor=8.0, original=4096),
                                dict(frequencies=[0.0, 3.0, -1e-3, 1e4, -7.5] * 6 + [1e-9, -2.0])])
def test_turns_are_exact_to_half_a_step(dk, kw):
    """2^-65 of a turn a position, 2^-34 at the farthest."""
    rope = dk.Rotary(64, **kw)
    for f, turn in zip(rope.frequencies, rope.turns.tolist()):
        off = Fraction(turn, 2 ** 64) - Fraction(f) / TURN
        assert abs(off - round(off)) <= Fraction(1, 2 ** 65)
