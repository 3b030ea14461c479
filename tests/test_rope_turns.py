"""mla_rope_init's whole-number frequencies, without a GPU."""
import math
from fractions import Fraction

import pytest

import mla_latent_kv_attention_gb300 as mla


@pytest.mark.parametrize("base", [10000.0, 500000.0, 1e6, 1.5, 1e30])
def test_turns_are_rounded_to_nearest(base):
    """The turns of a position as a float64 has them, to the nearest multiple of 2^-64."""
    for i, got in enumerate(mla.mla_rope_init(base).turns):
        turn = Fraction(base ** (-2 * i / 64) / (2 * math.pi))
        assert abs(got - (turn - math.floor(turn)) * 2 ** 64) <= Fraction(1, 2)


@pytest.mark.parametrize("base,factor,original", [(10000.0, 1.0, 0), (10000.0, 40.0, 0), (500000.0, 8.0, 0)])
def test_phase_at_far_positions(base, factor, original):
    """The phase of position m is off by at most m (2^-65 + 2^-50 f / 2 pi) turns: the rounding of
    the whole number and the relative error of the frequency in float64 (a power within 2^-52, two
    divisions and pi within 2^-53 each)."""
    rope = mla.mla_rope_init(base, factor=factor, original_positions=original)
    # pi to 60 digits, and the 64th root of the base by bisection in whole numbers
    pi = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)
    scale = 10 ** 40
    lo, hi = scale, int(base) * scale
    while hi - lo > 1:
        mid = (lo + hi) // 2
        if mid ** 64 <= int(base) * scale ** 64:
            lo = mid
        else:
            hi = mid
    root = Fraction(lo, scale)
    for i in (0, 1, 13, 31):
        turn = 1 / (root ** (2 * i) * Fraction(factor) * 2 * pi)
        for m in (1, 163840, 10 ** 6, 2 ** 40):
            off = Fraction(rope.turns[i] * m % 2 ** 64, 2 ** 64) - turn * m
            off -= round(off)
            assert abs(off) <= m * (Fraction(1, 2 ** 65) + turn / 2 ** 50)


@pytest.mark.parametrize("kw", [dict(factor=1e-320), dict(factor=5e-324, original_positions=4096)])
def test_stretches_past_float64_are_refused(kw):
    """f / factor overflows: no number of turns."""
    with pytest.raises(mla.MlaError) as e:
        mla.mla_rope_init(**kw)
    assert e.value.status == mla.MLA_ERR_INVALID_ARG
