"""The rotary plan's numbers on the host: fractions of a turn rounded to 2^-64, and amplitudes."""
import math
from fractions import Fraction

import pytest

from paged_kv_cache_47_gb300 import binding as b
from paged_kv_cache_47_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


# base, rotary_dim: slowest pairs from 1e-4 down to 1e-29 radians a position
@pytest.mark.parametrize("base,rd", [(10000.0, 128), (500000.0, 128), (1e8, 64), (1e15, 128), (1e20, 128), (1e30, 128)])
def test_turns_are_rounded(base, rd):
    p = b.RopePlan(rd, base=base).c
    odd = 0
    for i in range(rd // 2):
        turns = Fraction(base ** (-2.0 * i / rd)) / Fraction(2 * math.pi)
        # pow, 2 pi and the division: a few roundings of 2^-53 of the value; then half a step of 2^-64
        tol = turns * Fraction(8, 2 ** 53) + Fraction(1, 2 ** 65)
        assert abs(Fraction(p.turns[i], 2 ** 64) - turns) <= tol, i
        odd += p.turns[i] & 1
    if base >= 1e15:
        assert odd                                   # the last bit is in use


@pytest.mark.parametrize("factor,amplitude", [(0.25, 1.0), (1.0, 1.0), (math.e ** 2, 1.2), (16.0, 0.1 * math.log(16) + 1)])
def test_yarn_amplitude(factor, amplitude):
    # only a longer context raises it
    kw = dict(scaling="yarn", factor=factor, original_len=4096)
    assert b.RopePlan(64, **kw).c.amplitude == pytest.approx(amplitude, rel=2.0 ** -23)
    assert b.RopePlan(64, attention_factor=0.7, **kw).c.amplitude == pytest.approx(0.7, rel=2.0 ** -23)
