"""The stated bound of verkv_rope_turns over the whole range of frequencies, against exact rationals."""
import os
import re
from fractions import Fraction

import numpy as np
import pytest

from tests.test_rope_turns import PI
from verified_kv_cache_poissoncomp_gb300 import binding as B
from verified_kv_cache_poissoncomp_gb300 import build as build_mod


def stated(f):
    """Of a turn and position, as include/verkv.h gives it."""
    return abs(Fraction(f)) / 2 ** 54 + Fraction(1, 2 ** 63)


def off(f, t):
    # two frequencies' turns differ by whole turns at most where they are the same angle
    x = (Fraction(f) / (2 * PI) - Fraction(t, 1 << 64)) % 1
    return min(x, 1 - x)


@pytest.mark.parametrize("f", [1.0, 0.7, 1e-9, 2.0 ** -70, 0.0, 6.25, 6.2831853071795864, 6.3, 12.3, 12345.678, 1e6, 3e9, 2.0 ** 32 - 1e-6])
@pytest.mark.parametrize("sign", [1, -1])
def test_bound_of_every_frequency(f, sign):
    build_mod.build()
    t, = B.verkv_rope_turns([sign * f])
    assert off(sign * f, t) <= stated(f)
    rng = np.random.default_rng(1)
    near = [sign * f * (1 + x) for x in rng.uniform(-1e-9, 0, 20)]
    for g, t in zip(near, B.verkv_rope_turns(near)):
        assert off(g, t) <= stated(g)


def test_the_header_says_so():
    with open(os.path.join(build_mod.ROOT, "include", "verkv.h")) as f:
        text = re.sub(r"\s*\n \*\s*", " ", f.read())
    assert "p (|inv_freq[j]| 2^-54 + 2^-63) of a turn" in text
