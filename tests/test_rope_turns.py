"""Turns per position in 64-bit fixed point, against exact rational arithmetic, and the paged calls'
argument checks that need no GPU."""
import ctypes
from fractions import Fraction

import pytest

from verified_kv_cache_poissoncomp_gb300 import binding as B
from verified_kv_cache_poissoncomp_gb300 import build as build_mod

# pi to 60 digits (published)
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.lib()


@pytest.mark.parametrize("base,rd", [(1e4, 128), (1e6, 128), (5e5, 32), (1e4, 16)])
def test_turns_give_the_angle_of_far_positions(base, rd):
    freqs = [base ** (-2 * j / rd) for j in range(rd // 2)]
    turns = B.verkv_rope_turns(freqs)
    for f, t in zip(freqs, turns):
        for p in (0, 1, 4095, 131071, (1 << 31) - 1):
            want = (Fraction(f) * p / (2 * PI)) % 1
            got = Fraction((p * t) % (1 << 64), 1 << 64)
            off = abs(got - want)
            # 2^-53 relative from the division by 2 pi (its constant rounded too), 2^-64 from the fraction
            bound = p * (Fraction(f) * Fraction(1, 6) * Fraction(3, 1 << 53) + Fraction(1, 1 << 63))
            assert min(off, 1 - off) <= bound, (f, p)


def test_turns_of_unusual_frequencies():
    assert list(B.verkv_rope_turns([0.0])) == [0]
    # a frequency and its negative turn opposite ways
    a, b = B.verkv_rope_turns([0.3, -0.3])
    assert abs((a + b) % (1 << 64) - 0) <= 1 << 12 or (1 << 64) - (a + b) % (1 << 64) <= 1 << 12
    for bad in (float("nan"), float("inf"), 2.0 ** 32, -2.0 ** 32):
        with pytest.raises(B.VerkvError) as e:
            B.verkv_rope_turns([1.0, bad])
        assert e.value.status == B.VERKV_EINVAL
    assert B.lib().verkv_rope_turns(None, 1, None) == B.VERKV_EINVAL
    assert B.lib().verkv_rope_turns(None, 0, None) == B.VERKV_EINVAL


def test_null_context_is_refused(lib):
    assert lib.verkv_norm_rotate(None, 0, 1, None, None, None, None, None, None, None) == B.VERKV_EINVAL
    assert lib.verkv_paged_append(None, None, 1, None, None, None, None, None, None, None, None, None,
                                  None) == B.VERKV_EINVAL
    assert lib.verkv_paged_attend(None, None, 1, 1, None, None, None, None, None, 0.0, None, None, None,
                                  None, None, 0) == B.VERKV_EINVAL


def test_workspace_size_covers_smaller_calls():
    s = B.verkv_shape(1, 1, 8, 4, 128, 1, 1)
    size = lambda *a: B.verkv_paged_workspace_size(s, *a)  # noqa: E731
    whole = size(256, 4, 2048)
    assert whole > 0
    for seqs in (0, 1, 17, 256):
        for groups in (0, 1, 4):
            for q in (0, 1, 256, 2048):
                assert 0 < size(seqs, groups, q) <= whole
    assert size(-1, 0, 1) == size(1, -1, 1) == size(1, 0, -1) == size(1, 0, 1 << 30) == size(1 << 20, 0, 1) == 0
    assert B.verkv_paged_workspace_size(B.verkv_shape(1, 1, 8, 3, 128, 1, 1), 1, 0, 1) == 0


def test_structures_match_the_header():
    # 64-bit pointers and strides, natural alignment
    assert [ctypes.sizeof(c) for c in (B.verkv_rows, B.verkv_rope, B.verkv_head_norm, B.verkv_pages, B.verkv_span)] == \
        [24, 16, 24, 24, 32]
