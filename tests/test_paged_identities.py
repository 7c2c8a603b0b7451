"""The integer rewrites the paged attention kernels rely on, on the CPU, against what they stand for (the
kernels themselves are held to float64 by the GPU tests)."""
import numpy as np

ROOMS_MOST = 1 << 21  # steps of a line whose units may get rooms (csrc/paged.cuh)


def test_quotients_by_the_fast_reciprocal():
    # int(q + 1/2) is e for q within two units of the last place of e, a whole number below ROOMS_MOST; the
    # numerator e * y may round when it becomes a float32, by half a unit of its own
    rng = np.random.default_rng(3)
    e = np.concatenate([rng.integers(1, ROOMS_MOST, 200_000), ROOMS_MOST - 1 - np.arange(2000), 1 + np.arange(2000)])
    y = rng.integers(1, 153, e.size)
    few = e * y < ROOMS_MOST  # a line's steps are its segments' together
    e, y = e[few], y[few]
    assert np.array_equal((e * y).astype(np.float32).astype(np.int64), e * y)
    q = e.astype(np.float32)
    for ulps in (-2, -1, 0, 1, 2):
        off = q + np.float32(ulps) * np.spacing(q)
        assert np.array_equal((off + np.float32(0.5)).astype(np.int64), e), ulps
    # the quotient (e + r - 1/2) / r, cut: the least p with p r >= e, or one more or less (less is put right)
    r = rng.integers(1, 153, e.size)
    least = -(-e // r)
    for ulps in (-2, 0, 2):
        q = ((e.astype(np.float32) + r.astype(np.float32) - np.float32(0.5)) / r.astype(np.float32))
        p = (q + np.float32(ulps) * np.spacing(q)).astype(np.int64)
        p = p + (p * r < e)
        assert (p * r >= e).all() and (p <= least + 1).all()


def test_the_bound_is_the_kernels():
    import os

    from verified_kv_cache_poissoncomp_gb300 import build as build_mod
    with open(os.path.join(build_mod.CSRC, "paged.cuh")) as f:
        assert "constexpr int PAGED_ROOMS_MOST = 1 << 21;" in f.read()
