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


# ------------------------------------------------------------------------------------------------
# The workspace.  What a call lays out, as the launches are chosen (csrc/verkv_api.cu): k_paged's tiles of 16
# or 32 rows, k_paged_wide's of 128 or 256, by the rows of a segment on average.
def _laid_out(h, G, d, seqs, groups, q, own, prefix):
    """Bytes of the workspace that a call of these sizes uses."""
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    avg = lambda n: -(-q // max(n, 1)) * G  # noqa: E731
    levels = [(groups, avg(groups), 16)] * (prefix and groups > 0) + [(seqs, avg(seqs), 32)] * (own and seqs > 0)
    wide = [(n, r) for n, r, few in levels if r > few]
    few = [(n, r) for n, r, few in levels if r <= few]
    off = 256
    for line, tile, ctas in ((wide, 256 if all(r > 128 for _, r in wide) else 128, 152),
                             (few, 16 if all(r <= 16 for _, r in few) else 32, 304)):
        if not line:
            continue
        slots = sum(q // (tile // G) + n for n, _ in line) * h + ctas
        off = up(off + (1 + sum(n for n, _ in line)) * 8)
        off = up(off + slots * tile * 8)
        off = up(off + slots * tile * d * 4)
    return off


def _workspace_size():
    from verified_kv_cache_poissoncomp_gb300 import binding as B
    from verified_kv_cache_poissoncomp_gb300 import build as build_mod
    build_mod.build()
    return lambda h, G, d, *sizes: B.verkv_paged_workspace_size(B.verkv_shape(1, 1, h, G, d, 1, 1), *sizes)


def test_workspace_holds_what_any_smaller_call_lays_out():
    size = _workspace_size()
    rng = np.random.default_rng(11)
    log = lambda lo, hi: int(np.exp(rng.uniform(np.log(lo), np.log(hi + 1))))  # noqa: E731
    for _ in range(20_000):
        h, G, d = int(rng.choice([1, 2, 8])), int(rng.choice([1, 2, 4, 8])), int(rng.choice([64, 128]))
        seqs, groups, q = log(1, 3000), int(rng.integers(0, 2)) * log(1, 3000), log(1, 40000)
        have = size(h, G, d, seqs, groups, q)
        for _ in range(3):  # the call itself and smaller ones
            for own, prefix in ((1, 0), (0, 1), (1, 1)):
                assert _laid_out(h, G, d, seqs, groups, q, own, prefix) <= have, (h, G, d, seqs, groups, q, own, prefix)
            assert size(h, G, d, seqs, groups, q) <= have
            seqs, groups, q = log(1, seqs), int(rng.integers(0, groups + 1)), log(1, q)


def test_workspace_of_a_prompt_is_in_proportion():
    # a float32 partial row for each query row, and little more
    size = _workspace_size()
    for seqs, q in ((1, 2048), (1, 8192), (4, 4 * 8192), (1, 32768)):
        rows = q * 32
        assert size(8, 4, 128, seqs, 0, q) <= rows * 130 * 4 * 1.2 + (24 << 20)
    # a decode step of 256 sequences behind a prefix
    assert size(8, 4, 128, 256, 1, 256) < 80 << 20
