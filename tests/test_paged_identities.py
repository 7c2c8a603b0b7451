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
    for _ in range(3000):
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


# ------------------------------------------------------------------------------------------------
# Steps of a prompt's row tiles in closed form, and the place of a token's sequence by 32 probes a turn.
def _ramp(b, n, tt_shift, tile_shift):
    """csrc/paged.cuh, in its 32-bit arithmetic."""
    none = 0 if b >= 0 else min(n, -b >> tt_shift)
    n -= none
    y = b + ((none + 1) << tt_shift) + (1 << tile_shift) - 1
    w = n * (y >> tile_shift)
    u = 0xFFFFFFFF
    if tt_shift >= tile_shift:
        return w + (((((n * (n - 1)) & u) >> 1) << (tt_shift - tile_shift)) & u)
    shift = tile_shift - tt_shift
    j = n + ((y & ((1 << tile_shift) - 1)) >> tt_shift)
    q = j >> shift
    return w + ((((((q * (q - 1)) & u) >> 1) << shift) + (j & ((1 << shift) - 1)) * q) & u)


def test_steps_of_row_tiles_in_closed_form():
    rng = np.random.default_rng(5)
    for _ in range(2000):
        tt_shift, tile_shift = int(rng.integers(0, 9)), int(rng.choice([6, 7]))
        qn, length = int(rng.integers(1, 3000)), int(rng.choice([0, 1, 63, 64, 65, rng.integers(0, 6000)]))
        tt, T = 1 << tt_shift, 1 << tile_shift
        nt = -(-qn // tt)
        # what the last query of a tile sees
        seen = [min(max(length - (qn - 1 - (min(qn, (k + 1) * tt) - 1)), 0), length) for k in range(nt)]
        before = np.concatenate([[0], np.cumsum([-(-v // T) for v in seen])])
        for m in {0, 1, nt // 2, nt - 1, nt} | {int(x) for x in rng.integers(0, nt + 1, 3)}:
            if m > nt:
                continue
            w = -(-length // T) if m == nt and m > 0 else 0
            if nt > 1:
                w += _ramp(length - qn, min(m, nt - 1), tt_shift, tile_shift)
            assert w == before[m], (qn, length, tt, T, m)


def test_steps_of_row_tiles_up_to_31_bits():
    for tt_shift, tile_shift, n, b in ((8, 7, 46000, 0), (5, 7, 130000, -70), (0, 6, 360000, 9), (7, 7, 65000, -129), (8, 6, 32000, 5)):
        want = sum(-(-max(0, b + ((k + 1) << tt_shift)) // (1 << tile_shift)) for k in range(n))
        assert want < 1 << 31 and _ramp(b, n, tt_shift, tile_shift) == want


def _last_at_most(start, x):
    at, left, turns = -1, len(start), 0
    while left > 0:
        step, turns = (left + 31) >> 5, turns + 1
        lanes = np.arange(0, min(32 * step, left), step)
        c = int((start[at + 1 + lanes] <= x).sum())
        if c == 0:
            break
        at += 1 + (c - 1) * step
        left = min(step, left - (c - 1) * step) - 1
    return at, turns


def test_last_start_at_most():
    rng = np.random.default_rng(6)
    for _ in range(1500):
        n = int(rng.choice([0, 1, 30, 31, 32, 33, 255, 256, 1000, 65536, rng.integers(0, 3000)]))
        start = np.sort(rng.integers(0, max(2, n), n + 1))
        start[0] = 0
        x = int(rng.integers(0, max(2, n)))
        at, turns = _last_at_most(start, x)
        assert at == np.searchsorted(start, x, side="right") - 1 and turns <= 4
        rng.shuffle(start)  # out of order: still an index of the range
        assert -1 <= _last_at_most(start, x)[0] <= n
