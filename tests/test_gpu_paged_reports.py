"""What the device arrays of a call hold out of range is reported also where no page is read for it: starts of
queries that only prefixes are attended for, and lengths of a level whose bound is 0."""
import math

import pytest
import torch

from tests.test_gpu_paged import Case, ints
from verified_kv_cache_poissoncomp_gb300 import binding as B
from verified_kv_cache_poissoncomp_gb300.paged import PagedKV

pytestmark = pytest.mark.gpu


def status(c, *a, **kw):
    c.cache.attend(0, c.q, *a, **kw)
    return B.verkv_sync_status(c.cache.ctx)


@pytest.mark.parametrize("bound", [130, 0])
def test_starts_without_own_tokens(bound):
    c = Case([0] * 4, qs=[2, 1, 4, 3], prefixes=[130, 70] if bound else [0, 0], groups=[0, 2, 4], h=2, g=2, d=64)
    pre = dict(prefix_table=c.prefix_table, prefix_lengths=c.prefix_lengths, max_prefix=bound)
    for starts, want in (([0, 2, 3, 7, 10], B.VERKV_OK), ([0, 0, 0, 0, 10], B.VERKV_OK), ([0, 9, 5, 7, 10], B.VERKV_EINVAL),
                         ([0, 2, 3, 11, 10], B.VERKV_EINVAL), ([0, 2, 3, -1, 10], B.VERKV_EINVAL), ([0, 2, 3, 7, 9], B.VERKV_EINVAL),
                         ([1, 2, 3, 7, 10], B.VERKV_EINVAL)):
        assert status(c, None, None, 0, q_start=ints(starts), group_start=c.group_start, **pre) == want, starts
    for groups, want in (([0, 0, 4], B.VERKV_OK), ([0, 4, 4], B.VERKV_OK), ([0, 5, 4], B.VERKV_EINVAL), ([0, -1, 4], B.VERKV_EINVAL),
                         ([0, 2, 3], B.VERKV_EINVAL), ([1, 2, 4], B.VERKV_EINVAL)):
        assert status(c, None, None, 0, q_start=c.q_start, group_start=ints(groups), **pre) == want, groups
    # no prefix either: nothing but the starts is read
    assert status(c, None, None, 0, q_start=c.q_start) == B.VERKV_OK
    assert status(c, None, None, 0, q_start=ints([0, 9, 5, 7, 10])) == B.VERKV_EINVAL


def test_lengths_of_a_bound_of_zero():
    c = Case([0] * 3, qs=[2, 0, 4], prefixes=[130], h=2, g=2, d=64)
    pre = dict(prefix_table=c.prefix_table, prefix_lengths=c.prefix_lengths)
    assert status(c, c.table, c.lengths, 0, q_start=c.q_start, max_prefix=130, **pre) == B.VERKV_OK
    # a prefix whose bound was forgotten, and own tokens, of a sequence without queries too
    assert status(c, c.table, c.lengths, 0, q_start=c.q_start, **pre) == B.VERKV_EINVAL
    for i in range(3):
        for n in (1, -1):
            assert status(c, c.table, ints([n * (j == i) for j in range(3)]), 0, q_start=c.q_start, max_prefix=130, **pre) == B.VERKV_EINVAL
    assert status(c, c.table, c.lengths, 0, q_start=c.q_start, prefix_table=c.prefix_table, prefix_lengths=ints([0])) == B.VERKV_OK


def test_many_starts_and_lengths():
    # more of them than the grid has threads
    n = 3000
    c = Case([0], h=1, g=1, d=64)
    starts = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    starts[n] = 1
    table, lengths = torch.zeros((n, 1), dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    assert status(c, table, lengths, 0, q_start=starts) == B.VERKV_OK
    lengths[n - 1] = 1
    assert status(c, table, lengths, 0, q_start=starts) == B.VERKV_EINVAL
    starts[n - 1], lengths[n - 1] = 2, 0
    assert status(c, table, lengths, 0, q_start=starts) == B.VERKV_EINVAL


def test_a_grid_of_more_threads_than_32_bits_count():
    # 2^21 queries of 64 heads that see nothing: 2^25 blocks of 128 threads, all of which share the checks
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 60 GB")
    n, h = 1 << 21, 64
    c = PagedKV(h, 1, 64, num_pages=1)
    q = torch.zeros((1, h, 64), dtype=torch.bfloat16, device="cuda").expand(n, -1, -1)
    for starts, want in (([0, n], B.VERKV_OK), ([0, n - 1], B.VERKV_EINVAL), ([1, n], B.VERKV_EINVAL)):
        o, lse = c.attend(0, q, None, None, 0, q_start=ints(starts))
        assert B.verkv_sync_status(c.ctx) == want
    assert not o[::4096].any() and bool((lse == -math.inf).all())
