"""Queries that count nothing (lse -infinity, as a padded batch may have them) whose channels are no numbers."""
import math

import pytest
import torch

from tests.test_gpu_evict import KINDS, check_weigh
from tests.test_gpu_paged import Case

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), math.inf


@pytest.mark.parametrize("kind,dtype,d", KINDS)
@pytest.mark.parametrize("qs", [[1, 1, 1, 1], [3, 2, 0, 3], [5, 3, 4, 6], [20, 33, 7, 64], [130, 70, 1, 9]])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_a_query_that_counts_nothing_may_hold_anything(kind, dtype, d, qs, value):
    c = kind([300, 64, 17, 129], qs=qs, h=2, g=4, d=d, pt=16, dtype=dtype)
    _, lse = c.run()
    n = sum(qs)
    # whole queries, and one head of another: every value, or one channel of the last group
    for i in range(0, n, 3):
        c.q[i], lse[i] = value, -INF
    c.q[n - 1, 5, d - 1], lse[n - 1, 5] = value, -INF
    got, _ = check_weigh(c, lse=lse, weights=True, extra=5, apart=True)
    assert not bool(torch.isnan(got).any())


def test_all_of_a_batch_is_padding():
    for qs in (1, 9, 40):
        c = Case([40, 64], qs=[qs] * 2, h=2, g=4, pt=16)
        c.q.fill_(NAN)
        got, _ = check_weigh(c, lse=torch.full((2 * qs, 8), -INF, device="cuda"), weights=True)
