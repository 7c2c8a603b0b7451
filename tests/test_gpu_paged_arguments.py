"""Arguments of PagedKV.attend that say nothing without another one are refused, not left out."""
import pytest

from tests.test_gpu_paged import Case
from verified_kv_cache_poissoncomp_gb300 import binding as B

pytestmark = pytest.mark.gpu


def test_tables_and_lengths_come_together():
    c = Case([100, 33, 64], prefixes=[130], h=2, g=2, d=64)
    n0 = B.verkv_launch_counts(c.cache.ctx)
    for a, kw in (((None, c.lengths, 100), {}), ((c.table, None, 100), {}),
                  ((c.table, c.lengths, 100), dict(prefix_lengths=c.prefix_lengths, max_prefix=130)),
                  ((c.table, c.lengths, 100), dict(prefix_table=c.prefix_table, max_prefix=130))):
        with pytest.raises(ValueError):
            c.cache.attend(0, c.q, *a, **kw)
    assert B.verkv_launch_counts(c.cache.ctx) == n0
    c.check()
