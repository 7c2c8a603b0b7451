"""A copy that never comes: the kernels' waits give up, what is in flight lands before a CTA gives its
memory back, the host is told, and the next call is as good as any."""
import pytest
import torch

from tests.test_gpu_paged import BF, HF, Case
from verified_kv_cache_poissoncomp_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths,qs,prefix,d,dtype", [
    ([40], 1, 0, 128, BF),                # one step: every copy is issued before anything is waited for
    ([200, 130], 1, 0, 64, HF),           # fewer steps than the ring holds
    ([60000] * 4, 1, 0, 128, BF),         # more steps a CTA than the ring holds
    ([300, 700], 6, 0, 128, HF),          # 32 rows a unit
    ([60], 20, 900, 128, BF),             # 128 rows a unit
    ([3000] * 2, 20, 40000, 64, HF),
    ([60], 100, 900, 64, BF),             # 256 rows a unit
    ([3000], 200, 40000, 128, BF),
    ([400] * 40, 1, 9000, 128, BF)])      # both kernels side by side
def test_a_copy_that_never_comes(lengths, qs, prefix, d, dtype):
    c = Case(lengths, qs=[qs] * len(lengths), prefixes=[prefix] if prefix else (), h=2, g=4, d=d, pt=64, dtype=dtype)
    good = c.run()
    c.cache.sync()
    for _ in range(2):
        B.verkv_test_inject(c.cache.ctx, B.VERKV_INJECT_PAGED_STALL, 2_000_000)
        c.run()
        assert B.verkv_sync_status(c.cache.ctx) == B.VERKV_ETIMEOUT
        o, lse = c.run()
        assert B.verkv_sync_status(c.cache.ctx) == B.VERKV_OK
        assert torch.equal(o, good[0]) and torch.equal(lse, good[1])


def test_the_injection_is_checked():
    c = Case([40], h=1, g=1, d=64)
    for value in (0, 999, 1_000_000_001):
        with pytest.raises(B.VerkvError) as e:
            B.verkv_test_inject(c.cache.ctx, B.VERKV_INJECT_PAGED_STALL, value)
        assert e.value.status == B.VERKV_EINVAL
