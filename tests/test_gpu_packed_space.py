"""Attention over 4-bit pages in workspaces of just the size asked for, which is what 16-bit pages need: few rows behind a
prefix, where own tokens or the prefix are most of the work, and more."""
import pytest
import torch

from tests import packed_bound as K
from tests import paged_reference as R
from tests.test_gpu_packed import Packed
from tests.test_gpu_paged import BF, HF
from verified_kv_cache_poissoncomp_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [(BF, 128), (HF, 64)])
@pytest.mark.parametrize("g,qs", [(1, [1]), (1, [9]), (4, [1, 1]), (4, [1, 1, 1]), (4, [4]), (4, [1, 1, 1, 1]), (4, [3, 1]), (8, [1]), (8, [1, 1]), (8, [2]),
                                  (8, [1, 1, 1]), (4, [5, 6, 7])])
@pytest.mark.parametrize("own,prefix", [(3000, 70), (90, 5000), (700, 700)])
def test_the_size_asked_for_is_enough(dtype, d, g, qs, own, prefix):
    n = [own - 37 * i for i in range(len(qs))]
    c = Packed([max(x, 1) for x in n], qs=qs, prefixes=[prefix], h=3, g=g, d=d, pt=32, dtype=dtype)
    t = sum(qs)
    need = B.verkv_paged_workspace_size(c.cache.shape, len(qs), 1, t)
    room = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    assert room.data_ptr() % 256 == 0
    o, lse = torch.empty((t, 3 * g, d), dtype=dtype, device="cuda"), torch.empty((t, 3 * g), device="cuda")
    span = lambda table, lengths, most: B.verkv_span(table.data_ptr(), table.shape[0], table.shape[1], lengths.data_ptr(), most)  # noqa: E731
    call = lambda size: B.lib().verkv_paged_attend(  # noqa: E731
        c.cache.ctx, c.cache._layer(0), len(qs), t, B.verkv_rows(c.q.data_ptr(), 3 * g * d, d), c.q_start.data_ptr() if c.q_start is not None else None,
        span(c.table, c.lengths, c.max_length), span(c.prefix_table, c.prefix_lengths, c.max_prefix), None, 0.0, None, None,
        o.data_ptr(), lse.data_ptr(), room.data_ptr(), size)
    assert call(need - 1) == B.VERKV_EINVAL
    assert call(need) == B.VERKV_OK
    c.cache.sync()
    wo, wl, to, tl, _ = K.attend(c.q, c.kv[0], c.table, c.lengths, c.q_start, c.prefix_table, c.prefix_lengths)
    R.close(o, wo, to, "o")
    R.close(lse, wl, tl, "lse")
    assert bool((room[need:] == 0x5A).all())
