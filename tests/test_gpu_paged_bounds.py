"""Bounds that are not tight: a call's result is as exact with any bound, and the same bits again with the
same one.  (Another bound may cut the work elsewhere, so that partial sums are grouped differently.)"""
import pytest
import torch

from tests import paged_reference as R
from tests.test_gpu_paged import BF, HF, Case

pytestmark = pytest.mark.gpu


def wide_tables(c, pages):
    """The same tables with room for `pages` pages a row; what is behind a length may be anything."""
    for name in ("table", "prefix_table"):
        t = getattr(c, name)
        if t is not None:
            w = torch.full((t.shape[0], pages), -1, dtype=torch.int32, device="cuda")
            w[:, :t.shape[1]] = t
            setattr(c, name, w)


@pytest.mark.parametrize("lengths,qs,prefixes,groups,dtype,d", [
    ([300, 5, 800, 64] * 10, 1, [2000], None, BF, 128), ([512, 100, 3, 77, 512, 9, 0, 300], 1, [2048], None, BF, 128),
    ([90, 30], 3, [], None, HF, 64), ([40] * 12, 5, [900, 0, 333], [0, 5, 6, 12], HF, 128), ([700, 600], 90, [100], None, BF, 64)])
def test_results_do_not_depend_on_the_bounds(lengths, qs, prefixes, groups, dtype, d):
    c = Case(lengths, qs=[qs] * len(lengths), prefixes=prefixes, groups=groups, h=2, g=4, d=d, pt=64, dtype=dtype)
    most = 131072
    wide_tables(c, most // 64)
    own, pre = c.max_length, c.max_prefix
    for c.max_length in (own, own + 1, 4 * own, most):
        for c.max_prefix in ((pre, 3 * pre, most) if prefixes else (0,)):
            o, lse = c.check()
            for _ in range(3):
                o2, lse2 = c.run()
                assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_a_graph_of_far_bounds():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = Case([512, 100, 3, 77, 512, 9, 0, 300], prefixes=[2048], h=2, g=4, d=128, pt=64)
        wide_tables(c, 131072 // 64)
        c.max_length, c.max_prefix = 1 << 16, 131072
        eager = c.check()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            o, lse = c.run()
        for _ in range(3):
            graph.replay()
            c.cache.sync()
            assert torch.equal(o, eager[0]) and torch.equal(lse, eager[1])
        for n, p in ((1, 1), (0, 2048), (3, 0)):
            c.lengths.clamp_(max=n)
            c.prefix_lengths.fill_(p)
            graph.replay()
            c.cache.sync()
            wo, wl, to, tl = c.want()
            R.close(lse, wl, tl, "lse")
            R.close(o, wo, to, "o")
