"""The workspaces that a PagedKV holds: one, of the largest call so far, and those of captured graphs."""
import pytest
import torch

from tests.test_gpu_paged import BF, Case, ints
from verified_kv_cache_poissoncomp_gb300 import binding as B
from verified_kv_cache_poissoncomp_gb300.paged import PagedKV

pytestmark = pytest.mark.gpu


def held(c):
    return sum(s.numel() for s in c._spaces)


def test_growing_calls_hold_one_workspace():
    c = PagedKV(8, 4, 128, num_pages=2)
    table, lengths = torch.zeros((256, 1), dtype=torch.int32, device="cuda"), torch.zeros(256, dtype=torch.int32, device="cuda")
    q = torch.zeros((256, 32, 128), dtype=BF, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((256, 32), device="cuda")
    sizes = set()
    for n in range(1, 257):
        c.attend(0, q[:n], table[:n], lengths[:n], 64, prefix_table=table[:1], prefix_lengths=lengths[:1], max_prefix=64,
                 out=o[:n], lse=lse[:n])
        sizes.add(held(c))
    c.sync()
    need = B.verkv_paged_workspace_size(c.shape, 256, 1, 256)
    assert len(c._spaces) == 1 and need <= held(c) <= need * 3 // 2 and len(sizes) <= 8
    c.attend(0, q[:1], table[:1], lengths[:1], 64)  # a smaller call takes the same
    assert len(c._spaces) == 1 and held(c) in sizes
    # calls of many sizes are not remembered without end
    for n in range(5000):
        c._space(1, 0, 1 + n % 3 + n)
    assert len(c._needs) <= 4096


def test_a_captured_workspace_is_kept():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = Case([200, 90, 150, 64], prefixes=[500], h=2, g=4, pt=32)
        want = c.run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            o, lse = c.run()
        first = c.cache._spaces[-1]
        assert len(c.cache._spaces) == 1
        # larger calls, one after the other: the graph's workspace stays, of the others the last one
        for n in (64, 200, 900, 4000):
            q = c.q[:1].expand(n, -1, -1)
            c.cache.attend(0, q, c.table[:1].repeat(n, 1), c.lengths[:1].repeat(n), c.max_length)
        assert len(c.cache._spaces) == 2 and c.cache._spaces[0] is first
        junk = [torch.full((first.numel() // 4,), 7.0, device="cuda") for _ in range(4)]
        for _ in range(3):
            o.zero_()
            graph.replay()
            c.cache.sync()
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert all(bool((x == 7.0).all()) for x in junk)
        # a workspace that a capture makes is the graph's too
        c2 = Case([200, 90], h=2, g=4, pt=32)
        want = c2.run()
        c2.cache._spaces, c2.cache._space_bytes, c2.cache._space_held = [], 0, True
        graph2 = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph2, stream=s):
            o, lse = c2.run()
        own = c2.cache._spaces[-1]
        c2.cache.attend(0, c2.q[:1].expand(3000, -1, -1), c2.table[:1].repeat(3000, 1), c2.lengths[:1].repeat(3000), 200)
        assert c2.cache._spaces[0] is own and len(c2.cache._spaces) == 2
        graph2.replay()
        c2.cache.sync()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
