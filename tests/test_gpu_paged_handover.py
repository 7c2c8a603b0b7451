"""Two attention kernels side by side: the second one reads nothing before what the stream wrote ahead of
the call is there, call after call and in a graph."""
import pytest
import torch

from tests.test_gpu_paged import BF, HF, Case

pytestmark = pytest.mark.gpu

SHAPES = [([300 + 7 * i for i in range(40)], 1, [5000], BF, 128), ([90 + 31 * i for i in range(8)], 5, [3000], HF, 64),
          ([2000] * 3, 12, [700], BF, 128), ([50] * 160, 1, [4000], BF, 128)]


def sets(lengths, qs, prefixes, dtype, d):
    """A case, and several states of all that its calls read, with what the call makes of each."""
    c = Case(lengths, qs=[qs] * len(lengths), prefixes=prefixes, h=2, g=4, d=d, pt=64, dtype=dtype)
    got = []
    for k in range(3):
        perm = torch.randperm(c.kv.shape[1], device="cuda", generator=c.gen)
        back = torch.argsort(perm).to(torch.int32)
        # other queries, lengths, and the same pages at other places
        got.append({"q": torch.randn(c.q.shape, device="cuda", generator=c.gen).to(dtype),
                    "lengths": (c.lengths - 3 * k).clamp(min=0), "prefix_lengths": (c.prefix_lengths - 65 * k).clamp(min=0),
                    "kv": c.kv[:, perm].clone(), "table": back[c.table.long()], "prefix_table": back[c.prefix_table.long()]})
    for s in got:
        write(c, s)
        torch.cuda.synchronize()
        s["o"], s["lse"] = c.check()
        s["o"], s["lse"] = s["o"].clone(), s["lse"].clone()
    return c, got


def write(c, s):
    # the pages and the queries last: right ahead of the call
    for name in ("table", "prefix_table", "lengths", "prefix_lengths", "kv", "q"):
        getattr(c, name).copy_(s[name])


@pytest.mark.parametrize("lengths,qs,prefixes,dtype,d", SHAPES)
def test_what_is_written_right_ahead(lengths, qs, prefixes, dtype, d):
    c, got = sets(lengths, qs, prefixes, dtype, d)
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for k in range(600):
        s = got[k % 3]
        write(c, s)
        o, lse = c.run()
        bad += (o != s["o"]).any() | (lse != s["lse"]).any()
    c.cache.sync()
    assert not bad.item()


@pytest.mark.parametrize("lengths,qs,prefixes,dtype,d", SHAPES[:2])
def test_the_same_in_a_graph(lengths, qs, prefixes, dtype, d):
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        c, got = sets(lengths, qs, prefixes, dtype, d)
        graph, outs = torch.cuda.CUDAGraph(), []
        with torch.cuda.graph(graph, stream=st):
            for s in got + got:
                write(c, s)
                outs.append(c.run())
        bad = torch.zeros((), dtype=torch.int64, device="cuda")
        for _ in range(100):
            graph.replay()
            for s, (o, lse) in zip(got + got, outs):
                bad += (o != s["o"]).any() | (lse != s["lse"]).any()
        c.cache.sync()
        assert not bad.item()


def test_whatever_the_workspace_holds():
    # bytes of any kind, and what a call that was cut off would leave there
    lengths, qs, prefixes, dtype, d = SHAPES[0]
    c, got = sets(lengths, qs, prefixes, dtype, d)
    for fill in (0, 255, 0x71):
        for s in c.cache._spaces:
            s.fill_(fill)
        o, lse = c.run()
        c.cache.sync()
        assert torch.equal(o, got[-1]["o"]) and torch.equal(lse, got[-1]["lse"])
    word = c.cache._spaces[-1][:8]
    assert not word.any()  # cleared for the next call
    word.copy_(torch.tensor([0xF1, 0x28, 0x4B, 0xE6, 0x71, 0x3A, 0x5C, 0x9D], dtype=torch.uint8, device="cuda"))
    o, lse = c.run()
    c.cache.sync()
    assert torch.equal(o, got[-1]["o"]) and torch.equal(lse, got[-1]["lse"])
