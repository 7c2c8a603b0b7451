"""Attention over the paged cache against float64: shared prefixes, own pages, several queries a
sequence, a prior state, empty rows, garbage behind the lengths, graphs, refusals."""
import math

import pytest
import torch

from tests import paged_reference as R
from verified_kv_cache_poissoncomp_gb300 import binding as B
from verified_kv_cache_poissoncomp_gb300.paged import PagedKV, Rope

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
NAN = float("nan")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """A pool whose unused places hold NaN, tables in random page order, and random queries."""

    def __init__(self, lengths, qs=None, prefixes=(), groups=None, h=2, g=4, d=128, pt=16, dtype=BF, seed=0, spare=3,
                 layers=1, scale=1.0, kscale=1.0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        r = lambda *s: torch.randn(s, device="cuda", generator=gen).to(dtype)  # noqa: E731
        S = len(lengths)
        self.qs = qs or [1] * S
        self.max_length, self.max_prefix = max(lengths, default=0), max(prefixes, default=0)
        own, pre = max(1, -(-self.max_length // pt)), max(1, -(-self.max_prefix // pt))
        pages = S * own + len(prefixes) * pre + spare
        self.kv = torch.full((layers, pages, h, pt, 2, d), NAN, dtype=dtype, device="cuda")
        order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
        self.table = order[:S * own].view(S, own)
        self.prefix_table = order[S * own:S * own + len(prefixes) * pre].view(len(prefixes), pre) if prefixes else None
        for tab, ns in ((self.table, lengths), (self.prefix_table, prefixes)):
            for s, n in enumerate(ns):
                for p in range(-(-n // pt)):
                    c = min(pt, n - p * pt)
                    x = r(layers, h, c, 2, d)
                    x[..., 0, :] *= kscale
                    self.kv[:, tab[s, p].long(), :, :c] = x
        self.lengths, self.prefix_lengths = ints(list(lengths)), ints(list(prefixes)) if prefixes else None
        self.q_start = ints([sum(self.qs[:i]) for i in range(S + 1)]) if any(n != 1 for n in self.qs) else None
        self.group_start = ints(groups) if groups else None
        self.q = r(sum(self.qs), h * g, d) * scale
        self.prior = None
        self.gen, self.h, self.g, self.d = gen, h, g, d
        self.cache = PagedKV(h, g, d, kv=self.kv)

    def with_prior(self):
        n = self.q.shape[0]
        self.prior = (torch.randn((n, self.h * self.g, self.d), device="cuda", generator=self.gen),
                      2 + 2 * torch.randn((n, self.h * self.g), device="cuda", generator=self.gen))
        self.prior[1][0, 0], self.prior[0][0, 0] = -math.inf, NAN  # it summed nothing: its values are not used
        return self

    def run(self, layer=0, **kw):
        a = dict(q_start=self.q_start, prefix_table=self.prefix_table, prefix_lengths=self.prefix_lengths,
                 max_prefix=self.max_prefix, group_start=self.group_start, prior=self.prior)
        return self.cache.attend(layer, self.q, self.table, self.lengths, self.max_length, **{**a, **kw})

    def want(self, layer=0, scale=0.0):
        return R.attend(self.q, self.kv[layer], self.table, self.lengths, self.q_start, self.prefix_table,
                        self.prefix_lengths, self.group_start, scale, self.prior)

    def check(self, layer=0, scale=0.0, **kw):
        o, lse = self.run(layer, scale=scale, **kw)
        self.cache.sync()
        wo, wl, to, tl = self.want(layer, scale)
        R.close(lse, wl, tl, "lse")
        R.close(o, wo, to, "o")
        return o, lse


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pt", [16, 32, 64, 128, 256])
def test_pages_of_every_size(dtype, d, pt):
    # lengths around a page, a 16-token group, a 64-token step and several of each; one empty
    Case([1, 15, 16, 17, 63, 64, 65, 0, 127, 129, 300, 513], h=2, g=4, d=d, pt=pt, dtype=dtype).check()


@pytest.mark.parametrize("h,g", [(1, 1), (1, 2), (3, 4), (8, 4), (2, 8), (1, 8)])
def test_head_shapes(h, g):
    Case([70, 5, 200], h=h, g=g, prefixes=[333], pt=32).check()
    Case([70, 5, 200], qs=[3, 1, 6], h=h, g=g, prefixes=[333], pt=32, d=64).check()


@pytest.mark.parametrize("qs", [[1] * 7, [2, 1, 4, 3, 8, 5, 2], [1, 0, 3, 0, 0, 2, 1], [17, 40, 1, 9, 64, 5, 33]])
def test_queries_of_each_sequence(qs):
    # fewer cached tokens than queries in some: the first queries see nothing of their own
    c = Case([9, 1, 64, 3, 0, 200, 31], qs=qs, h=2, g=4, pt=16, dtype=HF)
    o, lse = c.check()
    first = sum(qs[:4])
    if qs[4]:
        assert not o[first].any() and bool((lse[first] == -math.inf).all())
    Case([9, 1, 64, 3, 0, 200, 31], qs=qs, h=2, g=4, pt=16, prefixes=[77], dtype=HF).check()


@pytest.mark.parametrize("seqs", [1, 3, 8, 9, 32, 33, 70, 150])
@pytest.mark.parametrize("prefix", [1, 64, 127, 1000, 4099])
def test_one_prefix_for_all(seqs, prefix):
    Case([(7 * i) % 90 for i in range(seqs)], prefixes=[prefix], h=1 + (seqs < 9), g=4, pt=64).check()


@pytest.mark.parametrize("rows,lengths,prefix", [
    (4, [4000, 9000, 2500, 0, 7001], 0), (4, [3000] * 3, 40001), (16, [2500] * 2, 30001), (32, [2000] * 3, 30001),
    (24, [9000, 1, 5000, 12000], 0), (64, [1000] * 2, 30001), (200, [6000, 300, 9001], 0), (400, [200], 30001)])
def test_long_runs(rows, lengths, prefix):
    # every CTA takes many steps of several units, and units end inside its run
    qs = max(1, rows // 4 // (len(lengths) if prefix else 1))
    Case(lengths, qs=[qs] * len(lengths), prefixes=[prefix] if prefix else (), h=8, g=4, d=64, pt=64).check()


@pytest.mark.parametrize("seqs,groups,qs,g", [(2000, 0, 1, 2), (2000, 500, 1, 8), (930, 310, 1, 8), (300, 0, 5, 8), (290, 290, 9, 4)])
def test_more_segments_than_are_kept_in_shared_memory(seqs, groups, qs, g):
    at = [i * seqs // max(groups, 1) for i in range(groups)] + [seqs] if groups else None
    Case([(5 * i) % 39 for i in range(seqs)], qs=[qs] * seqs, prefixes=[(11 * i) % 70 for i in range(groups)], groups=at,
         h=1, g=g, d=64, pt=16).check()


@pytest.mark.parametrize("prefixes", [[5000, 4990, 4999], [3000, 0, 2900], [700, 600, 650, 1], [1, 0, 0, 9000], [128, 129], [0, 0]])
@pytest.mark.parametrize("qs,g", [(1, 4), (9, 8), (40, 4)])
def test_few_groups_of_unequal_prefixes(prefixes, qs, g):
    # few units, which may each get as many runs of the line: some runs have nothing to do
    n = len(prefixes)
    Case([(37 * i) % 150 for i in range(6 * n)], qs=[qs] * (6 * n), prefixes=prefixes, groups=[6 * i for i in range(n + 1)],
         h=2, g=g, d=64, pt=64).check()


@pytest.mark.parametrize("qs", [[1] * 5, [9, 30, 9, 0, 12]])
@pytest.mark.parametrize("groups", [[0, 0, 5, 5], [0, 2, 2, 5], [0, 0, 0, 5], [0, 5, 5, 5]])
def test_groups_without_sequences(groups, qs):
    Case([70, 0, 5, 300, 129], qs=qs, prefixes=[900, 333, 64], groups=groups, h=2, g=4, d=64, pt=32).check()


@pytest.mark.parametrize("lengths,qs", [([5000], [70]), ([5000, 4700], [33, 34]), ([900, 0, 910], [40, 1, 50]), ([4000, 3990], [300, 1])])
def test_few_long_sequences_with_many_queries(lengths, qs):
    Case(lengths, qs=qs, h=2, g=4, d=128, pt=32).check()


@pytest.mark.parametrize("queries,length,g", [(701, 901, 2), (1100, 1100, 8), (333, 5000, 1)])
def test_a_prompt_among_decoding_sequences(queries, length, g):
    # most queries are one sequence's, and the others have one each
    Case([40, length, 0, 700], qs=[1, queries, 1, 1], prefixes=[129], h=2, g=g, d=128, pt=32).check()


@pytest.mark.parametrize("d,dtype,qs", [(64, BF, 1), (128, HF, 1), (128, BF, 3), (64, HF, 5)])
def test_groups_with_their_own_prefixes(d, dtype, qs):
    # groups of 40, 0, 1, 25 sequences; a prefix without tokens, prefixes without sequences
    groups = [0, 40, 40, 41, 66, 66]
    c = Case([(11 * i) % 130 for i in range(66)], qs=[1 + (i % qs) for i in range(66)], prefixes=[700, 300, 0, 129, 50],
             groups=groups, h=2, g=2, d=d, pt=32, dtype=dtype)
    c.check()
    c.with_prior().check()


@pytest.mark.parametrize("lengths,prefixes", [([30, 0, 500], ()), ([30, 0, 500], (100,)), ([0, 0, 0], ()), ([0, 0, 0], (65,))])
def test_prior_state(lengths, prefixes):
    c = Case(lengths, prefixes=prefixes, h=2, g=4).with_prior()
    c.check()
    c.prior[1][:] = 60.0  # all the weight is elsewhere
    o, lse = c.check()
    prior = c.prior[0].double().cpu()[1:]
    R.close(o[1:], prior, R.half_step(BF) * prior.abs() + 1e-6, "o of the prior")


def test_nothing_to_see():
    c = Case([0, 0], h=1, g=2, d=64)
    o, lse = c.check()
    assert not o.any() and bool((lse == -math.inf).all())
    # no own tokens at all, or none of anything
    c = Case([0] * 5, prefixes=[200], h=1, g=4)
    c.table = None
    o, lse = c.cache.attend(0, c.q, None, None, 0, prefix_table=c.prefix_table, prefix_lengths=c.prefix_lengths, max_prefix=200)
    wo, wl, to, tl = R.attend(c.q, c.kv[0], None, None, None, c.prefix_table, c.prefix_lengths)
    R.close(o, wo, to, "o")
    R.close(lse, wl, tl, "lse")
    o, lse = c.cache.attend(0, c.q, None, None, 0)
    assert not o.any() and bool((lse == -math.inf).all())
    c.cache.sync()


@pytest.mark.parametrize("kscale,scale", [(1.0, 30.0), (30.0, 1.0)])
def test_large_logits(kscale, scale):
    # one token takes nearly all the weight, and the running maximum rises late
    c = Case([400, 77, 1000], prefixes=[900], scale=scale, kscale=kscale, h=2, g=4, dtype=HF)
    c.check()
    Case([400] * 40, prefixes=[900], scale=scale, kscale=kscale, h=1, g=4, dtype=BF).check()


@pytest.mark.parametrize("scale", [0.3, -0.05, 1e-6])
def test_scale(scale):
    Case([100, 33], prefixes=[130], h=2, g=2, d=64).check(scale=scale)


def test_strided_queries_layers_and_given_outputs():
    c = Case([100, 33, 64], prefixes=[130], h=2, g=2, d=64, layers=3)
    wide = torch.full((3, 4 + 3, 128), NAN, dtype=BF, device="cuda")
    wide[:, 2:6, 64:] = c.q
    c.q = wide[:, 2:6, 64:]
    o, lse = torch.full((3, 4, 64), NAN, dtype=BF, device="cuda"), torch.full((3, 4), NAN, device="cuda")
    a, b = c.check(2, out=o, lse=lse)
    assert a is o and b is lse
    head_major = c.q.transpose(0, 1).contiguous().transpose(0, 1)  # heads outermost
    c.q = head_major
    o2, lse2 = c.check(2)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


def test_not_a_number_stays_in_its_sequence():
    c = Case([100, 33, 64], h=2, g=2, d=64)
    o, lse = c.run()
    page = int(c.table[1, 1])
    c.kv[0, page, 0, 3, 0, 5] = NAN  # a key of sequence 1, KV head 0
    o2, lse2 = c.run()
    c.cache.sync()
    assert bool(torch.isnan(o2[1, :2]).all()) and bool(torch.isnan(lse2[1, :2]).all())
    for x, y in ((o, o2), (lse, lse2)):
        assert torch.equal(x[0], y[0]) and torch.equal(x[2], y[2]) and torch.equal(x[1, 2:], y[1, 2:])
    c.q[2, 0, 0] = NAN
    o3, lse3 = c.run()
    assert bool(torch.isnan(o3[2, 0]).all()) and bool(torch.isnan(lse3[2, 0])) and torch.equal(o3[2, 1:], o[2, 1:])


@pytest.mark.parametrize("d,dtype,lengths", [(128, HF, (300, 60)), (64, BF, (300, 60)), (128, BF, (1200, 9, 40)), (64, HF, (129, 1, 128))])
def test_same_bits_with_units_of_one_step_behind_longer_ones(d, dtype, lengths):
    # a run of the line holds many units, and the warps that share a unit leave it at their own times
    n = 132
    c = Case(list(lengths) * (n // len(lengths)), qs=[9] * n, h=8, g=8, d=d, dtype=dtype, pt=64)
    o, lse = c.check()
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(1500):
        o1, lse1 = c.run()
        bad += (o1 != o).any() | (lse1 != lse).any()
    assert not bad.item()


def test_same_bits_again_and_whatever_the_bound():
    c = Case([300, 5, 800, 64] * 10, prefixes=[2000], h=2, g=4)
    o, lse = c.run()
    for _ in range(5):
        o2, lse2 = c.run()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    c.check()


def test_long_tables_pass_32_bits():
    # 9 GB of pages: elements past 2^32, tokens in the last pages
    h, pt, d = 8, 64, 128
    pages = (9 << 30) // (h * pt * 4 * d)
    kv = torch.empty((1, pages, h, pt, 2, d), dtype=BF, device="cuda")
    last = list(range(pages - 9, pages))
    for p in last:
        kv[0, p].normal_()
    assert kv[0, :last[0]].numel() > 1 << 32
    c = PagedKV(h, 1, d, kv=kv)
    q = torch.randn((2, h, d), device="cuda").to(BF)
    table, lengths = ints([last[:4], last[4:8]]), ints([250, 256])
    pre, plen = ints([[last[8]]]), ints([60])
    k = torch.randn((2, h, d), device="cuda").to(BF)
    c.append(0, k, k, ints([0, 1]), ints([249, 255]), table)
    assert torch.equal(kv[0, last[3], :, 57, 0], k[0]) and torch.equal(kv[0, last[7], :, 63, 1], k[1])
    o, lse = c.attend(0, q, table, lengths, 256, prefix_table=pre, prefix_lengths=plen, max_prefix=64)
    c.sync()
    wo, wl, to, tl = R.attend(q, kv[0], table, lengths, None, pre, plen)
    R.close(o, wo, to, "o")
    R.close(lse, wl, tl, "lse")


def test_captured_graph_follows_lengths_and_tables():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = Case([200, 90, 150, 64], prefixes=[500], h=2, g=4, pt=32)
        c.max_length, c.max_prefix = 224, 512
        c.run()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            o, lse = c.run()
        for lengths, plen in (([200, 90, 150, 64], 500), ([1, 0, 33, 200], 64), ([65, 64, 63, 0], 0)):
            c.lengths.copy_(ints([min(n, m) for n, m in zip(lengths, [200, 90, 150, 64])]))
            c.prefix_lengths.fill_(plen)
            c.q.normal_()
            graph.replay()
            c.cache.sync()
            wo, wl, to, tl = c.want()
            R.close(lse, wl, tl, "lse")
            R.close(o, wo, to, "o")
            o2, lse2 = c.run()  # an eager call between replays
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
            c.cache.sync()


def test_two_objects_on_two_streams():
    a = [torch.cuda.Stream() for _ in range(2)]
    cs = []
    for i, s in enumerate(a):
        with torch.cuda.stream(s):
            cs.append(Case([500, 30, 700] * 6, prefixes=[3000], h=2, g=4, seed=i))
            alone = cs[-1].run()
            cs[-1].cache.sync()
            cs[-1].alone = [x.clone() for x in alone]
    torch.cuda.synchronize()
    for _ in range(10):
        outs = []
        for c, s in zip(cs, a):
            with torch.cuda.stream(s):
                outs.append(c.run())
        torch.cuda.synchronize()
        for c, o in zip(cs, outs):
            assert torch.equal(o[0], c.alone[0]) and torch.equal(o[1], c.alone[1])


def test_bad_pages_lengths_and_starts_are_reported():
    c = Case([100, 33, 64], qs=[2, 1, 3], prefixes=[130], groups=[0, 3], h=2, g=2, d=64)
    good = c.run()
    c.cache.sync()
    pages = c.kv.shape[1]

    def reported(change, back):
        change()
        c.run()
        with pytest.raises(B.VerkvError) as e:
            c.cache.sync()
        assert e.value.status == B.VERKV_EINVAL
        back()
        o, lse = c.run()
        c.cache.sync()
        assert torch.equal(o, good[0]) and torch.equal(lse, good[1])

    for tab in (c.table, c.prefix_table):
        was = int(tab[0, 1])
        for x in (pages, -1, 1 << 30):
            reported(lambda: tab[0].__setitem__(1, x), lambda: tab[0].__setitem__(1, was))
    for arr, i, x in ((c.lengths, 1, 101), (c.lengths, 0, -1), (c.prefix_lengths, 0, 131), (c.q_start, 1, 7), (c.q_start, 0, 1),
                      (c.q_start, 2, 1), (c.q_start, 3, 5), (c.group_start, 0, 1), (c.group_start, 1, 2), (c.group_start, 1, 9)):
        was = int(arr[i])
        reported(lambda: arr.__setitem__(i, x), lambda: arr.__setitem__(i, was))


def test_a_spare_page_id_is_not_looked_at():
    # ids behind a sequence's last page may be anything
    c = Case([100, 33, 64], h=2, g=2, d=64, pt=16)
    good = c.run()
    c.table[1, 3:] = -1
    c.table[2, 4:] = 1 << 30
    o, lse = c.run()
    c.cache.sync()
    assert torch.equal(o, good[0]) and torch.equal(lse, good[1])


def test_refusals():
    c = Case([100, 33, 64], prefixes=[130], h=2, g=2, d=64)
    n0 = B.verkv_launch_counts(c.cache.ctx)
    full = dict(prefix_table=c.prefix_table, prefix_lengths=c.prefix_lengths, max_prefix=130)
    at = c.cache.attend
    for i, call in enumerate([
            lambda: at(0, c.q.half(), c.table, c.lengths, 100), lambda: at(0, c.q[:, :3], c.table, c.lengths, 100),
            lambda: at(1, c.q, c.table, c.lengths, 100), lambda: at(-1, c.q, c.table, c.lengths, 100),
            lambda: at(0, c.q, c.table.long(), c.lengths, 100), lambda: at(0, c.q, c.table, c.lengths[:2], 100),
            lambda: at(0, c.q, c.table[:, :2], c.lengths, 32), lambda: at(0, c.q, c.table, c.lengths, 100, q_start=c.lengths),
            lambda: at(0, c.q, c.table, c.lengths, 100, prior=(c.q, c.q)),
            lambda: at(0, c.q, c.table, c.lengths, 100, out=torch.empty_like(c.q)[:2]),
            lambda: at(0, c.q, c.table, c.lengths, 100, lse=torch.empty(3, 4))]):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    for i, call in enumerate([
            lambda: at(0, c.q, c.table, c.lengths, c.table.shape[1] * 16 + 1), lambda: at(0, c.q, c.table, c.lengths, -1),
            lambda: at(0, c.q[:2], c.table, c.lengths, 100), lambda: at(0, c.q, c.table, c.lengths, 100, scale=NAN),
            lambda: at(0, c.q, c.table, c.lengths, 100, group_start=ints([0])),
            lambda: at(0, c.q, c.table, c.lengths, 100, prefix_table=c.prefix_table.repeat(2, 1),
                       prefix_lengths=c.prefix_lengths.repeat(2), max_prefix=130),
            lambda: at(0, c.q, c.table, c.lengths, 100, **{**full, "max_prefix": 1 << 20})]):
        with pytest.raises(B.VerkvError) as e:
            call()
            pytest.fail(f"call {i} was not refused")
        assert e.value.status == B.VERKV_EINVAL
    # the workspace
    L, q = B.lib(), c.cache._rows(c.q, 3, 4, "q")
    own = B.verkv_span(c.table.data_ptr(), 3, c.table.shape[1], c.lengths.data_ptr(), 100)
    need = B.verkv_paged_workspace_size(c.cache.shape, 3, 0, 3)
    ws, o = torch.empty(need + 256, dtype=torch.uint8, device="cuda"), torch.empty_like(c.q)
    go = lambda p, n, out=o.data_ptr(): L.verkv_paged_attend(  # noqa: E731
        c.cache.ctx, c.cache._layer(0), 3, 3, q, None, own, None, None, 0.0, None, None, out, None, p, n)
    assert go(ws.data_ptr(), need - 1) == go(ws.data_ptr() + 16, need) == go(None, need) == B.VERKV_EINVAL
    assert go(ws.data_ptr(), need, None) == go(ws.data_ptr(), need, o.data_ptr() + 4) == B.VERKV_EINVAL
    assert B.verkv_launch_counts(c.cache.ctx) == n0
    with torch.cuda.stream(torch.cuda.Stream()):
        with pytest.raises(ValueError):
            at(0, c.q, c.table, c.lengths, 100)
    o, lse = at(0, c.q[:0], c.table[:0], c.lengths[:0], 0)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    assert B.verkv_launch_counts(c.cache.ctx) == n0
    assert go(ws.data_ptr(), need) == B.VERKV_OK  # lse is optional
    c.cache.sync()


def test_refusals_of_far_bounds():
    # a bound whose tokens or steps 31 bits do not count (the table is said to be as wide as that), and a
    # scale that float32 does not hold in units of log 2
    c = Case([100, 33, 64], h=2, g=2, d=64, pt=16)
    n0 = B.verkv_launch_counts(c.cache.ctx)
    L, q, o = B.lib(), c.cache._rows(c.q, 3, 4, "q"), torch.empty_like(c.q)
    ws, nbytes = c.cache._space(3, 0, 3)
    for bound, scale in ((1 << 30, 3e38), ((1 << 30) + 1, 0.0), ((1 << 31) - 1, 0.0), (100, -3e38)):
        own = B.verkv_span(c.table.data_ptr(), 3, 1 << 27, c.lengths.data_ptr(), bound)
        assert L.verkv_paged_attend(c.cache.ctx, c.cache._layer(0), 3, 3, q, None, own, None, None, scale, None, None,
                                    o.data_ptr(), None, ws, nbytes) == B.VERKV_EINVAL
    assert B.verkv_launch_counts(c.cache.ctx) == n0
    c.cache.sync()


def test_devices_without_an_index():
    c = Case([20, 3], h=1, g=2, d=64)
    rope = Rope([1.0] * 32, device="cuda")
    assert rope.dev == c.cache.dev == PagedKV(1, 2, 64, device="cuda").dev
    q, _ = c.cache.norm_rotate(c.q, None, ints([0, 0]), rope)
    c.cache.sync()
    assert torch.equal(q, c.q)


def test_the_callers_device_is_left_as_it_was():
    was = torch.cuda.current_device()
    c = Case([100, 33], h=2, g=2, d=64)
    c.run()
    c.cache.norm_rotate(c.q, None)
    assert torch.cuda.current_device() == was
    c.cache.sync()


def test_decode_behind_a_verified_context():
    """The operators as they are used: a prompt's keys rotated into the full cache, compressed, then
    decoded from: each step normalises and rotates, appends, attends its own pages, and joins what the
    library says of the compressed context -- here its exact attention, so that the whole is exact."""
    import numpy as np

    from verified_kv_cache_poissoncomp_gb300.engine import VerKV, default_cap

    b, h, g, d, n, steps, pt = 3, 2, 4, 64, 500, 21, 16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    r = lambda *s: torch.randn(s, device="cuda", generator=gen).to(BF)  # noqa: E731
    freqs = torch.tensor([1e4 ** (-2 * j / d) for j in range(d // 2)], dtype=torch.float64)
    rope, wq, wk = Rope(freqs), r(d), r(d)
    cache = PagedKV(h, g, d, page_tokens=pt, num_pages=b * 3 + 1)
    prompt_k, prompt_v = r(b * n, h, d), r(b * n, h, d)
    pos = torch.arange(n, dtype=torch.int32, device="cuda").repeat(b)
    kv = torch.empty((b, h, n, 2, d), dtype=BF, device="cuda")
    for s in range(b):
        part = slice(s * n, (s + 1) * n)
        cache.norm_rotate(None, prompt_k[part], pos[part], rope, None, wk, k_out=kv[s, :, :, 0].transpose(0, 1))
        kv[s, :, :, 1] = prompt_v[part].transpose(0, 1)
    eng = VerKV(b, 1, h, g, d, n, default_cap(n, 1 / 4))
    tau = np.random.default_rng(0).uniform(0.1, 1, (b * h, n)).astype(np.float32)
    eng.load(tau, kv.view(b * h, n, 2, d).view(torch.int16).cpu().numpy().view(np.uint16))
    eng.compress(1 / 4, 4, 16, seed=0)
    table = torch.arange(1, b * 3 + 1, dtype=torch.int32, device="cuda").view(b, 3).flip(1).contiguous()
    seq = torch.arange(b, dtype=torch.int32, device="cuda")
    length = torch.zeros(b, dtype=torch.int32, device="cuda")
    all_k = [kv[s, :, :, 0].double().cpu() for s in range(b)]
    all_v = [kv[s, :, :, 1].double().cpu() for s in range(b)]
    for step in range(steps):
        q, k, v = r(b, h * g, d), r(b, h, d), r(b, h, d)
        qr = cache.append(0, k, v, seq, length, table, length + n, rope, wk, q=q, q_weight=wq)
        length += 1
        o, lse = eng.attend_dense_host(0, qr.view(torch.int16))
        o, lse = cache.attend(0, qr, table, length, 48, prior=(o, lse))
        # and with the estimate of the verified path: the same call takes it
        eng.attend(0, qr.view(torch.int16), 0.05, 0.05)
        cache.attend(0, qr, table, length, 48, prior=eng.fetch_refine()[:2])
        cache.sync()
        eng.sync()
        at = torch.full((b,), n + step, dtype=torch.int32)
        kr, kt = R.norm_rotate(k, at, freqs, False, wk, 1e-6)
        qw, qt = R.norm_rotate(q, at, freqs, False, wq, 1e-6)
        R.close(qr, qw, qt, "q")
        page = table[:, step // pt].long()
        R.close(cache.kv[0, page, :, step % pt, 0], kr, kt, "k")
        for s in range(b):
            all_k[s] = torch.cat((all_k[s], cache.kv[0, page[s], :, step % pt, 0].double().cpu()[:, None]), 1)
            all_v[s] = torch.cat((all_v[s], v[s].double().cpu()[:, None]), 1)
            x = torch.einsum("hgd,hnd->hgn", qr[s].double().cpu().view(h, g, d), all_k[s]) / math.sqrt(d)
            p = torch.softmax(x, -1)
            want = torch.einsum("hgn,hnd->hgd", p, all_v[s])
            A = torch.einsum("hgn,hnd->hgd", p, all_v[s].abs())
            # the prior's own bar is 1e-3 of the largest value of o and of lse
            tol = 2 * R.half_step(BF) * A + 1e-3 * (want.abs().amax(-1, keepdim=True) + 2 * A)
            R.close(o[s].view(h, g, d), want, tol, f"o at step {step}")
            R.close(lse[s].view(h, g), torch.logsumexp(x, -1), torch.full((h, g), 1.1e-3, dtype=torch.float64), "lse")
    eng.close()
