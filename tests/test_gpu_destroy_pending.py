"""Contexts that go while work launched before, outside any capture, may still run: what it writes of the context's own
memory has to stay until then."""
import numpy as np
import pytest
import torch

from tests import parity as P
from verified_kv_cache_poissoncomp_gb300 import binding as B
from verified_kv_cache_poissoncomp_gb300 import inputs as I
from verified_kv_cache_poissoncomp_gb300.paged import PagedKV

pytestmark = pytest.mark.gpu


def engine(w, mode=B.VERKV_FETCH_MEMCPY):
    eng = P.make_engine(w, fetch_mode=mode)
    eng.compress(w.eta, w.n_sink, w.n_local, w.seed)
    eng.sync()
    return eng, torch.as_tensor(w.queries[0].view(np.int16)).to(eng.dev)


def test_a_selection_before_the_capture_is_waited_for():
    w = I.tiny()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        eng, q = engine(w)
        eng.attend(int(w.query_layer[0]), q, w.eps, w.delta)
        eng.fetch_refine()
        eng.sync()
        x = torch.zeros(8, device="cuda")
        graph, before = torch.cuda.CUDAGraph(), torch.cuda.Event()
        torch.cuda.synchronize()
        torch.cuda._sleep(40_000_000)  # some 20 ms
        before.record()
        eng.attend(int(w.query_layer[0]), q, w.eps, w.delta)
        graph.capture_begin(capture_error_mode="relaxed")
        x += 1
        eng.close()
        done = before.query()  # what is ahead of the selection
        x += 1
        graph.capture_end()
        assert done
        graph.replay()
        graph.replay()
    torch.cuda.synchronize()
    assert bool((x == 4).all())


def test_the_default_stream_is_waited_for():
    w = I.tiny()
    for mode in (B.VERKV_FETCH_MEMCPY, B.VERKV_FETCH_ZEROCOPY):
        eng, q = engine(w, mode)
        assert torch.cuda.current_stream().cuda_stream == 0
        after = torch.cuda.Event()
        torch.cuda._sleep(40_000_000)
        eng.attend(int(w.query_layer[0]), q, w.eps, w.delta)
        if mode == B.VERKV_FETCH_ZEROCOPY:
            eng.fetch_refine()
        after.record()
        eng.close()
        assert after.query()


def test_a_captured_selection_does_not_stand_for_the_last_one():
    # the selection in a capture has an event of its own: the one before it is still waited for
    w = I.tiny()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        eng, q = engine(w)
        layer = int(w.query_layer[0])
        eng.attend(layer, q, w.eps, w.delta)
        first = [t.clone() for t in eng.fetch_refine()[:2]]
        torch.cuda.synchronize()
        graph, before = torch.cuda.CUDAGraph(), torch.cuda.Event()
        torch.cuda._sleep(40_000_000)
        before.record()
        eng.attend(layer, q, w.eps, w.delta)
        graph.capture_begin(capture_error_mode="relaxed")
        eng.attend(layer, q, w.eps, w.delta)
        eng.close()
        done = before.query()
        graph.capture_end()  # (not replayed: its context is gone)
        assert done
        again, _ = engine(w)
        again.attend(layer, q, w.eps, w.delta)
        for a, b in zip(first, again.fetch_refine()[:2]):
            assert torch.equal(a, b)
        again.sync()
        again.close()


def test_objects_of_the_default_stream_go_during_a_capture():
    w = I.tiny()
    eng, q = engine(w)
    eng.attend(int(w.query_layer[0]), q, w.eps, w.delta)
    cache = PagedKV(2, 2, 64, num_pages=2)
    x = torch.zeros(8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x += 1
        eng.close()
        cache.close()
        x += 1
    graph.replay()
    torch.cuda.synchronize()
    assert bool((x == 2).all())
