"""Sizes that PagedKV.weigh and PagedKV.evict refuse before the library has them (as 32-bit numbers), without a GPU."""
import ctypes

import pytest
import torch

from verified_kv_cache_poissoncomp_gb300 import binding as B
from verified_kv_cache_poissoncomp_gb300 import paged


class Library:
    """Takes the calls down."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def cache(monkeypatch):
    """An object of tensors on the CPU, whose library only takes the calls down."""
    monkeypatch.setattr(paged, "_current_stream", lambda index: 0)
    monkeypatch.setattr(paged, "_empty_strided", None)
    monkeypatch.setattr(paged, "_capturing", lambda: False)
    c = object.__new__(paged.PagedKV)
    c.ctx, c.dev, c._index, c._raw_stream, c._lib = None, torch.device("cpu"), 0, 0, Library()
    c.dtype, c.h, c.hq, c.d, c.layers, c.bits = torch.bfloat16, 2, 4, 64, 1, 16
    c.shape = B.verkv_shape(1, 1, 2, 2, 64, 1, 1)
    c.kv = torch.zeros((1, 8, 2, 16, 2, 64), dtype=torch.bfloat16)
    c._base, c._layer_bytes, c._code = c.kv.data_ptr(), 0, B.VERKV_BF16
    c._pages = B.verkv_pages(B.VERKV_BF16, 16, 8, c._base)
    c._spaces, c._needs, c._space_at, c._space_bytes, c._space_held = [], {"evict": 0}, None, 0, True
    c._known = lambda key, need: 256
    monkeypatch.setattr(B, "verkv_paged_evict_workspace_size", lambda *args: 256)
    return c


def operands(n=3):
    return torch.zeros((n, 4, 64), dtype=torch.bfloat16), torch.zeros((n, 4)), torch.zeros((n, 2), dtype=torch.int32), torch.zeros(n, dtype=torch.int32)


def places(count, n=3):
    """Weights of so many places, without their memory."""
    return torch.empty((n, 2, count), device="meta") if count > 1 << 20 else torch.zeros((n, 2, count))


@pytest.mark.parametrize("count,max_length", [(0, 1), (0, 32), (16, 17), (8, -1), (8, 2 ** 32 + 8), (8, 8 - 2 ** 32), (0, -(2 ** 32))])
def test_places_hold_the_lengths(cache, count, max_length):
    q, lse, table, n = operands()
    w = places(count)
    for call in (lambda: cache.weigh(0, q, lse, table, n, max_length, w), lambda: cache.weigh(0, q, lse, table, n, max_length, out=w),
                 lambda: cache.evict(0, table, n, max_length, w, 5, 1, 1)):
        with pytest.raises(ValueError):
            call()
    assert not cache._lib.calls


def test_places_are_counted_in_32_bits(cache, monkeypatch):
    q, lse, table, n = operands()
    monkeypatch.setattr(paged.PagedKV, "_weights", lambda self, t, shape, name: 4096)
    for count in (2 ** 30 + 1, 2 ** 32, 2 ** 32 + 16):
        w = places(count)
        for call in (lambda: cache.weigh(0, q, lse, table, n, 16, w), lambda: cache.evict(0, table, n, 16, w, 5, 1, 1)):
            with pytest.raises(ValueError):
                call()
    assert not cache._lib.calls
    cache.weigh(0, q, lse, table, n, 16, places(2 ** 30))
    assert cache._lib.calls[0][1][-1] == 2 ** 30


@pytest.mark.parametrize("keep,first,last", [(0, 0, 0), (-1, 0, 0), (4, 5, 0), (4, 2, 3), (4, -1, 0), (4, 0, -1), (4, 2 ** 32, 0), (4, 0, 2 ** 32 + 1),
                                             (4, 2 - 2 ** 32, 0), (2 ** 32 + 4, 1, 1), (2 ** 31, 1, 1)])
def test_what_is_kept_holds_the_first_and_the_last(cache, keep, first, last):
    _, _, table, n = operands()
    with pytest.raises(ValueError):
        cache.evict(0, table, n, 16, places(16), keep, first, last)
    assert not cache._lib.calls


def test_what_is_allowed_goes_on(cache):
    q, lse, table, n = operands()
    assert cache.weigh(0, q, lse, table, n, 16).shape == (3, 2, 16)
    cache.weigh(0, q, lse, table, n, 16, places(20))
    cache.evict(0, table, n, 16, places(16), 4, 2, 2)
    cache.evict(0, table, n, 0, places(0), 4, 4, 0)
    names = [name for name, _ in cache._lib.calls]
    assert names == ["verkv_paged_weigh"] * 2 + ["verkv_paged_evict"] * 2
    assert [a[-1] for name, a in cache._lib.calls[:2]] == [16, 20]
    # no lengths, no places: nothing to do
    assert cache.weigh(0, q, lse, table, n, 0).shape == (3, 2, 0)
    assert len(cache._lib.calls) == 4
    # no sequences: nothing to do, whatever the sizes
    q, lse, table, n = operands(0)
    assert cache.weigh(0, q, lse, table, n, 64).shape == (0, 2, 64)
    assert cache.weigh(0, q, lse, table, n, 64, places(10, 0)).shape == (0, 2, 10)
    assert cache.evict(0, table, n, 64, places(10, 0), 32, 4, 32)[1].shape == (0, 2, 32)
    assert len(cache._lib.calls) == 4
    assert isinstance(cache._lib.calls[2][1][3], B.verkv_span) and ctypes.sizeof(B.verkv_span) == 40 - 8
