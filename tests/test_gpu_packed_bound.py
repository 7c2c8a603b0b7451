"""Attention over 4-bit pages, each output against a bound of its own sums (packed_bound.py), and all of them by their root
mean square."""
import pytest
import torch

from tests import packed_bound as K
from tests import packed_reference as P
from tests import paged_reference as R
from tests.test_gpu_packed import Packed
from tests.test_gpu_paged import BF, HF

pytestmark = pytest.mark.gpu


def check(c, scale=0.0, rms=True):
    o, lse = c.run(scale=scale)
    c.cache.sync()
    wo, wl, to, tl, more = K.attend(c.q, c.kv[0], c.table, c.lengths, c.q_start, c.prefix_table, c.prefix_lengths, c.group_start,
                                    scale, c.prior)
    R.close(lse, wl, tl, "lse")
    R.close(o, wo, to, "o")
    if rms:
        n = c.max_length + c.max_prefix
        assert K.rms(o.double().cpu() - wo) <= K.rms_bound(wo, more["size"], n, c.q.dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pt", [16, 64, 256])
def test_pages_of_every_size(dtype, d, pt):
    check(Packed([1, 15, 16, 17, 63, 64, 65, 0, 127, 129, 300, 513], h=2, g=4, d=d, pt=pt, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("h,g,qs", [(1, 1, [1, 1, 1]), (3, 4, [3, 1, 6]), (2, 8, [5, 17, 2])])
def test_queries_prefixes_and_a_prior(dtype, h, g, qs):
    check(Packed([70, 5, 200], qs=qs, h=h, g=g, prefixes=[333], pt=32, dtype=dtype).with_prior(), rms=False)
    check(Packed([70, 5, 200], qs=qs, h=h, g=g, prefixes=[90, 33], groups=[0, 1, 3], pt=32, d=64, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lengths,prefix,qs", [([4000, 9000, 2500, 0, 7001], 0, 1), ([2000] * 3, 20001, 2), ([300, 6000], 0, 7), ([5, 60, 33], 4099, 1)])
def test_long_runs(dtype, lengths, prefix, qs):
    check(Packed(lengths, qs=[qs] * len(lengths), prefixes=[prefix] if prefix else (), h=2, g=4, d=64 if qs == 2 else 128, pt=64, dtype=dtype))


@pytest.mark.parametrize("size", [1e-4, 300.0])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_small_and_large_values(size, dtype):
    c = Packed([400, 90], h=2, g=4, pt=16, dtype=dtype)
    x = torch.randn((1, c.kv.shape[1], 2, 16, 2, 128), device="cuda", generator=c.gen)
    x[..., 1, :] *= size
    c.kv.copy_(P.pack(x.to(dtype)))
    check(c, rms=dtype is BF)
