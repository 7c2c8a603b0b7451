"""Attention over 4-bit pages where a few tokens have the weight: the result is their values, whose sums over codes the tensor
cores may cut short."""
import pytest
import torch

from tests import packed_bound as K
from tests import paged_reference as R
from tests.test_gpu_packed import Packed
from tests.test_gpu_paged import BF, HF

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,g,qs", [(4, 1, 1), (4, 4, 1), (2, 8, 2), (2, 8, 5)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_codes_of_either_half_of_a_byte_are_summed_alike(dtype, d, h, g, qs):
    c = Packed([20 + 3 * i for i in range(40)], qs=[qs] * 40, h=h, g=g, d=d, pt=16, dtype=dtype, scale=3.0, kscale=2.0)
    o, lse = c.run()
    c.cache.sync()
    wo, wl, to, tl, _ = K.attend(c.q, c.kv[0], c.table, c.lengths, c.q_start)
    R.close(lse, wl, tl, "lse")
    R.close(o, wo, to, "o")
    if dtype is BF:
        return
    # Where results are near 0 (below 2^-6: their own rounding is 2^-18 at most) other errors can be seen.  Nibble i of a word is channel
    # i d / 8 + w: those of even i, held as 16 n like the odd ones, are off alike; held as n, by 16 times as much
    near, low = wo.abs() < 2.0 ** -6, torch.arange(d) // (d // 8) % 2 == 0
    off = o.double().cpu() - wo
    rms = [K.rms(off[..., x][near[..., x]]) for x in (low, ~low)]
    assert int(near.sum()) > 100  # (enough of them)
    assert rms[0] < 2 * rms[1]
