"""Attention over 4-bit pages whose values are far below 1, far above it, of unlike sizes in a row or along a sequence, or
behind a token that takes nearly all weight."""
import math

import pytest
import torch

from tests import packed_bound as K
from tests import packed_reference as P
from tests import paged_reference as R
from tests.test_gpu_paged import BF, HF, ints
from verified_kv_cache_poissoncomp_gb300.paged import PagedKV

pytestmark = pytest.mark.gpu


class Long:
    """One long sequence whose pages many sequences have in their tables, so that a CTA's run takes much of it: values
    v [tokens][h][d], and behind a first token of 2^gap times the others' weight."""

    def __init__(self, v, dtype, gap, g=1, q=1, pt=64, seqs=None, at=0):
        n, h, d = v.shape
        seqs = seqs or -(-220 * 304 * 64 // (n * h))  # some 100 turns a CTA at least
        gen = torch.Generator().manual_seed(n)
        kv = torch.zeros((1, n // pt, h, pt, 2, d))
        k = torch.randn((n, h, d), generator=gen) * 0.1
        k[..., :32] = 0
        k[at, :, :32] = gap * math.log(2) / 32
        for j, x in enumerate((k, v)):
            kv[0, :, :, :, j] = x.view(n // pt, pt, h, d).transpose(1, 2)
        self.kv = P.pack(kv.to(dtype)).cuda()
        self.one = (torch.randn((q, h * g, d), generator=gen) * 0.1).to(dtype).cuda()
        self.one[..., :32] = 1
        self.q = self.one.repeat(seqs, 1, 1)
        self.table = torch.arange(n // pt, dtype=torch.int32, device="cuda").repeat(seqs, 1)
        self.lengths = ints([n] * seqs)
        self.q_start = ints(range(0, seqs * q + 1, q)) if q > 1 else None
        self.cache = PagedKV(h, g, d, kv=self.kv, bits=4, dtype=dtype)
        self.n, self.seqs, self.count = n, seqs, q

    def check(self):
        o, lse = self.cache.attend(0, self.q, self.table, self.lengths, self.n, self.q_start, scale=1.0)
        self.cache.sync()
        starts = [0, self.count] if self.count > 1 else None
        wo, wl, to, tl, _ = K.attend(self.one, self.kv[0], self.table[:1], [self.n], starts, scale=1.0)
        R.close(o, wo.repeat(self.seqs, 1, 1), to.repeat(self.seqs, 1, 1), "o")
        R.close(lse, wl.repeat(self.seqs, 1), tl.repeat(self.seqs, 1), "lse")


def values(n, h, d, seed=0):
    return 1 + 0.3 * torch.randn((n, h, d), generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d,g,q", [(128, 1, 1), (128, 4, 3), (128, 8, 4), (64, 1, 1), (64, 8, 2)])
@pytest.mark.parametrize("size,gap", [(1.0, 20), (1e-1, 18), (1e-2, 20), (1e-3, 20), (1e-4, 18), (1e-4, 20)])
def test_behind_a_token_of_nearly_all_weight(dtype, d, g, q, size, gap):
    v = values(8192, 2, d) * size
    v[0] = 0
    Long(v, dtype, gap, g, q).check()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
def test_channels_of_unlike_sizes(dtype, d):
    v = values(4096, 2, d, 1)
    v[0] = 0
    for group, size in enumerate([1e-3, 500.0, 3e-2, 8.0][:d // 32]):
        v[..., 32 * group:32 * group + 32] *= size
    Long(v, dtype, 14, 4).check()
    Long(v, dtype, 0, 4, seqs=3).check()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("at", [0, 2000])
def test_sizes_that_rise_or_fall_along_a_sequence(dtype, up, at):
    n = 4096
    v = values(n, 2, 128, 2)
    size = 2.0 ** torch.linspace(-12, 12, n)
    v *= (size if up else size.flip(0))[:, None, None]
    Long(v, dtype, 10, 2, at=at).check()
    v[::977] *= 1.0 if dtype is BF else 0.5
    Long(v, dtype, 0, 2, q=3, seqs=2).check()


@pytest.mark.parametrize("size", [1e-6, 3e4, 1e5, 1e6])
@pytest.mark.parametrize("d", [64, 128])
def test_values_at_the_ends_of_what_steps_reach(size, d):
    v = values(512, 2, d, 3) * size * torch.where(torch.rand((512, 2, d), generator=torch.Generator().manual_seed(4)) < 0.5, -1.0, 1.0)
    Long(v, BF, 0, 4, seqs=3).check()
    if size < 65504 / 3:
        Long(v, HF, 3, 4, seqs=3).check()
