"""The bound that attention over 4-bit pages is held to, without a GPU: it lets roundings through, and refuses outputs
that lost a part of the values."""
import pytest
import torch

from tests import packed_bound as K
from tests import packed_reference as P
from tests import paged_reference as R


def case(n, d, dtype, size, seed=0, h=2, g=2):
    gen = torch.Generator().manual_seed(seed)
    pages = -(-n // 16)
    kv = torch.randn((1, pages, h, 16, 2, d), generator=gen)
    kv[..., 1, :] *= size
    q = torch.randn((1, h * g, d), generator=gen).to(dtype)
    table = torch.randperm(pages, generator=gen).to(torch.int32)[None]
    return q, P.pack(kv.to(dtype))[0], table, [n]


@pytest.mark.parametrize("size", [1e-3, 1.0, 100.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,d", [(40, 128), (400, 128), (400, 64), (4000, 128)])
def test_lost_values_are_refused(n, d, dtype, size):
    q, pool, table, lengths = case(n, d, dtype, size)
    o, lse, to, tl, more = K.attend(q, pool, table, lengths)
    assert not ((o.to(dtype).double() - o).abs() > to).any()  # the rounded result passes
    # an all-zero output, the floors alone, and an output without one warp's blocks of V fail nearly everywhere
    f, z, _ = K.parts(pool)
    f, z = (R.gather(x, table[0], n)[:, :, 1] for x in (f, z))
    k = R.gather(P.unpack(pool[None])[0][0], table[0], n)[:, :, 0]
    p = torch.softmax(torch.einsum("hgd,hnd->hgn", q[0].double().view(2, 2, d), k) * d ** -0.5, -1)
    there = (torch.arange(n) // 16 % 4 != 1).double()
    part = torch.einsum("hgn,hnd->hgd", p * there, f + z).reshape(o[0].shape)[None]
    for lost, share in ((torch.zeros_like(o), 0.9), (more["floors"], 0.99), (part, 0.7 if n > 64 else 0.9)):
        assert float(((lost - o).abs() > to).double().mean()) > share
    # one block of 16 is seen in most outputs of up to 400 tokens, and by the root mean square in longer ones too
    there = (torch.arange(n) // 16 != 2).double()
    part = torch.einsum("hgn,hnd->hgd", p * there, f + z).reshape(o[0].shape)[None]
    assert K.rms(part - o) > 10 * K.rms_bound(o, more["size"], n, dtype)
    if n <= 400:
        assert float(((part - o).abs() > to).double().mean()) > 0.5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_products_that_vanish_are_refused(dtype):
    # a token of 2^20 times the others' weight whose values are 0: the others' codes may not get lost behind it
    n, d = 8192, 128
    q, pool, table, lengths = case(n, d, dtype, 1.0, h=1, g=1)
    gen = torch.Generator().manual_seed(1)
    kv = torch.zeros((1, n // 16, 1, 16, 2, d))
    kv[..., 1, :] = 1e-2 * (1 + 0.3 * torch.randn(kv.shape[:-2] + (d,), generator=gen))
    kv[0, int(table[0, 0]), 0, 0, 0, :32] = 20 * 0.6931 / 32
    kv[0, int(table[0, 0]), 0, 0, 1] = 0
    q = torch.zeros_like(q)
    q[..., :32] = 1
    pool = P.pack(kv.to(dtype))[0]
    o, lse, to, tl, more = K.attend(q, pool, table, lengths, scale=1.0)
    assert float(((more["floors"] - o).abs() > to).double().mean()) > 0.99
    assert not ((o.to(dtype).double() - o).abs() > to).any()
