"""Attention over pages multiplies V with weights of two 16-bit parts wherever a unit has up to 128 rows:
the result is held to its own rounding and the errors of the logits, without a rounding of the weights."""
import pytest
import torch

from tests import paged_reference as R
from tests.test_gpu_paged import BF, HF, Case

pytestmark = pytest.mark.gpu


def check(c):
    o, lse = c.run()
    c.cache.sync()
    wo, wl, to, tl = c.want()
    # A = sum p |v| / sum p: the same weights on the values' magnitudes
    kv = c.kv.clone()
    kv[..., 1, :] = kv[..., 1, :].abs()
    A = R.attend(c.q, kv[0], c.table, c.lengths, c.q_start, c.prefix_table, c.prefix_lengths, c.group_start)[0]
    # A weight's first part is off by u of it at most, u half a step of the type, the second part by u of
    # what that left out: u^2 A stands for u A in the bound of R.attend.
    u = R.half_step(c.q.dtype)
    R.close(lse, wl, tl, "lse")
    R.close(o, wo, to - (u - u * u) * (1 + u) * A * 1.001, "o")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
def test_one_query_a_sequence(dtype, d, g):
    check(Case([2, 3, 15, 17, 64, 65, 100, 300, 5, 1, 0], h=2, g=g, d=d, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("qs", [[1, 3, 2, 0, 1], [5, 8, 1, 7, 6], [9, 4, 8, 2, 12], [30, 25, 32, 9, 16]])
def test_several_queries_a_sequence(dtype, d, qs):
    # up to 16, up to 32 and up to 128 rows a unit
    check(Case([40, 9, 130, 64, 257], qs=qs, h=2, g=4, d=d, pt=32, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seqs", [1, 2, 3, 4, 5, 9, 31, 32])
def test_prefix_of_few_rows(dtype, d, seqs):
    # 4 and 8 rows, 12 and 16, and up to 128 of the prefix, beside own tokens of 4 rows
    check(Case([(13 * i) % 70 for i in range(seqs)], prefixes=[333], h=2, g=4, d=d, pt=64, dtype=dtype))


def test_groups_of_unequal_sizes():
    check(Case([(13 * i) % 70 for i in range(20)], prefixes=[333, 64, 129], groups=[0, 1, 17, 20], h=2, g=4, d=128, pt=64))
