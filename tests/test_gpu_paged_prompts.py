"""Prompts that attend their own pages in many row tiles: where each tile's work begins on the line of work."""
import pytest

from tests.test_gpu_paged import BF, HF, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths,qs,g,d,dtype", [
    ([1500], [1500], 1, 64, BF),                         # 256 queries a tile: two steps more each
    ([900, 700, 1], [900, 650, 1], 2, 128, HF),          # 128: one step
    ([700, 0, 333], [700, 3, 400], 8, 64, BF),           # 32: a step every fourth tile; more queries than tokens
    ([40, 600], [40, 20], 4, 128, BF),                   # tiles of 128 rows
    ([130, 70, 200, 5], [6, 5, 8, 4], 4, 128, HF),       # of 32 rows
    ([513, 64, 90] * 3, [9, 8, 1] * 3, 2, 64, BF),
    ([300] * 30, [2] * 30, 4, 64, HF)])
def test_prompts(lengths, qs, g, d, dtype):
    Case(lengths, qs=qs, h=2, g=g, d=d, pt=32, dtype=dtype).check()
    Case(lengths, qs=qs, prefixes=[200], h=1, g=g, d=d, pt=32, dtype=dtype).with_prior().check()


def test_thousands_of_sequences():
    # the place of a query among them: 33, 1025 and 4097 starts
    for seqs in (32, 1024, 4096):
        Case([(3 * i) % 20 for i in range(seqs)], qs=[(i % 3 == 0) + (i % 7 == 0) for i in range(seqs)], h=1, g=1, d=64).check()
