"""New outputs of PagedKV's calls are what torch.empty would make where a program has changed what that does."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from tests.test_gpu_paged import BF
from verified_kv_cache_poissoncomp_gb300.paged import PagedKV

pytestmark = pytest.mark.gpu


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.made = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if "empty" in str(func):
            self.made.append(tuple(out.shape))
        return out


def calls(c):
    q = torch.zeros((3, 4, 64), dtype=BF, device="cuda")
    table, n = torch.zeros((3, 1), dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    yield c.norm_rotate(q, None)[0]
    yield from c.attend(0, q, table, n, 16)
    lse = torch.zeros((3, 4), device="cuda")
    w = c.weigh(0, q, lse, table, n, 16)
    yield w
    yield c.evict(0, table, n, 16, w, 5, 1, 1)[1]


def test_a_dispatch_mode_sees_them():
    c = PagedKV(2, 2, 64, num_pages=4)
    list(calls(c))  # (the workspace)
    with Seen() as seen:
        got = [tuple(x.shape) for x in calls(c)]
    c.sync()
    assert got == [(3, 4, 64), (3, 4, 64), (3, 4), (3, 2, 16), (3, 2, 5)]
    assert seen.made == got


@pytest.mark.parametrize("fill", [True, False])
def test_deterministic_algorithms_fill_them(fill):
    c = PagedKV(2, 2, 64, num_pages=4)
    was = torch.utils.deterministic.fill_uninitialized_memory
    torch.use_deterministic_algorithms(True)
    torch.utils.deterministic.fill_uninitialized_memory = fill
    try:
        for dtype in (BF, torch.float32):
            a = [c._empty((5, 7, 11), dtype) for _ in range(4)]
            if fill:
                assert all(bool(torch.isnan(x).all()) for x in a)
    finally:
        torch.use_deterministic_algorithms(False)
        torch.utils.deterministic.fill_uninitialized_memory = was


def test_in_inference_mode():
    c = PagedKV(2, 2, 64, num_pages=4)
    with torch.inference_mode():
        for shape in ((3, 4), (3, 4, 64), (2, 0, 5)):
            assert c._empty(shape, BF).is_inference() and torch.empty(shape, device="cuda").is_inference()
    for x in calls(c):
        assert not x.is_inference() and not x.requires_grad
    with torch.inference_mode():
        for x in calls(c):
            assert x.is_inference()
    c.sync()
