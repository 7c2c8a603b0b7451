"""The kernels' wait limits begin when the kernels ahead of the call on its stream are done: a kernel that
lets its successor start early and then takes long is nobody's failure."""
import ctypes
import subprocess

import pytest
import torch

from tests.test_gpu_paged import BF, HF, Case
from verified_kv_cache_poissoncomp_gb300 import binding as B
from verified_kv_cache_poissoncomp_gb300 import build as build_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def long_kernel(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("long") / "liblong.so")
    subprocess.run([build_mod.nvcc(), *build_mod.ARCH, "-O2", "-shared", "-Xcompiler", "-fPIC", "-o", lib,
                    f"{build_mod.ROOT}/tests/long_kernel.cu"], check=True)
    f = ctypes.CDLL(lib).long_kernel
    f.argtypes = [ctypes.c_int, ctypes.c_void_p]
    return f


@pytest.mark.parametrize("lengths,qs,prefix,d,dtype", [
    ([40], 1, 0, 128, BF), ([6000] * 4, 1, 0, 64, HF), ([300, 700], 6, 0, 128, BF), ([60], 20, 900, 128, HF),
    ([60], 100, 900, 64, BF), ([400] * 40, 1, 9000, 128, BF)])
def test_a_long_kernel_ahead(long_kernel, lengths, qs, prefix, d, dtype):
    c = Case(lengths, qs=[qs] * len(lengths), prefixes=[prefix] if prefix else (), h=2, g=4, d=d, pt=64, dtype=dtype)
    good = c.run()
    c.cache.sync()
    for _ in range(3):
        B.verkv_test_inject(c.cache.ctx, B.VERKV_INJECT_PAGED_LIMIT, 2_000_000)
        assert long_kernel(20_000, c.cache.stream.cuda_stream) == 0
        o, lse = c.run()
        assert B.verkv_sync_status(c.cache.ctx) == B.VERKV_OK
        assert torch.equal(o, good[0]) and torch.equal(lse, good[1])


def test_the_limit_is_checked():
    c = Case([40], h=1, g=1, d=64)
    for value in (0, 999, 1_000_000_001):
        with pytest.raises(B.VerkvError) as e:
            B.verkv_test_inject(c.cache.ctx, B.VERKV_INJECT_PAGED_LIMIT, value)
        assert e.value.status == B.VERKV_EINVAL
