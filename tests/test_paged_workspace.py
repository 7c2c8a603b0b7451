"""What verkv_paged_attend's workspace takes, without a GPU: what calls over 16-bit pages need, whose size is asked for without
saying what the pages hold; 4-bit pages make do with it."""
import pytest

from verified_kv_cache_poissoncomp_gb300 import binding as B

CALLS = [(1, 0, 1), (1, 1, 1), (2, 1, 2), (3, 1, 3), (4, 1, 4), (1, 1, 4), (5, 2, 5), (8, 1, 8), (34, 2, 102), (256, 1, 256),
         (32, 0, 32), (1, 1, 8192), (1, 0, 8192)]
SIZES = {(8, 4, 128): [5210112, 5359872, 5659392, 5958912, 6258432, 6258432, 16675072, 17041152, 44397824, 68962048, 14911744, 300054272, 157615872],
         (2, 8, 64): [2608000, 2646016, 2722048, 7900672, 7942912, 7875328, 8052736, 8111872, 16273152, 23795456, 11491584, 82319104, 45012736],
         (1, 1, 64): [2578696, 2587408, 2596384, 2605360, 2614336, 2588992, 2631760, 2658688, 8115552, 15212288, 5417472, 17303296, 12504832]}


@pytest.mark.parametrize("shape", list(SIZES))
def test_sizes(shape):
    from verified_kv_cache_poissoncomp_gb300 import build
    build.build()
    sh = B.verkv_shape(1, 1, *shape, 1, 1)
    assert [B.verkv_paged_workspace_size(sh, *call) for call in CALLS] == SIZES[shape]
