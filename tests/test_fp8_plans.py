"""The rule that tiles vnm_fp8_linear, without a GPU: the sizes that the GPU tests run take the
tilings that they say, and no tiling that the rule gives is without such a size."""
import math
import random

import pytest

from fp8_shapes import ONE_BLOCK, SHAPES, several_tiles
from structured_sparse_matmul_gb300 import vnm
from test_abi import libvnm  # noqa: F401  (fixture)

SMS = 152


@pytest.mark.parametrize("plan,T,R,K,several,rows", [(*s, rows) for s in SHAPES for rows in (1, 128)]
                         + [(*s, 1) for s in ONE_BLOCK])
def test_shapes_take_their_tiling(libvnm, plan, T, R, K, several, rows):  # noqa: F811
    assert vnm.vnm_testing_fp8_linear_plan(T, R, K, rows, SMS) == plan
    assert several_tiles(plan, T, R, SMS) == several


def test_every_tiling_has_a_shape(libvnm):  # noqa: F811
    rng = random.Random(5)
    have = {(plan, several) for plan, _, _, _, several in SHAPES}
    for _ in range(60000):
        T, R, K = (int(round(math.exp(rng.uniform(0, math.log(n))))) for n in (8192, 40000, 32768))
        plan = vnm.vnm_testing_fp8_linear_plan(T, R, K, rng.choice([1, 128]), SMS)
        key = (plan, several_tiles(plan, T, R, SMS))
        assert key in have, (key, T, R, K)


def test_refusals(libvnm):  # noqa: F811
    for bad in ((0, 1, 1, 1, 152), (1, 0, 1, 1, 152), (1, 1, 0, 1, 152), (1, 1, 1, 2, 152), (1, 1, 1, 1, 0)):
        with pytest.raises(vnm.VnmError) as e:
            vnm.vnm_testing_fp8_linear_plan(*bad)
        assert e.value.code == vnm.VNM_ERR_INVALID_ARG
