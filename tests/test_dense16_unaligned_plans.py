"""The plans of products whose outputs' rows do not start on 16 bytes, without a GPU: the listed shapes take them, and
they hold every tiling of pairs of CTAs."""
import pytest

from structured_sparse_matmul_gb300 import vnm
from test_abi import libvnm  # noqa: F401  (fixture)
from dense16_unaligned_shapes import BACKWARD, DENSE, GATED, SMS

plan = vnm.vnm_testing_dense_plan


def test_the_listed_plans(libvnm):  # noqa: F811
    for want, T, R, K, (xt, wt) in DENSE:
        assert plan(0, T, R, K, SMS, xt, wt, aligned=False) == want, (T, R, K)
    for want, T, F, K, keep in GATED:
        assert plan(3, T, F, K, SMS, keep=keep, aligned=False) == want, (T, F, K)
    for dx, dw, T, F, K in BACKWARD:
        assert (plan(1, T, K, F, SMS, w_transposed=True, aligned=False), plan(2, F, K, T, SMS, True, True, aligned=False)) == (dx, dw), (T, F, K)


def test_every_tiling_of_pairs_is_listed():
    widths, splits = {(0, n, 1) for n in (128, 160, 192, 224, 256)}, {(0, 256, s) for s in (2, 3, 4)}
    assert widths | splits == {p for p, *_ in DENSE}
    assert widths <= {p for p, _, _, K, _ in DENSE if K <= 1024}
    assert {(0, n, 1) for n in (128, 192, 256)} <= {p for p, *_, keep in GATED if keep == 0} & {p for p, *_, keep in GATED if keep == 1}
    assert {(0, 256, s) for s in (1, 2, 4)} <= {p for p, *_, keep in GATED if keep == 2}


def test_plan_refusals(libvnm):  # noqa: F811
    for aligned in (2, -1):
        with pytest.raises(vnm.VnmError):
            plan(0, 1, 1, 1, SMS, aligned=aligned)
