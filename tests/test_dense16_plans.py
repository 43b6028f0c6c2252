"""How the dense 16-bit layers tile a product, without a GPU: every way is taken by a shape that the GPU
tests run, and no plan asks for what its kernel does not have."""
import random

import pytest

from structured_sparse_matmul_gb300 import vnm
from test_abi import libvnm  # noqa: F401  (fixture)
from dense16_shapes import BACKWARD, DENSE, GATED, SMS

plan = vnm.vnm_testing_dense_plan


def test_the_listed_plans(libvnm):  # noqa: F811
    for want, T, R, K, (xt, wt) in DENSE:
        assert plan(0, T, R, K, SMS, xt, wt) == want, (T, R, K)
    for want, T, F, K, keep in GATED:
        assert plan(3, T, F, K, SMS, keep=keep) == want, (T, F, K)
    for dx, dw, T, F, K in BACKWARD:
        assert (plan(1, T, K, F, SMS, w_transposed=True), plan(2, F, K, T, SMS, True, True)) == (dx, dw), (T, F, K)


def test_every_kernel_is_listed():
    few, widths = (8, 0, 1), (16, 32, 64, 128)
    dense, both = {p for p, *_, t in DENSE if not t[0]}, {p for p, *_, t in DENSE if t[0]}
    for found, wide in ((dense, widths), (both, (64, 128))):
        assert {p[0] for p in found if p[0] > 8} == set(wide)
        assert {(0, n, 1) for n in (128, 160, 192, 224, 256)} | {(0, 256, s) for s in (2, 3, 4)} <= found
    assert few in dense
    keeps = {k: {p for p, *_, keep in GATED if keep == k} for k in (0, 1, 2)}
    assert {p[0] for p in keeps[0] | keeps[1]} == {p[0] for p in keeps[2]} | {8} == set(widths) | {0, 8}
    assert {(0, 256, s) for s in (1, 2, 3, 4)} <= keeps[2]
    assert {(0, n, 1) for n in (128, 192, 256)} | {(0, 256, s) for s in (2, 3, 4)} <= keeps[0] | keeps[1]


@pytest.mark.parametrize("sms", [1, 76, 132, 152, 160])
def test_plans_are_ones_that_the_kernels_have(libvnm, sms):  # noqa: F811
    rng = random.Random(sms)
    for _ in range(4000):
        kind = rng.choice([0, 1, 2, 3])
        T, R, K = (int(2 ** rng.uniform(0, 14)) for _ in range(3))
        xt, wt = {0: (rng.random() < 0.5, rng.random() < 0.5), 1: (False, True), 2: (True, True), 3: (False, False)}[kind]
        keep = rng.choice([0, 1, 2, 3]) if kind == 3 else 0
        tile, rows, splits = plan(kind, T, R, K, sms, xt, wt, keep)
        blocks = -(-K // 64) * (2 if kind == 1 else 1)
        assert 1 <= splits <= blocks
        if tile == 8:
            assert T <= 16 and kind in (0, 3) and keep < 2 and not (xt or wt)
        elif tile == 0:
            assert rows in ((128, 192, 256) if kind == 3 else (128, 160, 192, 224, 256)) and splits <= 4 and (splits == 1 or rows == 256) and (keep < 2 or rows == 256)
        else:
            assert tile in ((64, 128) if xt else (16, 32, 64, 128)) and splits <= (4 if keep >= 2 else 8)


def test_plan_refusals(libvnm):  # noqa: F811
    for bad in ((4, 1, 1, 1, 152), (-1, 1, 1, 1, 152), (0, 0, 1, 1, 152), (0, 1, 1, -1, 152), (0, 1, 1, 1, 0)):
        with pytest.raises(vnm.VnmError):
            plan(*bad)
    with pytest.raises(vnm.VnmError):
        plan(3, 1, 1, 1, 152, keep=4)
