"""fp32 outputs take the tensor cores' truncated sums out every 1024 elements of K: held to less than the same sums lose
without that.

The tensor cores lose about K * 2^-30 of random sums' norm: at K = 8192 7.6e-6 (9e-6 was measured), in chunks of 1024 an eighth
of it, up to 1.13e-6. The chunks' sums are added in fp32, eight roundings of up to 2^-24 each, in quadrature 2e-7, and those of
a split or a warp as many again: 1.2e-6 in all. Chunks of 2048 would lose 2.25e-6. 1.7e-6 lies between."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense16_util import BF16, DEV, F16, F32, NONE, generator, operand  # noqa: E402

K = 8192
FAR = 1.7e-6


def far(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


# (few tokens; narrow tiles of each width, with and without splits of K; pairs of CTAs; K over pairs)
@pytest.mark.parametrize("T,R", [(1, 256), (8, 1000), (16, 256), (33, 4096), (200, 300), (500, 2100), (700, 700), (1000, 4096), (2000, 2000), (4096, 1024), (3000, 4104)])
@pytest.mark.parametrize("turned", [(False, False), (False, True), (True, True)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_products(T, R, turned, dtype):
    g = generator(T, R, 71)
    x, w = (torch.randn(n, K, generator=g, device=DEV).to(dtype) for n in (T, R))
    Y = torch.empty((T, R), dtype=F32, device=DEV)
    vnm.vnm_dense_linear(operand(x, turned[0]), operand(w, turned[1]), Y)
    assert far(Y, x.double() @ w.double().t()) <= FAR
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK


@pytest.mark.parametrize("F,D", [(1024, 256), (2048, 1024), (4096, 1024)])
def test_weights_gradients(F, D):
    """(of operands that dG and dU hold exactly)"""
    g = generator(F, D, 72)
    x, dy = (torch.randn(K, n, generator=g, device=DEV).bfloat16() for n in (D, F))
    one, w = torch.ones((K, F), dtype=BF16, device=DEV), torch.zeros((F, D), dtype=BF16, device=DEV)
    dwg, dwu = (torch.empty((F, D), device=DEV) for _ in range(2))
    vnm.vnm_gated_linear_backward(dy, x, w, w, one, one, act=NONE, dwg=dwg, dwu=dwu)
    want = dy.double().t() @ x.double()
    assert far(dwg, want) <= FAR and far(dwu, want) <= FAR
