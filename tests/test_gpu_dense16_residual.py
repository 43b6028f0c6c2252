"""The residual is added once, to the whole sum: a residual far larger than the parts that a sum over a long K is put
together from does not take them in one by one, each rounded to its own spacing."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense16_util import BF16, DEV, F16, F32, NONE, RELU, canvas, generator, operand, pitched, untouched, whole  # noqa: E402

BIG = 2.0 ** 24  # fp32's spacing is 2 from here on


def spread(rows, K, dtype):
    """A row's only elements are ones, 1024 apart."""
    v = torch.zeros((rows, K), dtype=dtype, device=DEV)
    v[:, 5::1024] = 1
    return v


# (few tokens; narrow tiles; pairs of CTAs of one round and of several; K over pairs)
@pytest.mark.parametrize("T,R,K", [(4, 300, 4096), (40, 130, 4096), (2304, 2048, 4096), (4096, 1024, 8192), (3000, 4100, 4096), (1432, 1031, 4096)])
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("pad,offset", [(None, 0), (1, 1)])
def test_a_large_residual(T, R, K, turned, pad, offset):
    """2^24 plus K / 1024 ones is exact in fp32; one more at a time it stays 2^24."""
    x, w = operand(spread(T, K, BF16), turned), operand(spread(R, K, F32).to(BF16), turned)
    Y, buf = canvas(T, R, F32, -R % 8 if pad is None else pad, offset)
    two = torch.full((R,), 2.0, device=DEV)
    for act, bias in ((NONE, None), (NONE, two), (RELU, None)):
        Y.fill_(BIG)
        vnm.vnm_dense_linear(x, w, Y, bias=bias, act=act, residual=Y)
        assert (Y == BIG + K // 1024 + (0 if bias is None else 2)).all(), (act, bias is not None, Y.unique())
    assert untouched(Y, buf)
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK


@pytest.mark.parametrize("T,F,K", [(4096, 640, 640), (4096, 2048, 2048), (4096, 4096, 1024)])
def test_gradients_added_to_large_ones(T, F, K):
    dy = spread(F, T, F16).t().contiguous()
    one = torch.ones((T, F), dtype=F16, device=DEV)
    x, w = torch.ones((T, K), dtype=F16, device=DEV), torch.zeros((F, K), dtype=F16, device=DEV)
    dwg, dwu = (torch.full((F, K), BIG, device=DEV) for _ in range(2))
    vnm.vnm_gated_linear_backward(dy, x, w, w, one, one, act=NONE, dwg=dwg, dwu=dwu, accumulate=True)
    assert (dwg == BIG + T // 1024).all() and (dwu == BIG + T // 1024).all()


@pytest.mark.parametrize("T,R,K", [(2304, 2048, 3000), (4096, 1024, 2500), (3000, 4100, 2048), (5000, 1048, 4200)])
def test_the_same_bits_as_added_afterwards(T, R, K):
    """The sums without a residual plus the residual, rounded once; in place too."""
    g = generator(T, R, K, 51)
    x, w = (pitched(torch.randn(*s, generator=g, device=DEV).to(BF16)) for s in ((T, K), (R, K)))
    res, plain, Y = whole(g, T, R, F32, 3, 100.0), torch.empty((T, R), device=DEV), torch.empty((T, R), device=DEV)
    vnm.vnm_dense_linear(x, w, plain)
    vnm.vnm_dense_linear(x, w, Y, residual=res)
    assert torch.equal(Y, plain + res)
    vnm.vnm_dense_linear(x, w, res, residual=res)
    assert torch.equal(Y, res)
