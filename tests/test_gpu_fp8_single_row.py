"""A single row of 8-bit values has no pitch: it is served whatever its length or its tensor's
strides, as long as it starts on 16 bytes."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense_util import DEV, check_linear, linear64, quantize  # noqa: E402

E4M3 = torch.float8_e4m3fn


def _operand(n, K, rows, seed, single):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q, s = quantize(torch.randn(n, K, generator=g, device=DEV), rows, E4M3)
    if n == 1 and single == "contiguous":
        q = q.contiguous()
    elif n == 1 and single == "strided":  # the first row of a matrix whose rows are 7 bytes longer
        buf = torch.full((3, K + 7), 0x7F, dtype=torch.uint8, device=DEV)
        buf[0, :K] = q.view(torch.uint8)[0]
        q = buf.view(E4M3)[:1, :K]
        assert q.stride() == (K + 7, 1)
    return q, s


# one token (few-token kernel), one output of a few tokens and of many (tiles), both
@pytest.mark.parametrize("T,R", [(1, 300), (5, 1), (200, 1), (1, 1)])
@pytest.mark.parametrize("K", [1, 15, 130, 1000, 1041])
@pytest.mark.parametrize("single", ["contiguous", "strided"])
def test_single_row(T, R, K, single):
    xq, xs = _operand(T, K, 1, K, single)
    wq, ws = _operand(R, K, 128, K + 1, single)
    Y = torch.full((T, R), float("nan"), device=DEV)
    vnm.vnm_fp8_linear(xq, xs, wq, ws, Y)
    check_linear(Y, linear64(xq.contiguous(), xs, wq.contiguous(), ws, None, 0), K, 0)
