"""Numbers that do not fit the C ABI's 32 bits are refused, not cut down to ones that do."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense_util import DEV  # noqa: E402

E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("act", [1 << 32, (1 << 32) + 2, -(1 << 32)])
def test_activation(act):
    q, s, Y = torch.zeros((2, 128), dtype=torch.uint8, device=DEV).view(E4M3), torch.ones((2, 1), device=DEV), torch.empty((2, 2), device=DEV)
    with pytest.raises(vnm.VnmError) as e:
        vnm.vnm_fp8_linear(q, s, q, s, Y, act=act)
    assert e.value.code == vnm.VNM_ERR_INVALID_ARG


@pytest.mark.parametrize("rows", [(1 << 32) + 1, (1 << 32) + 128])
def test_block_rows(rows):
    x = torch.ones((1, 128), device=DEV)
    q, s = torch.empty((1, 128), dtype=E4M3, device=DEV), torch.empty((1, 1), device=DEV)
    with pytest.raises(vnm.VnmError) as e:
        vnm.vnm_fp8_quantize(x, q, s, block_rows=rows)
    assert e.value.code == vnm.VNM_ERR_INVALID_ARG
