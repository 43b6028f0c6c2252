"""A time-out of a vnm_fp8_linear call that was given no status words is kept for
vnm_fp8_linear_get_status: pipeline stages whose loads are never issued make the
bounded waits run out."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense_util import DEV, check_linear, linear64, quantize  # noqa: E402

E4M3 = torch.float8_e4m3fn


# split K, and the persistent pairs' second tile
@pytest.mark.parametrize("T,R,K,skip", [(16, 512, 4096, 2), (2500, 2000, 1024, 9)])
def test_time_out_without_status_words(T, R, K, skip):
    g = torch.Generator(device=DEV).manual_seed(T)
    xq, xs = quantize(torch.randn(T, K, generator=g, device=DEV), 1, E4M3)
    wq, ws = quantize(torch.randn(R, K, generator=g, device=DEV), 128, E4M3)
    Y, own = torch.empty((T, R), device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    assert vnm.vnm_fp8_linear_get_status() == vnm.VNM_OK
    vnm.vnm_testing_fp8_linear_skip_stage(xq, xs, wq, ws, Y, skip, status=None)
    assert vnm.vnm_fp8_linear_get_status() == vnm.VNM_ERR_TIMEOUT
    assert vnm.vnm_fp8_linear_get_status() == vnm.VNM_OK  # cleared
    vnm.vnm_testing_fp8_linear_skip_stage(xq, xs, wq, ws, Y, skip, status=own)
    assert vnm.vnm_fp8_linear_get_status() == vnm.VNM_OK and own[0].item() == vnm.VNM_ERR_TIMEOUT
    vnm.vnm_fp8_linear(xq, xs, wq, ws, Y)
    assert vnm.vnm_fp8_linear_get_status() == vnm.VNM_OK
    check_linear(Y, linear64(xq, xs, wq, ws, None, 0), K, 0)
