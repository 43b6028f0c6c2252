"""vnm_fp8_linear leaves what lies behind Y's columns as it was, where Y's rows start on 16 bytes and do not
end on 16 (a tensor memory store would write the rest of the last 16)."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense_util import DEV, check_linear, linear64, quantize  # noqa: E402


@pytest.mark.parametrize("R", [2001, 2002, 2004, 2007, 2008])
@pytest.mark.parametrize("y_type", [torch.bfloat16, torch.float32])
def test_row_ends(R, y_type):
    T, K = 2500, 256
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert vnm.vnm_testing_fp8_linear_plan(T, R, K, 128, sms)[0] == 0  # pairs of CTAs
    g = torch.Generator(device=DEV).manual_seed(R)
    xq, xs = quantize(torch.randn(T, K, generator=g, device=DEV), 1, torch.float8_e4m3fn)
    wq, ws = quantize(torch.randn(R, K, generator=g, device=DEV), 128, torch.float8_e4m3fn)
    buf = torch.full((T, 2016), 7.0, dtype=y_type, device=DEV)
    vnm.vnm_fp8_linear(xq, xs, wq, ws, buf[:, :R])
    check_linear(buf[:, :R], linear64(xq, xs, wq, ws, None, 0), K, 0)
    assert (buf[:, R:] == 7.0).all()
