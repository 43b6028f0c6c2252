"""vnm_fp8_linear where Y's rows start on 16 bytes and end anywhere: the boxes inside Y go by tensor memory stores, the
last columns by the warps, from two boxes in turn over several tiles. The bits of rows that start anywhere, which
the warps copy all."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense_util import DEV, check_linear, linear64, quantize  # noqa: E402


@pytest.mark.parametrize("T,R,K", [(2500, 2001, 256), (4111, 4097, 384), (9000, 1030, 128), (8192, 2815, 128), (300, 30001, 256), (2500, 2500, 1024)])
@pytest.mark.parametrize("y_type", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act,bias,rows", [(vnm.VNM_ACT_NONE, False, 128), (vnm.VNM_ACT_RELU, True, 1), (vnm.VNM_ACT_GELU, True, 128)])
def test_row_ends(T, R, K, y_type, act, bias, rows):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert vnm.vnm_testing_fp8_linear_plan(T, R, K, rows, sms)[0] == 0  # pairs of CTAs
    g = torch.Generator(device=DEV).manual_seed(R)
    xq, xs = quantize(torch.randn(T, K, generator=g, device=DEV), 1, torch.float8_e4m3fn)
    wq, ws = quantize(torch.randn(R, K, generator=g, device=DEV), rows, torch.float8_e4m3fn)
    b = torch.randn(R, generator=g, device=DEV).to(y_type) if bias else None
    wide = -(-R // 8) * 8 + 8
    starts, odd = (torch.full((T, n), 7.0, dtype=y_type, device=DEV) for n in (wide, wide + 1))
    vnm.vnm_fp8_linear(xq, xs, wq, ws, odd[:, :R], bias=b, act=act)
    for _ in range(2):
        starts[:, :R] = float("nan")
        vnm.vnm_fp8_linear(xq, xs, wq, ws, starts[:, :R], bias=b, act=act)
        assert torch.equal(starts[:, :R], odd[:, :R])
    assert (starts[:, R:] == 7.0).all() and (odd[:, R:] == 7.0).all()
    check_linear(starts[:, :R], linear64(xq, xs, wq, ws, b, act), K, act)
    assert vnm.vnm_fp8_linear_get_status() == vnm.VNM_OK
