"""Every tiling of vnm_fp8_linear against 64 bits: each width of a tile, each split of K, one tile a
CTA and several, and each pair of 8-bit formats in each kernel."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense_util import DEV, check_linear, linear64, quantize  # noqa: E402
from fp8_shapes import ONE_BLOCK, SHAPES, several_tiles  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def _run(plan, T, R, K, rows, y_type=F32, bias_type=None, act=0, fx=E4M3, fw=E4M3):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert vnm.vnm_testing_fp8_linear_plan(T, R, K, rows, sms) == plan
    g = torch.Generator(device=DEV).manual_seed(T + R + K)
    xq, xs = quantize(torch.randn(T, K, generator=g, device=DEV), 1, fx)
    wq, ws = quantize(0.05 * torch.randn(R, K, generator=g, device=DEV), rows, fw)
    bias = torch.randn(R, generator=g, device=DEV).to(bias_type) if bias_type is not None else None
    Y = [torch.full((T, R), float("nan"), dtype=y_type, device=DEV) for _ in range(2)]
    for y in Y:
        vnm.vnm_fp8_linear(xq, xs, wq, ws, y, bias=bias, act=act)
    assert vnm.vnm_fp8_linear_get_status() == vnm.VNM_OK
    assert torch.equal(Y[0], Y[1])
    check_linear(Y[0], linear64(xq, xs, wq, ws, bias, act), K, act, f"{plan} {T}x{R}x{K}")
    return sms


@pytest.mark.parametrize("plan,T,R,K,several,rows", [(*s, rows) for s in SHAPES for rows in (1, 128)]
                         + [(*s, 1) for s in ONE_BLOCK])
def test_sums(plan, T, R, K, several, rows):
    sms = _run(plan, T, R, K, rows)
    assert several_tiles(plan, T, R, sms) == several


@pytest.mark.parametrize("plan,T,R,K,several", [s for s in SHAPES if s[3] <= 1100])
@pytest.mark.parametrize("y_type,bias_type,act", [(BF16, F32, 2), (F16, F16, 1)])
def test_bias_activation_and_rounding(plan, T, R, K, several, y_type, bias_type, act):
    _run(plan, T, R, K, 128, y_type, bias_type, act)


@pytest.mark.parametrize("plan,T,R,K", [((8, 1), 1, 300, 640), ((8, 1), 8, 300, 700), ((16, 4), 9, 3001, 1000),
                                        ((128, 2), 777, 1000, 1041), ((0, 1), 600, 2050, 300)])
@pytest.mark.parametrize("fx,fw", [(E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2), (E5M2, E5M2)])
def test_formats(plan, T, R, K, fx, fw):
    _run(plan, T, R, K, 128, fx=fx, fw=fw)
