"""Every way that the dense 16-bit layers tile a product, bit for bit on whole numbers: outputs of 16 and 32
bits, with all that follows the sums, rows of any alignment, and the same bits again from a second call."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense16_util import (BF16, DEV, F16, F32, NONE, RELU, SILU, act64, act_bound, canvas, check, generator, operand, pitched,  # noqa: E402
                          untouched, whole, widened)
from dense16_shapes import BACKWARD, DENSE, GATED, SMS  # noqa: E402
from dense_util import check_quantized  # noqa: E402
from test_gpu_gated import check_gradients, checkpoint, groups, layer  # noqa: E402


def _sms():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sms != SMS:
        pytest.skip(f"the shapes are for {SMS} SMs")


@pytest.mark.parametrize("plan,T,R,K,turned", DENSE)
def test_dense(plan, T, R, K, turned):
    _sms()
    assert vnm.vnm_testing_dense_plan(0, T, R, K, SMS, *turned) == plan
    g = generator(T, R, K)
    x, w = operand(whole(g, T, K, BF16, 2), turned[0]), operand(whole(g, R, K, BF16, 2), turned[1])
    z = x.double() @ w.double().t()
    b = whole(g, 1, R, F32)[0].contiguous()
    for out, act, pad, offset, with_res in ((BF16, NONE, -R % 8, 0, False), (BF16, RELU, -R % 8, 0, True), (F32, NONE, -R % 8, 0, True),
                                            (BF16, NONE, 1, 1, True), (F32, RELU, 1, 1, False)):
        res = canvas(T, R, out, pad, offset)[0] if with_res else None
        if with_res:
            res.copy_(whole(g, T, R, out, 9))
        want = act64(z + b.double(), act) + (res.double() if with_res else 0)
        Y, buf = canvas(T, R, out, pad, offset)
        for _ in range(2):
            Y.fill_(float("nan"))
            vnm.vnm_dense_linear(x, w, Y, bias=b, act=act, residual=res)
            assert torch.equal(Y, want.float().to(out)), (out, act, pad, (Y.double() - want).abs().max().item())
        assert untouched(Y, buf)
        if with_res:  # added to in place
            vnm.vnm_dense_linear(x, w, res, bias=b, act=act, residual=res)
            assert torch.equal(res, want.float().to(out)), (out, act, pad)
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK


@pytest.mark.parametrize("plan,T,F,K,keep", GATED)
def test_gated(plan, T, F, K, keep):
    _sms()
    assert vnm.vnm_testing_dense_plan(3, T, F, K, SMS, keep=keep) == plan
    g = generator(T, F, K)
    x, wg, wu = layer(g, T, F, K, BF16)
    G, U = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    bound = act_bound(G, SILU) * U.abs() + 2.0 ** -23 * (act64(G, SILU) * U).abs()
    for pad, offset in ((-F % 16, 0), (1, 1)):
        Y, buf = canvas(T, F, BF16, pad, offset)
        kept = {}
        if keep == 1:
            kept = {k: canvas(T, F, BF16, pad, offset)[0] for k in "gu"}
        elif keep == 2:
            raw = {k: torch.full((T * (F + pad) + offset,), 0x55, dtype=torch.uint8, device=DEV) for k in "gu"}
            kept = {k: raw[k][offset:].view(T, F + pad)[:, :F].view(torch.float8_e4m3fn) for k in "gu"}
            kept.update({k + "_scale": torch.full((T, groups(F)), float("nan"), device=DEV) for k in "gu"})
        vnm.vnm_gated_linear(x, wg, wu, Y, act=SILU, **kept)
        check(Y, act64(G, SILU) * U, bound, f"{plan} pad {pad}")
        assert untouched(Y, buf)
        if keep == 1:
            assert torch.equal(kept["g"], G.bfloat16()) and torch.equal(kept["u"], U.bfloat16())
        elif keep == 2:
            check_quantized(kept["g"], kept["g_scale"], G, 1, 0.0)
            check_quantized(kept["u"], kept["u_scale"], U, 1, 0.0)
            for k in "gu":
                assert pad == 0 or (raw[k][offset:].view(T, F + pad)[:, F:] == 0x55).all()
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK


@pytest.mark.parametrize("dx,dw,T,F,K", BACKWARD)
@pytest.mark.parametrize("keep", [None, torch.float8_e4m3fn])
def test_backward(dx, dw, T, F, K, keep):
    _sms()
    assert vnm.vnm_testing_dense_plan(1, T, K, F, SMS, w_transposed=True) == dx
    assert vnm.vnm_testing_dense_plan(2, F, K, T, SMS, True, True) == dw
    g = generator(T, F, K)
    x, wg, wu = (pitched(torch.randn(*s, generator=g, device=DEV).bfloat16()) for s in ((T, K), (F, K), (F, K)))
    dy = pitched(torch.randn(T, F, generator=g, device=DEV).bfloat16())
    (a, sa), (b, sb) = checkpoint(g, T, F, keep, BF16)
    out = [canvas(*s, BF16, pad)[0] for s, pad in (((T, K), -K % 8), ((F, K), -K % 8), ((F, K), -K % 8), ((T, F), -F % 8))]
    vnm.vnm_gated_linear_backward(dy, x, wg, wu, a, b, sa, sb, act=SILU, dx=out[0], dwg=out[1], dwu=out[2], h=out[3])
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK
    check_gradients(dy, x, wg, wu, widened(a, sa), widened(b, sb), SILU, *out, BF16)
    again = [torch.empty_like(v) for v in out]
    vnm.vnm_gated_linear_backward(dy, x, wg, wu, a, b, sa, sb, act=SILU, dx=again[0], dwg=again[1], dwu=again[2], h=again[3])
    assert all(torch.equal(p, q) for p, q in zip(out, again))
