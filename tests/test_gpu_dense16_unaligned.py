"""Pairs of CTAs where outputs, residuals or checkpoints do not start on 16 bytes, each of them by itself and all
together, bit for bit on whole numbers; rows that start on 2, 4 or 8 bytes take the copies' ways by elements and by words."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense16_util import (BF16, DEV, F16, F32, NONE, RELU, SILU, act64, act_bound, canvas, check, generator, operand, pitched,  # noqa: E402
                          untouched, whole, widened)
from dense16_unaligned_shapes import BACKWARD, DENSE, GATED, SMS  # noqa: E402
from dense_util import check_quantized  # noqa: E402
from test_gpu_gated import check_gradients, checkpoint, groups, layer  # noqa: E402


def _sms():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sms != SMS:
        pytest.skip(f"the shapes are for {SMS} SMs")


def matrix(rows, cols, dtype, start):
    """A canvas whose rows start ``start`` bytes past 16 (rows of a multiple of 16 bytes), or, for
    "odd", anywhere."""
    if start == "odd":
        return canvas(rows, cols, dtype, 1 + cols % 2, 1)  # (rows of odd length)
    per = 16 // dtype.itemsize
    return canvas(rows, cols, dtype, -cols % per + per, start // dtype.itemsize)


@pytest.mark.parametrize("plan,T,R,K,turned", DENSE)
@pytest.mark.parametrize("out", [BF16, F32])
def test_dense(plan, T, R, K, turned, out):
    _sms()
    assert vnm.vnm_testing_dense_plan(0, T, R, K, SMS, *turned, aligned=False) == plan
    g = generator(T, R, K, 61)
    top = 2 if K < 30000 else 1
    x, w = operand(whole(g, T, K, BF16, top), turned[0]), operand(whole(g, R, K, BF16, top), turned[1])
    z, b = x.double() @ w.double().t(), whole(g, 1, R, F32)[0].contiguous()
    for start, res_start, act, bias in (("odd", None, NONE, False), ("odd", "odd", NONE, True), (4, 0, RELU, True), (8, 4, NONE, False),
                                        (0, "odd", NONE, True), (0, 8, RELU, False), (0, 4, NONE, False), (4, None, RELU, True),
                                        ("odd", 0, NONE, False)):
        Y, buf = matrix(T, R, out, start)
        res = None
        if res_start is not None:
            res = matrix(T, R, out, res_start)[0]
            res.copy_(whole(g, T, R, out, 9))
        want = act64(z + (b.double() if bias else 0), act) + (res.double() if res is not None else 0)
        for _ in range(2):
            Y.fill_(float("nan"))
            vnm.vnm_dense_linear(x, w, Y, bias=b if bias else None, act=act, residual=res)
            assert torch.equal(Y, want.float().to(out)), (start, res_start, act, bias)
        assert untouched(Y, buf), (start, res_start)
        if res is not None:
            vnm.vnm_dense_linear(x, w, res, bias=b if bias else None, act=act, residual=res)
            assert torch.equal(res, Y), (res_start, act, bias)
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK


@pytest.mark.parametrize("plan,T,F,K,keep", GATED)
def test_gated(plan, T, F, K, keep):
    _sms()
    assert vnm.vnm_testing_dense_plan(3, T, F, K, SMS, keep=keep, aligned=False) == plan
    g = generator(T, F, K, 62)
    x, wg, wu = layer(g, T, F, K, F16)
    G, U = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    bound = act_bound(G, SILU) * U.abs() + 2.0 ** -23 * (act64(G, SILU) * U).abs()
    for start, g_start, u_start in (("odd", "odd", "odd"), (4, 0, 0), (0, "odd", "odd"), (0, 0, 4), (8, 4, 8), (0, 8, 0)):
        Y, buf = matrix(T, F, F16, start)
        kept, raw = {}, {}
        for k, s in (("g", g_start), ("u", u_start)):
            if keep == 1:
                kept[k], raw[k] = matrix(T, F, F16, s)
            elif keep == 2:
                ld, first = (F + 1, 1) if s == "odd" else (-(-F // 16) * 16 + 16, s)
                raw[k] = torch.full((T * ld + first,), 0x55, dtype=torch.uint8, device=DEV)
                kept[k] = raw[k][first:].view(T, ld)[:, :F].view(torch.float8_e4m3fn)
                kept[k + "_scale"] = torch.full((T, groups(F)), float("nan"), device=DEV)
        vnm.vnm_gated_linear(x, wg, wu, Y, act=SILU, **kept)
        check(Y, act64(G, SILU) * U, bound, (start, g_start, u_start))
        assert untouched(Y, buf)
        for k, want in (("g", G), ("u", U)):
            if keep == 1:
                assert torch.equal(kept[k], want.half()) and untouched(kept[k], raw[k]), (start, g_start, u_start)
            elif keep == 2:
                check_quantized(kept[k], kept[k + "_scale"], want, 1, 0.0)
                outside = torch.ones(raw[k].numel(), dtype=torch.bool, device=DEV)
                inside = kept[k].storage_offset() + torch.arange(T, device=DEV)[:, None] * kept[k].stride(0) + torch.arange(F, device=DEV)
                outside[inside.reshape(-1)] = False
                assert (raw[k][outside] == 0x55).all(), (start, g_start, u_start)
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK


@pytest.mark.parametrize("dx,dw,T,F,K", BACKWARD)
@pytest.mark.parametrize("start", ["odd", 4, 8])
def test_backward(dx, dw, T, F, K, start):
    _sms()
    assert vnm.vnm_testing_dense_plan(1, T, K, F, SMS, w_transposed=True, aligned=False) == dx
    assert vnm.vnm_testing_dense_plan(2, F, K, T, SMS, True, True, aligned=False) == dw
    g = generator(T, F, K, 63)
    x, wg, wu = (pitched(torch.randn(*s, generator=g, device=DEV).bfloat16()) for s in ((T, K), (F, K), (F, K)))
    dy = matrix(T, F, BF16, start)[0]
    dy.copy_(torch.randn(T, F, generator=g, device=DEV))
    (a, sa), (b, sb) = checkpoint(g, T, F, None, BF16)
    for out, accumulate in ((BF16, False), (F32, True), (BF16, True)):
        o = [matrix(*s, dt, start) for s, dt in (((T, K), BF16), ((F, K), out), ((F, K), out), ((T, F), BF16))]
        if accumulate:
            o[1][0].fill_(1.5), o[2][0].fill_(1.5)
        vnm.vnm_gated_linear_backward(dy, x, wg, wu, a, b, sa, sb, act=SILU, dx=o[0][0], dwg=o[1][0], dwu=o[2][0], h=o[3][0], accumulate=accumulate)
        assert vnm.vnm_dense_get_status() == vnm.VNM_OK
        check_gradients(dy, x, wg, wu, widened(a, sa), widened(b, sb), SILU, *(v for v, _ in o), BF16, 1.5 if accumulate else 0.0)
        assert all(untouched(v, buf) for v, buf in o)
