"""vnm_dense_linear: the dense 16-bit product with bias, activation and residual, and its gradients'
products, against 64-bit forms."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense16_util import (BF16, DEV, F16, F32, GELU, NONE, RELU, SILU, ULP, act64, act_bound, canvas, check, generator,  # noqa: E402
                          operand, pitched, untouched, whole)

SIZES = [(1, 1, 1), (1, 16, 64), (1, 1000, 1041), (2, 7, 8), (3, 129, 63), (5, 300, 65), (8, 130, 200), (8, 64, 2100), (9, 17, 9),
         (16, 300, 1041), (17, 64, 64), (33, 1, 300), (40, 1000, 72), (64, 129, 513), (65, 130, 128), (100, 257, 1), (130, 300, 4200),
         (257, 255, 511), (300, 2050, 129), (600, 520, 2500), (1200, 3000, 200)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,R,K", SIZES)
def test_exact_sums(T, R, K, dtype):
    """Whole numbers: bit for bit, for every order of the operands, with nothing written beside Y."""
    g = generator(T, R, K, 1)
    x, w = whole(g, T, K, dtype), whole(g, R, K, dtype)
    want = x.double() @ w.double().t()
    for tx, tw in ((False, False), (False, True), (True, True), (True, False)):
        for out in (dtype, F32):
            Y, buf = canvas(T, R, out, pad=3)
            vnm.vnm_dense_linear(operand(x, tx), operand(w, tw), Y)
            assert vnm.vnm_dense_get_status() == vnm.VNM_OK
            assert torch.equal(Y, want.float().to(out)), (tx, tw, out, (Y.double() - want).abs().max().item())
            assert untouched(Y, buf)


@pytest.mark.parametrize("T,R,K", [(1, 300, 200), (8, 17, 64), (16, 300, 1041), (40, 130, 72), (300, 520, 129), (600, 1001, 300)])
@pytest.mark.parametrize("out,bias,aligned", [(F16, F32, True), (F16, F16, False), (F32, BF16, True), (F32, F32, False)])
@pytest.mark.parametrize("act", [NONE, RELU, GELU, SILU])
def test_epilogue(T, R, K, out, bias, aligned, act):
    """Bias, activation and residual in fp32, rounded once; the residual also in place."""
    g = generator(T, R, K, act)
    x, w = whole(g, T, K, F16, unit=0.125), whole(g, R, K, F16, unit=0.25)
    b = whole(g, 1, R, bias, unit=0.25)[0].contiguous()
    pad, offset = (-R % 8, 0) if aligned else (1, 1)
    res, _ = canvas(T, R, out, pad, offset)
    res.copy_(whole(g, T, R, out, top=9, unit=0.5))
    z = x.double() @ w.double().t() + b.double()
    want, bound = act64(z, act), act_bound(z, act)
    if act != NONE and act != RELU:
        bound = bound + ULP * (want.abs() + res.double().abs())  # the sum with the residual
    Y, buf = canvas(T, R, out, pad, offset)
    vnm.vnm_dense_linear(pitched(x), pitched(w), Y, bias=b, act=act, residual=res)
    check(Y, want + res.double(), bound)
    assert untouched(Y, buf)
    Z = res.clone() if aligned else res
    vnm.vnm_dense_linear(pitched(x), pitched(w), Z, bias=b, act=act, residual=Z)
    assert torch.equal(Y, Z)
    vnm.vnm_dense_linear(pitched(x), pitched(w), Y, bias=b, act=act)
    check(Y, want, act_bound(z, act))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,R,K", [(1, 256, 11008), (16, 256, 11008), (200, 300, 8192), (700, 700, 8192), (2000, 2000, 5000)])
def test_long_sums(T, R, K, dtype):
    """Real numbers: K additions of truncated sums; fp32 outputs take their sums out every 2048 elements,
    which holds random sums to 2048 * 2^-23 of the result's norm, and in truth far closer."""
    g = generator(T, R, K, 3)
    x, w = torch.randn(T, K, generator=g, device=DEV).to(dtype), torch.randn(R, K, generator=g, device=DEV).to(dtype)
    want, mag = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
    for out in (dtype, F32):
        Y = torch.empty((T, R), dtype=out, device=DEV)
        vnm.vnm_dense_linear(x, w, Y)
        check(Y, want, (min(K, 2048 if out == F32 else K) + K // 2048 + 16) * ULP * mag)
        if out == F32:
            assert ((Y.double() - want).norm() / want.norm()).item() <= 2048 * ULP


@pytest.mark.parametrize("T,R,K", [(8, 40, 64), (600, 520, 300)])
def test_infinities_and_nan_stay_in_their_rows(T, R, K):
    g = generator(T, R, 4)
    x, w = whole(g, T, K, F16), whole(g, R, K, F16)
    want = x.double() @ w.double().t()
    x[T - 1, 3], w[5, 7] = float("nan"), float("inf")
    Y = torch.empty((T, R), dtype=F16, device=DEV)
    vnm.vnm_dense_linear(pitched(x), pitched(w), Y)
    assert Y[T - 1].isnan().all() and not torch.isfinite(Y[:, 5]).any()
    keep = torch.ones(R, dtype=torch.bool, device=DEV)
    keep[5] = False
    assert torch.equal(Y[: T - 1, keep], want[: T - 1, keep].half())


def test_empty_sizes():
    x, w, b = torch.empty((3, 0), dtype=F16, device=DEV), torch.empty((5, 0), dtype=F16, device=DEV), torch.randn(5, device=DEV).half()
    res = torch.randn(3, 5, device=DEV).half()
    Y = torch.full((3, 5), float("nan"), dtype=F16, device=DEV)
    vnm.vnm_dense_linear(x, w, Y, bias=b, act=RELU, residual=res)
    assert torch.equal(Y, (b.float().clamp_min(0) + res.float()).half())
    vnm.vnm_dense_linear(x, w, Y)
    assert (Y == 0).all()
    vnm.vnm_dense_linear(torch.empty((0, 8), dtype=F16, device=DEV), torch.empty((5, 8), dtype=F16, device=DEV), Y[:0])
    vnm.vnm_dense_linear(torch.empty((3, 8), dtype=F16, device=DEV), torch.empty((0, 8), dtype=F16, device=DEV), Y[:, :0])


def test_gradients_against_formula_and_differences():
    """dX and dW as products of the transposed views; against a central difference of the 64-bit form."""
    T, R, K = 70, 90, 100
    g = generator(5)
    x, w, dy = (pitched(torch.randn(*s, generator=g, device=DEV).half()) for s in ((T, K), (R, K), (T, R)))
    dx, dw = torch.empty((T, K), device=DEV), torch.ones((R, K), device=DEV)
    vnm.vnm_dense_linear(dy, w.t(), dx)
    vnm.vnm_dense_linear(dy.t(), x.t(), dw, residual=dw)  # added to
    dw -= 1
    x64, w64, d64 = x.double(), w.double(), dy.double()
    check(dx, d64 @ w64, (R + 8) * ULP * (d64.abs() @ w64.abs()))
    check(dw, d64.t() @ x64, (T + 8) * ULP * (d64.abs().t() @ x64.abs()) + 2 * ULP)

    def loss(a, b):
        return ((a @ b.t()) * d64).sum()

    for base, grad, f in ((x64, dx, lambda v: loss(v, w64)), (w64, dw, lambda v: loss(x64, v))):
        way = torch.randn(base.shape, generator=g, device=DEV, dtype=torch.float64)
        diff = (f(base + way) - f(base - way)).item() / 2  # (the loss is linear)
        assert abs((grad.double() * way).sum().item() - diff) <= 1e-5 * (grad.double().norm() * way.norm()).item()


@pytest.mark.parametrize("T,R,K", [(4, 520, 640), (24, 520, 640), (600, 520, 640)])
def test_streams_and_graph(T, R, K):
    """On another stream, and captured and replayed on new inputs."""
    g = generator(T, 6)
    w = whole(g, R, K, BF16)
    x, x2 = whole(g, T, K, BF16), whole(g, T, K, BF16)
    Y, side = torch.empty((T, R), dtype=BF16, device=DEV), torch.cuda.Stream()
    torch.cuda.synchronize()
    vnm.vnm_dense_linear(x, w, Y, stream=side)
    side.synchronize()
    assert torch.equal(Y, (x.double() @ w.double().t()).bfloat16())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vnm.vnm_dense_linear(x, w, Y)
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, (x2.double() @ w.double().t()).bfloat16())


@pytest.mark.parametrize("T,R,K,skip", [(16, 512, 4096, 2), (40, 300, 8192, 9), (2500, 2000, 1024, 9)])
@pytest.mark.parametrize("out", [F16, F32])
def test_time_out(T, R, K, skip, out):
    """A stage that never arrives: the waits run out, the error is kept, the next call is right."""
    g = generator(T, 7)
    x, w = whole(g, T, K, F16), whole(g, R, K, F16)
    Y, own = torch.empty((T, R), dtype=out, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK
    vnm.vnm_testing_dense_linear_skip_stage(x, w, Y, skip)
    assert vnm.vnm_dense_get_status() == vnm.VNM_ERR_TIMEOUT
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK
    vnm.vnm_testing_dense_linear_skip_stage(x, w, Y, skip, status=own)
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK and own[0].item() == vnm.VNM_ERR_TIMEOUT
    vnm.vnm_dense_linear(x, w, Y)
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK
    assert torch.equal(Y, (x.double() @ w.double().t()).float().to(out))


def test_refusals():
    x, w, Y = (torch.zeros(*s, dtype=F16, device=DEV) for s in ((16, 64), (32, 64), (16, 32)))
    wide = torch.zeros(32, 130, dtype=F16, device=DEV)
    for bad in (lambda: vnm.vnm_dense_linear(x.float(), w, Y), lambda: vnm.vnm_dense_linear(x, w.bfloat16(), Y),
                lambda: vnm.vnm_dense_linear(x, w, Y.t()), lambda: vnm.vnm_dense_linear(x[:, :60], w, Y),
                lambda: vnm.vnm_dense_linear(x, w, Y.bfloat16()), lambda: vnm.vnm_dense_linear(x, w, Y, residual=Y.float()),
                lambda: vnm.vnm_dense_linear(x, w, Y, bias=torch.zeros(31, device=DEV)),
                lambda: vnm.vnm_dense_linear(x, w, Y, act=4), lambda: vnm.vnm_dense_linear(x, w, Y, act=1 << 33),
                lambda: vnm.vnm_dense_linear(x, wide[:, 1:65], Y), lambda: vnm.vnm_dense_linear(x, wide[:, 2:66], Y),
                lambda: vnm.vnm_dense_linear(x[:1].expand(16, 64), w, Y), lambda: vnm.vnm_dense_linear(x.cpu(), w, Y),
                lambda: vnm.vnm_dense_linear(x, w, Y, status=torch.zeros(2, dtype=torch.int32, device=DEV)),
                lambda: vnm.vnm_dense_linear(x, w[:, ::2], Y)):
        with pytest.raises((ValueError, vnm.VnmError)):
            bad()
    torch.cuda.synchronize()
