"""Products with a scale a row on both sides and many K blocks, as a weight gradient over a batch
of tokens is: the ring that the scales pass through turns over several times, by loads of four
blocks where the scales' rows are 16 aligned bytes, by single ones elsewhere and for the
blocks that are left."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense_util import DEV, check_linear, groups, linear64, quantize  # noqa: E402

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def _laid_out(s, how):
    """The same scales in other strides, NaN between them."""
    n, G = s.shape
    pad = {"aligned": (-(-G // 4) * 4, 0), "unaligned": (-(-G // 4) * 4 + 4, 1), "odd rows": (G | 1, 0)}.get(how)
    if pad is None:  # by group
        out = torch.full((G, n + 3), float("nan"), device=DEV)[:, :n].t()
    else:
        out = torch.full((n, pad[0]), float("nan"), device=DEV)[:, pad[1]:pad[1] + G]
    out.copy_(s)
    return out


# one tile a pair and several; K of whole and of broken groups of four blocks, a last block that is short
@pytest.mark.parametrize("T,R,K", [(4096, 1024, 2048), (1500, 1490, 4200), (2600, 2300, 2150), (2304, 2304, 1408)])
@pytest.mark.parametrize("x_scales,w_scales", [("aligned", "aligned"), ("unaligned", "aligned"), ("aligned", "odd rows"),
                                               ("by group", "by group")])
def test_many_blocks(T, R, K, x_scales, w_scales):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert vnm.vnm_testing_fp8_linear_plan(T, R, K, 1, sms) == (0, 1)
    g = torch.Generator(device=DEV).manual_seed(K)
    xq, xs = quantize(torch.randn(T, K, generator=g, device=DEV), 1, E5M2)
    wq, ws = quantize(torch.randn(R, K, generator=g, device=DEV), 1, E4M3)
    ref = linear64(xq, xs, wq, ws, None, 0)
    xl, wl = _laid_out(xs, x_scales), _laid_out(ws, w_scales)
    Y = [torch.full((T, R), float("nan"), device=DEV) for _ in range(4)]
    for y in Y:
        vnm.vnm_fp8_linear(xq, xl, wq, wl, y)
    assert vnm.vnm_fp8_linear_get_status() == vnm.VNM_OK
    check_linear(Y[0], ref, K, 0, f"{T}x{R}x{K}")
    assert all(torch.equal(Y[0], y) for y in Y)


# the same ring of the narrow tiles (a scale a token), several tiles a CTA
@pytest.mark.parametrize("T,R,K", [(36, 39990, 2100), (69, 19676, 1170)])
@pytest.mark.parametrize("x_scales", ["aligned", "unaligned", "by group"])
@pytest.mark.parametrize("rows", [1, 128])
def test_many_blocks_of_few_tokens(T, R, K, x_scales, rows):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert vnm.vnm_testing_fp8_linear_plan(T, R, K, rows, sms)[0] in (64, 128)
    g = torch.Generator(device=DEV).manual_seed(K)
    xq, xs = quantize(torch.randn(T, K, generator=g, device=DEV), 1, E4M3)
    wq, ws = quantize(torch.randn(R, K, generator=g, device=DEV), rows, E4M3)
    Y = torch.full((T, R), float("nan"), device=DEV)
    vnm.vnm_fp8_linear(xq, _laid_out(xs, x_scales), wq, ws, Y)
    check_linear(Y, linear64(xq, xs, wq, ws, None, 0), K, 0, f"{T}x{R}x{K}")


def test_weight_gradient_of_a_batch():
    """dW = dY^T X over 4096 tokens, both operands by the library's quantiser, transposed: against
    64 bits of what they stand for, and within the quantisation of the gradient itself."""
    T, R, D = 4096, 600, 520
    g = torch.Generator(device=DEV).manual_seed(7)
    dy, x = torch.randn(T, R, generator=g, device=DEV), torch.randn(T, D, generator=g, device=DEV)
    ops = []
    for t, fp8 in ((dy, E5M2), (x, E4M3)):
        qt = torch.empty((t.shape[1], T), dtype=fp8, device=DEV)
        st = torch.empty((t.shape[1], groups(T)), device=DEV)
        vnm.vnm_fp8_quantize(t, qt=qt, st=st)
        ops += [qt, st]
    dW = torch.empty((R, D), device=DEV)
    vnm.vnm_fp8_linear(*ops, dW)
    check_linear(dW, linear64(*ops, None, 0), T, 0)
    plain = dy.double().t() @ x.double()
    # e5m2 within 2^-3 of a normal value, e4m3 within 2^-4; the errors' signs are random
    assert (dW.double() - plain).norm() <= 0.2 * plain.norm()
