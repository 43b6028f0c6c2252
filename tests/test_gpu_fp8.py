"""The block-scaled 8-bit quantiser and Linear layer against plain 64-bit forms."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense_util import DEV, check_linear, check_quantized, groups, linear64, padded, quantize  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def _randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


def _outputs(R, C, rows, fp8, pad=0):
    q, qt = (padded(*n, torch.uint8, pad).view(fp8) if pad == 0 else
             torch.zeros((n[0], n[1] + pad), dtype=torch.uint8, device=DEV).view(fp8)[:, :n[1]] for n in ((R, C), (C, R)))
    return q, torch.empty((-(-R // rows), groups(C)), device=DEV), qt, torch.empty((-(-C // rows), groups(R)), device=DEV)


# ------------------------------------------------------------------ quantiser


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("fp8", [E4M3, E5M2])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 4096), (128, 128), (127, 129), (300, 70), (257, 1001), (640, 384)])
def test_quantize(R, C, rows, fp8, dtype):
    x = (_randn(R, C, seed=R + C) * torch.exp(2 * _randn(R, 1, seed=1))).to(dtype)
    q, s, qt, st = _outputs(R, C, rows, fp8)
    vnm.vnm_fp8_quantize(x, q, s, qt, st, block_rows=rows)
    check_quantized(q, s, x, rows, 0.0, "plain")
    check_quantized(qt, st, x.t(), rows, 0.0, "transposed")
    if rows == 128:
        assert torch.equal(s, st.t())
        assert torch.equal(q.contiguous().view(torch.uint8), qt.contiguous().view(torch.uint8).t())


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("only", ["plain", "transposed"])
def test_quantize_one_side(rows, only):
    x = _randn(200, 333, seed=2).to(F16)
    q, s, qt, st = _outputs(200, 333, rows, E4M3)
    if only == "plain":
        vnm.vnm_fp8_quantize(x, q, s, block_rows=rows)
        check_quantized(q, s, x, rows, 0.0)
    else:
        vnm.vnm_fp8_quantize(x, qt=qt, st=st, block_rows=rows)
        check_quantized(qt, st, x.t(), rows, 0.0)


@pytest.mark.parametrize("R,C,pad,off", [(130, 140, 4, 0), (130, 144, 16, 8), (131, 144, 3, 1), (64, 256, 8, 3)])
def test_quantize_strides_and_canaries(R, C, pad, off):
    x = torch.zeros((R, C + pad + off), dtype=F16, device=DEV)[:, off:off + C]
    x.copy_(_randn(R, C, seed=4).to(F16))
    bq = torch.full((R + 2, C + pad + off), 0x55, dtype=torch.uint8, device=DEV)
    bt = torch.full((C + 2, R + pad + off), 0x55, dtype=torch.uint8, device=DEV)
    q, qt = bq.view(E4M3)[1:R + 1, off:off + C], bt.view(E4M3)[1:C + 1, off:off + R]
    s, st = torch.empty((groups(C), R), device=DEV).t(), torch.empty((C, groups(R) + 2), device=DEV)[:, 1:-1]
    vnm.vnm_fp8_quantize(x, q, s, qt, st)
    check_quantized(q, s, x, 1, 0.0)
    check_quantized(qt, st, x.t(), 1, 0.0)
    bq[1:R + 1, off:off + C] = 0x55
    bt[1:C + 1, off:off + R] = 0x55
    assert (bq == 0x55).all() and (bt == 0x55).all()


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_zeros_tiny_huge_and_non_finite(rows):
    x = _randn(256, 512, seed=6)
    x[0:128, 0:128] = 0.0
    x[0:128, 128:256] = 1e-38
    x[0:128, 256:384] *= 1e37
    x[130, 5] = float("inf")
    x[200, 300] = float("nan")
    q, s, qt, st = _outputs(256, 512, rows, E4M3)
    vnm.vnm_fp8_quantize(x, q, s, qt, st, block_rows=rows)
    check_quantized(q, s, x, rows, 0.0, "plain")
    check_quantized(qt, st, x.t(), rows, 0.0, "transposed")
    assert (s[0, 0] == 2.0 ** -100) and (q[0, :128].float() == 0).all()


def test_quantize_ties_to_even_and_the_ends_of_the_range():
    # the scale is exactly 1: ties between e4m3 neighbours go to the even mantissa
    x = torch.zeros((1, 128), device=DEV)
    vals = [448.0, 17.0, 19.0, 432.0, 2.0 ** -10, 3 * 2.0 ** -10, -17.0, 2.0 ** -11]
    want = [448.0, 16.0, 20.0, 448.0, 0.0, 2.0 ** -8, -16.0, 0.0]
    x[0, :8] = torch.tensor(vals, device=DEV)
    q, s, _, _ = _outputs(1, 128, 1, E4M3)
    vnm.vnm_fp8_quantize(x, q, s)
    assert s.item() == 1.0
    assert q[0, :8].float().tolist() == want


# ------------------------------------------------------------------ Linear layer


def _operands(T, R, K, rows, fx, fw, seed):
    xq, xs = quantize(_randn(T, K, seed=seed), 1, fx)
    wq, ws = quantize(0.05 * _randn(R, K, seed=seed + 1), rows, fw)
    return xq, xs, wq, ws


def _linear(T, R, K, rows=128, fx=E4M3, fw=E4M3, y_type=F32, bias_type=None, act=0, seed=0):
    xq, xs, wq, ws = _operands(T, R, K, rows, fx, fw, seed + T + R + K)
    bias = _randn(R, seed=seed + 5).to(bias_type) if bias_type is not None else None
    Y = torch.full((T, R), float("nan"), dtype=y_type, device=DEV)
    status = torch.zeros(3, dtype=torch.int32, device=DEV)
    vnm.vnm_fp8_linear(xq, xs, wq, ws, Y, bias=bias, act=act, status=status)
    assert status.tolist() == [0, 0, 0]
    check_linear(Y, linear64(xq, xs, wq, ws, bias, act), K, act, f"{T}x{R}x{K}")
    return xq, xs, wq, ws, bias, Y


# every tile width of the tokens, every split of K, ragged edges of all three sizes, K under one block
@pytest.mark.parametrize("T", [1, 2, 16, 17, 32, 33, 64, 65, 130])
@pytest.mark.parametrize("R,K", [(1, 1), (128, 128), (130, 1000), (300, 4096), (5, 200)])
@pytest.mark.parametrize("rows", [1, 128])
def test_few_tokens(T, R, K, rows):
    _linear(T, R, K, rows)


@pytest.mark.parametrize("T,R,K", [(2500, 2000, 300), (2432, 2048, 512), (131, 20000, 129), (1300, 3333, 1041)])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("y_type", [F16, F32])
def test_many_tiles(T, R, K, rows, y_type):
    _linear(T, R, K, rows, y_type=y_type)


@pytest.mark.parametrize("T,R,K", [(3, 200, 640), (2500, 2000, 256)])
@pytest.mark.parametrize("y_type,bias_type", [(F16, F16), (BF16, BF16), (F32, F32), (F16, F32), (BF16, F16)])
@pytest.mark.parametrize("act", [0, 1, 2])
def test_types_bias_and_activations(T, R, K, y_type, bias_type, act):
    _linear(T, R, K, y_type=y_type, bias_type=bias_type, act=act)


@pytest.mark.parametrize("T,R,K", [(9, 256, 384), (2500, 2000, 256)])
@pytest.mark.parametrize("fx,fw", [(E5M2, E4M3), (E4M3, E5M2), (E5M2, E5M2)])
def test_formats(T, R, K, fx, fw):
    _linear(T, R, K, fx=fx, fw=fw)


@pytest.mark.parametrize("T,R,K", [(7, 300, 700), (2500, 2000, 300)])
def test_exact_products(T, R, K):
    """Small whole numbers and scales that are powers of two: every sum is exact."""
    g = torch.Generator(device=DEV).manual_seed(8)
    xq, wq = (torch.randint(-3, 4, (n, -(-K // 16) * 16), generator=g, device=DEV).float().to(E4M3)[:, :K] for n in (T, R))
    xs = 2.0 ** torch.randint(-3, 3, (T, groups(K)), generator=g, device=DEV).float()
    ws = 2.0 ** torch.randint(-3, 3, (groups(R), groups(K)), generator=g, device=DEV).float()
    Y = torch.empty((T, R), device=DEV)
    vnm.vnm_fp8_linear(xq, xs, wq, ws, Y)
    assert torch.equal(Y.double(), linear64(xq, xs, wq, ws, None, 0)[0])


@pytest.mark.parametrize("T,R,K,pad", [(5, 250, 300, 3), (33, 256, 256, 8), (2500, 2000, 256, 3), (2500, 2000, 256, 8),
                                       (2500, 2000, 256, 16)])
@pytest.mark.parametrize("y_type", [BF16, F32])
def test_output_strides_and_canaries(T, R, K, pad, y_type):
    xq, xs, wq, ws = _operands(T, R, K, 128, E4M3, E4M3, 3)
    buf = torch.full((T + 2, R + pad), 7.0, dtype=y_type, device=DEV)
    Y = buf[1:T + 1, :R]
    vnm.vnm_fp8_linear(xq, xs, wq, ws, Y)
    check_linear(Y, linear64(xq, xs, wq, ws, None, 0), K, 0)
    buf[1:T + 1, :R] = 7.0
    assert (buf == 7.0).all()


@pytest.mark.parametrize("T,R,K", [(5, 250, 300), (2500, 2000, 300)])
def test_scale_strides_and_operand_padding(T, R, K):
    """Scales by group and with gaps; NaN bytes in the operands' row padding."""
    xq, xs, wq, ws = _operands(T, R, K, 128, E4M3, E4M3, 4)
    ld = -(-K // 16) * 16 + 32
    bx, bw = (torch.full((n, ld), 0x7F, dtype=torch.uint8, device=DEV) for n in (T, R))
    bx[:, :K], bw[:, :K] = xq.view(torch.uint8), wq.view(torch.uint8)
    xs2 = torch.full((2 * groups(K), T + 3), float("nan"), device=DEV)[::2, 1:T + 1].t()
    ws2 = torch.full((groups(K), groups(R)), float("nan"), device=DEV).t()
    xs2.copy_(xs)
    ws2.copy_(ws)
    Y = torch.empty((T, R), device=DEV)
    vnm.vnm_fp8_linear(bx.view(E4M3)[:, :K], xs2, bw.view(E4M3)[:, :K], ws2, Y)
    check_linear(Y, linear64(xq, xs, wq, ws, None, 0), K, 0)


@pytest.mark.parametrize("T,R,K", [(4, 300, 512), (2500, 2000, 256)])
def test_non_finite_values_stay_in_their_rows(T, R, K):
    xq, xs, wq, ws = _operands(T, R, K, 1, E4M3, E4M3, 6)
    xs[1, 1] = float("nan")
    wq.view(torch.uint8)[7, 130] = 0x7F
    Y = torch.empty((T, R), device=DEV)
    vnm.vnm_fp8_linear(xq, xs, wq, ws, Y, act=vnm.VNM_ACT_RELU)
    assert Y[1].isnan().all() and Y[:, 7].isnan().all()
    t, r = [i for i in range(T) if i != 1], [i for i in range(R) if i != 7]
    ref = linear64(xq[t].contiguous(), xs[t], wq[r].contiguous(), ws[r], None, 1)
    check_linear(Y[t][:, r], ref, K, 1)


@pytest.mark.parametrize("T,R,K", [(0, 64, 128), (8, 0, 128)])
def test_empty(T, R, K):
    vnm.vnm_fp8_linear(torch.empty((T, K), dtype=E4M3, device=DEV), torch.empty((T, 1), device=DEV),
                       torch.empty((R, K), dtype=E4M3, device=DEV), torch.empty((groups(R), 1), device=DEV),
                       torch.empty((T, R), device=DEV))


@pytest.mark.parametrize("act", [0, 1, 2])
def test_no_columns_gives_the_bias(act):
    bias = _randn(70, seed=9)
    Y = torch.full((5, 70), float("nan"), device=DEV)
    vnm.vnm_fp8_linear(torch.empty((5, 0), dtype=E4M3, device=DEV), torch.empty((5, 0), device=DEV),
                       torch.empty((70, 0), dtype=E4M3, device=DEV), torch.empty((1, 0), device=DEV), Y, bias=bias, act=act)
    b = bias.double()
    want = b if act == 0 else b.clamp_min(0) if act == 1 else b * 0.5 * torch.erfc(-b / 2.0 ** 0.5)
    assert ((Y.double() - want).abs() <= 8 * 2.0 ** -23 * bias.double().abs()).all()


@pytest.mark.parametrize("T,R,K", [(16, 4096, 4096), (2500, 2000, 1024)])
def test_same_bits_every_time_and_on_another_stream(T, R, K):
    xq, xs, wq, ws = _operands(T, R, K, 128, E4M3, E4M3, 7)
    Y = [torch.empty((T, R), device=DEV) for _ in range(3)]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    vnm.vnm_fp8_linear(xq, xs, wq, ws, Y[0])
    vnm.vnm_fp8_linear(xq, xs, wq, ws, Y[1])
    vnm.vnm_fp8_linear(xq, xs, wq, ws, Y[2], stream=st)
    torch.cuda.synchronize()
    assert torch.equal(Y[0], Y[1]) and torch.equal(Y[0], Y[2])


def test_graph_capture():
    T, R, K = 4, 512, 1024
    xq, xs, wq, ws = _operands(T, R, K, 128, E4M3, E4M3, 8)
    x = _randn(T, K, seed=1).to(F16)
    Y, q, s = torch.empty((T, R), device=DEV), *_outputs(T, K, 1, E4M3)[:2]
    vnm.vnm_fp8_linear(xq, xs, wq, ws, Y)  # attributes are set on the first call
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vnm.vnm_fp8_quantize(x, q, s)
        vnm.vnm_fp8_linear(q, s, wq, ws, Y)
    x.copy_(_randn(T, K, seed=2).to(F16))
    g.replay()
    torch.cuda.synchronize()
    check_quantized(q, s, x, 1, 0.0)
    check_linear(Y, linear64(q, s, wq, ws, None, 0), K, 0)


# ------------------------------------------------------------------ gradients


def test_gradients_of_the_layer():
    """Y = X W^T, dX = dY W and dW = dY^T X as three products, all on operands
    quantised by the library: against the 64-bit products of the values the
    8-bit operands stand for, and within the quantisation's error (each element within 2^-4 of
    itself or of its group's end of range) of the gradients of the unquantised layer."""
    T, R, K = 200, 300, 260
    x, w, dy = _randn(T, K, seed=1), 0.1 * _randn(R, K, seed=2), _randn(T, R, seed=3)

    def both(t, rows, fp8):
        n = [torch.zeros((a, -(-b // 16) * 16), dtype=torch.uint8, device=DEV).view(fp8)[:, :b] for a, b in (t.shape, t.shape[::-1])]
        s = [torch.empty((-(-a // rows), groups(b)), device=DEV) for a, b in (t.shape, t.shape[::-1])]
        vnm.vnm_fp8_quantize(t, n[0], s[0], n[1], s[1], block_rows=rows)
        return n[0], s[0], n[1], s[1]

    xq, xs, xt, xts = both(x, 1, E4M3)
    wq, ws, wt, wts = both(w, 128, E4M3)
    dq, ds, dt, dts = both(dy, 1, E5M2)
    for (a, sa, b, sb), plain in (((xq, xs, wq, ws), x.double() @ w.double().t()),
                                  ((dq, ds, wt, wts), dy.double() @ w.double()),
                                  ((dt, dts, xt, xts), dy.double().t() @ x.double())):
        Y = torch.empty((a.shape[0], b.shape[0]), device=DEV)
        vnm.vnm_fp8_linear(a, sa, b, sb, Y)
        ref = linear64(a, sa, b, sb, None, 0)
        check_linear(Y, ref, a.shape[1], 0)
        # e5m2 is within 2^-3 of each normal value, e4m3 within 2^-4; the sums' signs are random
        assert ((Y.double() - plain).norm() <= 0.2 * plain.norm())


def test_gradient_against_differences():
    """The layer is linear in X: the difference of Y along one X element is the
    column that dX's product uses."""
    T, R, K = 3, 140, 150
    xq, xs, wq, ws = _operands(T, R, K, 128, E4M3, E4M3, 11)
    dy = torch.ones((T, R), device=DEV)
    wt = torch.zeros((K, -(-R // 16) * 16), dtype=torch.uint8, device=DEV).view(E4M3)[:, :R]
    wt.view(torch.uint8).copy_(wq.view(torch.uint8).t())
    dq, ds = quantize(dy, 1, E4M3)
    dX = torch.empty((T, K), device=DEV)
    vnm.vnm_fp8_linear(dq, ds, wt, ws.t(), dX)
    for k in (0, 77, 149):
        buf = [torch.zeros((T, -(-K // 16) * 16), dtype=torch.uint8, device=DEV).view(E4M3)[:, :K] for _ in range(2)]
        for t, v in zip(buf, (2.0, -2.0)):
            t.view(torch.uint8).copy_(xq.view(torch.uint8))
            t[:, k] = torch.full((T,), v, device=DEV).to(E4M3)
        Y = [torch.empty((T, R), device=DEV) for _ in range(2)]
        for t, y in zip(buf, Y):
            vnm.vnm_fp8_linear(t, xs, wq, ws, y)
        num = (Y[0].double() - Y[1].double()).sum(1) / (4.0 * xs[:, k // 128].double())
        # dY of ones is 448 times 1 / 448: one rounding of the scale; the sums cancel to 1e-5 of their terms
        size = linear64(torch.ones_like(num)[:, None].expand(T, R).float().to(E4M3), torch.ones((T, groups(R)), device=DEV),
                        wt[k:k + 1], ws.t()[k // 128:k // 128 + 1], None, 0)[1][:, 0]
        big = linear64(xq, xs, wq, ws, None, 0)[1].sum(1) / xs[:, k // 128].double()
        assert ((dX[:, k].double() - num).abs() <= 2e-5 * (size + big)).all()


def test_binding_refusals():
    xq, xs, wq, ws = _operands(4, 256, 256, 128, E4M3, E4M3, 12)
    Y = torch.empty((4, 256), device=DEV)
    ok = dict(xq=xq, x_scale=xs, wq=wq, w_scale=ws, Y=Y)
    for bad in (dict(Y=Y[:3]), dict(Y=Y.double()), dict(xq=xq.view(torch.uint8)), dict(wq=wq[:, :255]), dict(x_scale=xs.double()),
                dict(x_scale=xs[:, :1]), dict(w_scale=ws[:1]), dict(w_scale=torch.empty((3, 2), device=DEV)),
                dict(bias=torch.empty(255, device=DEV)), dict(Y=torch.empty((4, 256))),
                dict(status=torch.zeros(2, dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError):
            vnm.vnm_fp8_linear(**{**ok, **bad})
    # rows that a tensor-memory copy cannot read
    odd = torch.zeros((4, 257), dtype=torch.uint8, device=DEV).view(E4M3)
    for bad in (dict(xq=odd[:, :256]), dict(xq=torch.zeros((4, 272), dtype=torch.uint8, device=DEV).view(E4M3)[:, 1:257]),
                dict(act=9)):
        with pytest.raises(vnm.VnmError) as e:
            vnm.vnm_fp8_linear(**{**ok, **bad})
        assert e.value.code == vnm.VNM_ERR_INVALID_ARG
    x = _randn(4, 256, seed=1)
    q, s, qt, st = _outputs(4, 256, 1, E4M3)
    for kw in (dict(q=q, s=s[:, :1]), dict(q=q[:3], s=s), dict(q=q.float(), s=s), dict(q=q, s=s, qt=qt.view(E5M2), st=st)):
        with pytest.raises(ValueError):
            vnm.vnm_fp8_quantize(x, **kw)
    for kw in (dict(), dict(q=q), dict(s=s), dict(q=q, s=torch.empty((2, 2), device=DEV), block_rows=2)):
        with pytest.raises(vnm.VnmError) as e:
            vnm.vnm_fp8_quantize(x, **kw)
        assert e.value.code == vnm.VNM_ERR_INVALID_ARG


@pytest.mark.parametrize("T,R,K,skip", [(16, 512, 4096, 2), (2500, 2000, 1024, 3), (2500, 2000, 1024, 9)])
def test_bounded_wait_reports_timeout_and_device_stays_usable(T, R, K, skip):
    """A stage whose loads are never issued (split K, and the persistent grid): the
    waits run out after about a second, the status says so, the next call is right."""
    xq, xs, wq, ws = _operands(T, R, K, 128, E4M3, E4M3, 13)
    Y = torch.empty((T, R), device=DEV)
    status = torch.zeros(3, dtype=torch.int32, device=DEV)
    vnm.vnm_testing_fp8_linear_skip_stage(xq, xs, wq, ws, Y, skip, status=status)
    torch.cuda.synchronize()
    assert status[0].item() == vnm.VNM_ERR_TIMEOUT
    status.zero_()
    vnm.vnm_fp8_linear(xq, xs, wq, ws, Y, status=status)
    assert status.tolist() == [0, 0, 0]
    check_linear(Y, linear64(xq, xs, wq, ws, None, 0), K, 0)


@pytest.mark.parametrize("y_type", [F32, F16])
@pytest.mark.parametrize("T,R,K", [(200, 300, 260), (300, 2200, 130), (1100, 1060, 100)])
def test_outputs_that_end_inside_a_tile(T, R, K, y_type):
    """Tiles of which only some of the output boxes exist, many times: a box past the
    edge must not reuse memory that a box before it is still being stored from."""
    xq, xs, wq, ws = _operands(T, R, K, 128, E4M3, E4M3, 14)
    ref = linear64(xq, xs, wq, ws, None, 0)
    Y = [torch.full((T, R), float("nan"), dtype=y_type, device=DEV) for _ in range(24)]
    for y in Y:
        vnm.vnm_fp8_linear(xq, xs, wq, ws, y)
    for y in Y:
        check_linear(y, ref, K, 0)


@pytest.mark.parametrize("T,R,K,off", [(300, 301, 100, 0), (2500, 1999, 130, 0), (2500, 2003, 130, 1), (600, 2050, 70, 3)])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("y_type", [F16, F32])
def test_outputs_of_any_alignment(T, R, K, off, rows, y_type):
    """Rows of Y that TMA cannot write: odd widths, and a start off every alignment but the type's."""
    xq, xs, wq, ws = _operands(T, R, K, rows, E4M3, E4M3, 15)
    buf = torch.full((T + 2, R + off), 7.0, dtype=y_type, device=DEV)
    Y = buf[1:T + 1, off:]
    vnm.vnm_fp8_linear(xq, xs, wq, ws, Y)
    check_linear(Y, linear64(xq, xs, wq, ws, None, 0), K, 0)
    buf[1:T + 1, off:] = 7.0
    assert (buf == 7.0).all()


@pytest.mark.parametrize("T,R,K", [(1, 33, 1259), (3, 16, 127), (8, 40, 129), (5, 17, 1)])
def test_last_rows_end_with_their_storage(T, R, K):
    """Operands whose storage ends with the last row's last element: nothing past it is read
    into the sums (the storage is cut from buffers of NaN bytes)."""
    xq, xs, wq, ws = _operands(T, R, K, 1, E4M3, E4M3, 16)
    ld = -(-K // 16) * 16
    flat = [torch.full(((n - 1) * ld + K + 64,), 0x7F, dtype=torch.uint8, device=DEV) for n in (T, R)]
    cut = [f[: (n - 1) * ld + K].as_strided((n, K), (ld, 1)) for f, n in zip(flat, (T, R))]
    cut[0].copy_(xq.view(torch.uint8))
    cut[1].copy_(wq.view(torch.uint8))
    Y = torch.empty((T, R), device=DEV)
    vnm.vnm_fp8_linear(cut[0].view(E4M3), xs, cut[1].view(E4M3), ws, Y)
    check_linear(Y, linear64(xq, xs, wq, ws, None, 0), K, 0)
