"""vnm_gated_linear and its backward pass against 64-bit forms: checkpoints in 16 and 8 bits, every
activation, ragged sizes, strides, and a whole block of them."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense16_util import (BF16, DEV, F16, F32, GELU, NONE, RELU, ROUND, SILU, ULP, act64, act_bound, canvas, check,  # noqa: E402
                          generator, pitched, slope64, untouched, whole, widened)
from dense_util import check_quantized  # noqa: E402

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
SIZES = [(1, 1, 8), (1, 300, 200), (3, 129, 65), (8, 128, 64), (8, 11, 2100), (9, 130, 72), (16, 300, 1041), (33, 257, 64),
         (64, 128, 300), (100, 1000, 129), (130, 131, 520), (300, 520, 1), (600, 1100, 260)]


def groups(n):
    return -(-n // 128)


def layer(g, T, F, K, dtype):
    """x, wg, wu with sums that are exact in fp32 and, for the products of two, in 24 bits."""
    return pitched(whole(g, T, K, dtype, 1)), pitched(whole(g, F, K, dtype, 1)), pitched(whole(g, F, K, dtype, 1, 0.5))


@pytest.mark.parametrize("dtype,act", [(F16, SILU), (BF16, GELU), (F16, RELU), (BF16, NONE)])
@pytest.mark.parametrize("T,F,K", SIZES)
def test_forward(T, F, K, dtype, act):
    g = generator(T, F, K)
    x, wg, wu = layer(g, T, F, K, dtype)
    G, U = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    want, bound = act64(G, act) * U, act_bound(G, act) * U.abs() + ULP * (act64(G, act) * U).abs()
    Y, buf = canvas(T, F, dtype, pad=1)
    vnm.vnm_gated_linear(x, wg, wu, Y, act=act)
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK
    check(Y, want, bound)
    assert untouched(Y, buf)
    for pad, offset in ((-F % 8, 0), (3, 1)):
        Y2 = canvas(T, F, dtype, pad, offset)[0]
        (a, abuf), (b, bbuf) = canvas(T, F, dtype, pad, offset), canvas(T, F, dtype, pad, offset)
        vnm.vnm_gated_linear(x, wg, wu, Y2, act=act, g=a, u=b)
        assert torch.equal(a, G.float().to(dtype)) and torch.equal(b, U.float().to(dtype)) and untouched(a, abuf) and untouched(b, bbuf)
        check(Y2, want, bound)
    for fp8, pad in ((E4M3, -F % 8), (E5M2, 3)):
        q = [torch.full((T, F + pad), 0x55, dtype=torch.uint8, device=DEV) for _ in range(2)]
        s = [torch.full((groups(F), T), float("nan"), device=DEV).t() for _ in range(2)]  # (any strides)
        views = [v.view(fp8)[:, :F] for v in q]
        vnm.vnm_gated_linear(x, wg, wu, Y, act=act, g=views[0], u=views[1], g_scale=s[0], u_scale=s[1])
        check(Y, want, bound)
        check_quantized(views[0], s[0], G, 1, 0.0)
        check_quantized(views[1], s[1], U, 1, 0.0)
        assert (q[0][:, F:] == 0x55).all() and (q[1][:, F:] == 0x55).all()
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK


def test_forward_nan_groups():
    """A NaN in a row of x makes its checkpoints' groups NaN and no other row's; an Inf in a row of Wg one group."""
    T, F, K = 40, 300, 64
    g = generator(1)
    x, wg, wu = layer(g, T, F, K, F16)
    x[3, 5], wg[200, 7] = float("nan"), float("inf")
    x[:, 7] = 1
    Y = torch.empty((T, F), dtype=F16, device=DEV)
    a, b = (torch.empty((T, F), dtype=E4M3, device=DEV) for _ in range(2))
    sa, sb = (torch.empty((T, 3), device=DEV) for _ in range(2))
    vnm.vnm_gated_linear(x, wg, wu, Y, g=a, u=b, g_scale=sa, u_scale=sb)
    assert sa[3].isnan().all() and sb[3].isnan().all() and a[3].float().isnan().all() and b[3].float().isnan().all()
    rest = torch.arange(T, device=DEV) != 3
    assert sa[rest][:, 1].isnan().all() and not sa[rest][:, [0, 2]].isnan().any() and not sb[rest].isnan().any()


def test_forward_empty_sizes():
    x, w = torch.empty((3, 0), dtype=F16, device=DEV), torch.empty((130, 0), dtype=F16, device=DEV)
    Y = torch.full((3, 130), float("nan"), dtype=F16, device=DEV)
    a, b = (torch.full((3, 130), 0x55, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2))
    sa, sb = (torch.full((3, 2), float("nan"), device=DEV) for _ in range(2))
    vnm.vnm_gated_linear(x, w, w, Y, g=a, u=b, g_scale=sa, u_scale=sb)
    assert (Y == 0).all() and (a.float() == 0).all() and (b.float() == 0).all() and (sa == 2.0 ** -100).all() and (sb == 2.0 ** -100).all()
    vnm.vnm_gated_linear(x[:0], w, w, Y[:0])
    vnm.vnm_gated_linear(torch.empty((3, 8), dtype=F16, device=DEV), torch.empty((0, 8), dtype=F16, device=DEV),
                         torch.empty((0, 8), dtype=F16, device=DEV), Y[:, :0])


def checkpoint(g, T, F, keep, dtype):
    """Gate and up projections as a forward pass keeps them, and the values they stand for."""
    out = []
    for _ in range(2):
        v = torch.randn(T, F, generator=g, device=DEV) * 2
        if keep is None:
            out.append((v.to(dtype), None))
        else:
            q, s = torch.empty((T, F), dtype=keep, device=DEV), torch.empty((T, groups(F)), device=DEV)
            vnm.vnm_fp8_quantize(v, q, s)
            out.append((q, s))
    return out[0], out[1]


def gradients64(dy, x, wg, wu, G, U, act):
    a, s, d = act64(G, act), slope64(G, act), dy.double()
    return d * U * s, d * a, a * U


def check_gradients(dy, x, wg, wu, G, U, act, dx, dwg, dwu, h, dtype, base=0.0):
    """dG and dU are rounded to 16 bits (r of each, or half a subnormal's spacing) from fp32 products of
    functions good to 16 ulp of terms no larger than |dy U| (1 + |G|) and |dy| |G|; then K additions."""
    r, tiny = ROUND[dtype]
    x64, wg64, wu64, d = x.double(), wg.double(), wu.double(), dy.double()
    dG, dU, H = gradients64(dy, x, wg, wu, G, U, act)
    eG = r * dG.abs() + 16 * ULP * (d * U).abs() * (1 + G.abs()) + tiny
    eU = r * dU.abs() + 16 * ULP * d.abs() * G.abs() + tiny
    T, F = dy.shape

    def product(parts, n):
        want = sum(p @ q for p, _, q in parts)
        return want, sum(e @ q.abs() + (n + 20) * ULP * ((p.abs() + e) @ q.abs()) for p, e, q in parts)

    want, bound = product([(dG, eG, wg64), (dU, eU, wu64)], 2 * F)
    check(dx, want, bound, "dx")
    for got, p, e in ((dwg, dG, eG), (dwu, dU, eU)):
        want, bound = product([(p.t(), e.t(), x64)], T)
        check(got, want + base, bound + 2 * ULP * abs(base), "dw")
    check(h, H, 16 * ULP * (1 + G.abs()) * U.abs(), "h")


@pytest.mark.parametrize("dtype,act", [(F16, SILU), (BF16, GELU), (BF16, SILU), (F16, RELU)])
@pytest.mark.parametrize("keep", [None, E4M3, E5M2])
@pytest.mark.parametrize("T,F,K", [(1, 1, 1), (1, 300, 200), (7, 129, 65), (33, 257, 64), (100, 1000, 129), (300, 131, 520), (700, 520, 300)])
def test_backward(T, F, K, keep, dtype, act):
    g = generator(T, F, K, 8)
    x, wg, wu = (pitched(torch.randn(*s, generator=g, device=DEV).to(dtype)) for s in ((T, K), (F, K), (F, K)))
    dy = canvas(T, F, dtype, pad=1)[0]
    dy.copy_(torch.randn(T, F, generator=g, device=DEV))
    (a, sa), (b, sb) = checkpoint(g, T, F, keep, dtype)
    G, U = widened(a, sa), widened(b, sb)
    for out, accumulate in ((dtype, False), (F32, True)):
        dx, xbuf = canvas(T, K, dtype, pad=5)
        dwg, gbuf = canvas(F, K, out, pad=2)
        dwu, ubuf = canvas(F, K, out, pad=2)
        h, hbuf = canvas(T, F, dtype, pad=1)
        if accumulate:
            dwg.fill_(1.5), dwu.fill_(1.5)
        vnm.vnm_gated_linear_backward(dy, x, wg, wu, a, b, sa, sb, act=act, dx=dx, dwg=dwg, dwu=dwu, h=h, accumulate=accumulate)
        assert vnm.vnm_dense_get_status() == vnm.VNM_OK
        check_gradients(dy, x, wg, wu, G, U, act, dx, dwg, dwu, h, dtype, 1.5 if accumulate else 0.0)
        assert untouched(dx, xbuf) and untouched(dwg, gbuf) and untouched(dwu, ubuf) and untouched(h, hbuf)
    # each output alone gives the same bits, from the inputs that it needs alone
    e = [torch.empty_like(v) for v in (dx, dwg, dwu, h)]
    vnm.vnm_gated_linear_backward(dy, None, wg, wu, a, b, sa, sb, act=act, dx=e[0])
    e[1].fill_(1.5), e[2].fill_(1.5)
    vnm.vnm_gated_linear_backward(dy, x, None, None, a, b, sa, sb, act=act, dwg=e[1], dwu=e[2], accumulate=True)
    vnm.vnm_gated_linear_backward(None, None, None, None, a, b, sa, sb, act=act, h=e[3])
    for got, want in zip(e, (dx, dwg, dwu, h)):
        assert torch.equal(got, want)
    in_place = dy.clone()
    vnm.vnm_gated_linear_backward(in_place, None, wg, wu, a, b, sa, sb, act=act, dx=e[0], h=in_place)
    assert torch.equal(e[0], dx) and torch.equal(in_place, h)


def test_backward_without_tokens():
    w = torch.zeros((40, 16), dtype=F16, device=DEV)
    e = torch.empty((0, 40), dtype=F16, device=DEV)
    dwg, dwu = torch.full((40, 16), 3.0, device=DEV), torch.full((40, 16), 3.0, device=DEV)
    args = (e, torch.empty((0, 16), dtype=F16, device=DEV), w, w, e, e)
    vnm.vnm_gated_linear_backward(*args, dwg=dwg, dwu=dwu, accumulate=True, dx=torch.empty((0, 16), dtype=F16, device=DEV))
    assert (dwg == 3).all() and (dwu == 3).all()
    vnm.vnm_gated_linear_backward(*args, dwg=dwg, dwu=dwu)
    assert (dwg == 0).all() and (dwu == 0).all()


def test_backward_against_differences():
    """The gradients of sum(Y * D) along random directions, against central differences of the 64-bit form."""
    T, F, K = 50, 70, 60
    g = generator(9)
    x, wg, wu = (pitched((s * torch.randn(*n, generator=g, device=DEV)).to(F16)) for s, n in ((1, (T, K)), (0.2, (F, K)), (0.2, (F, K))))
    d = torch.randn(T, F, generator=g, device=DEV).half()
    Y, a, b = (torch.empty((T, F), dtype=F16, device=DEV) for _ in range(3))
    vnm.vnm_gated_linear(x, wg, wu, Y, act=SILU, g=a, u=b)
    dx, dwg, dwu = torch.empty((T, K), dtype=F16, device=DEV), torch.empty((F, K), device=DEV), torch.empty((F, K), device=DEV)
    vnm.vnm_gated_linear_backward(d, x, wg, wu, a, b, act=SILU, dx=dx, dwg=dwg, dwu=dwu)

    def loss(p, q, r):
        return (act64(p @ q.t(), SILU) * (p @ r.t()) * d.double()).sum()

    at = [x.double(), wg.double(), wu.double()]
    for i, grad in enumerate((dx, dwg, dwu)):
        way = torch.randn(at[i].shape, generator=g, device=DEV, dtype=torch.float64)
        step = [v.clone() for v in at]
        step[i] = at[i] + 1e-4 * way
        up = loss(*step)
        step[i] = at[i] - 1e-4 * way
        diff = (up - loss(*step)).item() / 2e-4
        # 16-bit roundings of g, u, dG, dU and dx, 2^-11 each at most, against the norms
        assert abs((grad.double() * way).sum().item() - diff) <= 6 * 2.0 ** -11 * (grad.double().norm() * way.norm()).item()


@pytest.mark.parametrize("T", [4, 40, 300])
def test_a_training_step_captured(T):
    """Forward with an 8-bit checkpoint, down projection onto the residual stream, and the backward pass, captured
    into a graph and replayed on new inputs: the same bits as the calls one by one."""
    D, F = 256, 520
    g = generator(T, 10)

    def step(x, res, dz, w, out):
        wg, wu, wd = w
        vnm.vnm_gated_linear(x, wg, wu, out["y"], g=out["g"], u=out["u"], g_scale=out["gs"], u_scale=out["us"])
        vnm.vnm_dense_linear(out["y"], wd, out["z"], residual=res)
        vnm.vnm_dense_linear(dz, wd.t(), out["dy"])
        vnm.vnm_gated_linear_backward(out["dy"], x, wg, wu, out["g"], out["u"], out["gs"], out["us"], dx=out["dx"], dwg=out["dwg"],
                                      dwu=out["dwu"], h=out["h"], workspace=out["ws"])
        vnm.vnm_dense_linear(dz.t(), out["h"].t(), out["dwd"])

    def outputs():
        n = dict(device=DEV, dtype=BF16)
        o = {k: torch.full(s, float("nan"), **n) for k, s in dict(y=(T, F), z=(T, D), dy=(T, F), dx=(T, D), dwg=(F, D), dwu=(F, D),
                                                                  h=(T, F), dwd=(D, F)).items()}
        o.update({k: torch.empty((T, F), dtype=E4M3, device=DEV) for k in "gu"}, gs=torch.empty((T, 5), device=DEV),
                 us=torch.empty((T, 5), device=DEV),
                 ws=torch.empty(vnm.vnm_gated_linear_backward_workspace_size(T, F), dtype=torch.uint8, device=DEV))
        return o

    w = [(0.05 * torch.randn(*s, generator=g, device=DEV)).bfloat16() for s in ((F, D), (F, D), (D, F))]
    ins = [[torch.randn(T, D, generator=g, device=DEV).bfloat16() for _ in range(3)] for _ in range(2)]
    eager = outputs()
    step(*ins[1], w, eager)
    captured, held = outputs(), [v.clone() for v in ins[0]]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(*held, w, captured)
    for h, v in zip(held, ins[1]):
        h.copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    for k in eager:
        if k != "ws":
            assert torch.equal(eager[k].view(torch.uint8), captured[k].view(torch.uint8)), k
    x, res, dz = (v.double() for v in ins[1])
    wg, wu, wd = (v.double() for v in w)
    y64 = act64(x @ wg.t(), SILU) * (x @ wu.t())

    def far(got, want):
        return ((got.double() - want).norm() / want.norm()).item()

    # roundings to bf16, 2^-8 at most each, and of the checkpoints to e4m3, 2^-4
    assert far(eager["z"], y64 @ wd.t() + res) < 2.0 ** -6
    assert far(eager["h"], y64) < 2.0 ** -3 and far(eager["dwd"], dz.t() @ y64) < 2.0 ** -3
    d = dz @ wd
    dG, dU = d * (x @ wu.t()) * slope64(x @ wg.t(), SILU), d * act64(x @ wg.t(), SILU)
    assert far(eager["dx"], dG @ wg + dU @ wu) < 2.0 ** -3
    assert far(eager["dwg"], dG.t() @ x) < 2.0 ** -3 and far(eager["dwu"], dU.t() @ x) < 2.0 ** -3


def test_refusals():
    T, F, K = 16, 40, 64
    x, w, Y = (torch.zeros(*s, dtype=F16, device=DEV) for s in ((T, K), (F, K), (T, F)))
    q, s = torch.zeros((T, F), dtype=torch.uint8, device=DEV).view(E4M3), torch.zeros((T, 1), device=DEV)
    f = vnm.vnm_gated_linear
    for bad in (lambda: f(x, w, w.bfloat16(), Y), lambda: f(x, w, w, Y.float()), lambda: f(x, w, w[:39], Y), lambda: f(x, w, w, Y, g=Y),
                lambda: f(x, w, w, Y, g=q, u=q), lambda: f(x, w, w, Y, g=q, u=q, g_scale=s), lambda: f(x, w, w, Y, act=-1),
                lambda: f(x, w, w, Y, g=q, u=q.view(torch.uint8).view(E5M2), g_scale=s, u_scale=s),
                lambda: f(x, w, w, Y, g=Y.float(), u=Y.float()), lambda: f(x, w, w, Y, g=Y.bfloat16(), u=Y.bfloat16()),
                lambda: f(x, w.t().contiguous().t(), w, Y), lambda: f(x, w, w, Y, g=q, u=q, g_scale=s, u_scale=s.double())):
        with pytest.raises((ValueError, vnm.VnmError)):
            bad()
    b = vnm.vnm_gated_linear_backward
    dw, ws = torch.zeros((F, K), dtype=F16, device=DEV), torch.zeros(4 * T * F - 1, dtype=torch.uint8, device=DEV)
    for bad in (lambda: b(Y, x, w, w, Y, None, dx=x), lambda: b(Y, x, w, w, Y, Y, dwg=dw), lambda: b(Y, x, w, w, Y, Y, dwg=dw, dwu=dw),
                lambda: b(Y, x, w, w, q, q, dx=x), lambda: b(None, x, w, w, Y, Y, dx=x), lambda: b(Y, None, w, w, Y, Y, dwg=dw, dwu=w),
                lambda: b(Y, x, None, w, Y, Y, dx=x), lambda: b(Y, x, w, w, Y, Y, dx=torch.zeros_like(x), workspace=ws),
                lambda: b(Y, x, w, w, Y, Y, dx=x.float()), lambda: b(Y, x, w, w, Y, Y, dx=torch.zeros_like(x), act=7),
                lambda: b(Y, x, w, w, Y, Y, dwg=dw, dwu=dw.float())):
        with pytest.raises((ValueError, vnm.VnmError)):
            bad()
    torch.cuda.synchronize()
