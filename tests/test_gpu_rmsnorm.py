"""RMS norm with the residual's addition and an 8-bit output, and its backward
pass, against plain 64-bit forms."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense_util import DEV, ROUND, check_quantized, groups, norm64, padded  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
EPS = 1e-6
# rstd: at most 64 fp32 additions one after another (and the warp and CTA
# trees) of squares, half of whose relative error reaches rstd, then a division, a
# sum, a root and a reciprocal
RSTD_REL = 2.0 ** -18
# y before its rounding: rstd and three products
Y_REL = RSTD_REL + 3 * 2.0 ** -24


def _inputs(T, D, dtype, seed, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def make(scale=1.0):
        t = padded(T, D, dtype, pad)
        t.copy_((scale * torch.randn(T, D, generator=g, device=DEV)).to(dtype))
        return t

    w = (1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(dtype)
    return make, w


def _check_forward(x, r, w, h, y, rstd, q, s, eps=EPS):
    want_h, want_r, want_y = norm64(x, r, w, eps, x.dtype)
    if h is not None:
        assert torch.equal(h, want_h)
    if rstd is not None:
        assert ((rstd.double() - want_r).abs() <= RSTD_REL * want_r).all()
    if y is not None:
        u, tiny = ROUND[x.dtype]
        assert ((y.double() - want_y).abs() <= (u + 2 * Y_REL) * want_y.abs() + tiny).all()
    if q is not None:
        check_quantized(q, s, want_y, 1, Y_REL)


# one token to many; widths under a group, odd, one over a group, of the workloads, and longer than the registers hold
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("T,D", [(1, 1), (1, 4096), (3, 127), (5, 129), (2, 1001), (700, 128), (700, 520), (401, 4096),
                                 (33, 11008), (330, 12288), (2, 16388), (3, 40001)])
def test_forward(T, D, dtype):
    make, w = _inputs(T, D, dtype, T + D)
    x, r = make(), make()
    h, y = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(T, device=DEV)
    q, s = torch.empty((T, D), dtype=torch.float8_e4m3fn, device=DEV), torch.empty((T, groups(D)), device=DEV)
    vnm.vnm_rmsnorm(x, w, EPS, residual=r, h=h, y=y, rstd=rstd, q=q, q_scale=s)
    _check_forward(x, r, w, h, y, rstd, q, s)


@pytest.mark.parametrize("outputs,residual", [(o, r) for o in ("y", "q", "y rstd", "q rstd", "h q", "h y", "y q")
                                              for r in (True, False) if r or "h" not in o])
@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("D", [384, 1003])
def test_outputs_are_independent(outputs, residual, weight, D):
    T, dtype = 17, F16
    make, w = _inputs(T, D, dtype, 3)
    x, r = make(), make() if residual else None
    w = w if weight else None
    h = torch.empty_like(x) if "h" in outputs else None
    y = torch.empty_like(x) if "y" in outputs else None
    rstd = torch.empty(T, device=DEV) if "rstd" in outputs else None
    q = torch.empty((T, D), dtype=torch.float8_e5m2, device=DEV) if "q" in outputs else None
    s = torch.empty((T, groups(D)), device=DEV) if "q" in outputs else None
    vnm.vnm_rmsnorm(x, w, EPS, residual=r, h=h, y=y, rstd=rstd, q=q, q_scale=s)
    _check_forward(x, r, w, h, y, rstd, q, s)


# row strides that allow vector accesses and that do not, scales in either order, a start off the alignment
@pytest.mark.parametrize("D,pad,off", [(512, 8, 0), (512, 3, 0), (512, 4, 1), (516, 0, 0), (100, 28, 2)])
@pytest.mark.parametrize("by_group", [False, True])
def test_strides_and_canaries(D, pad, off, by_group):
    T, dtype = 6, BF16
    make, w = _inputs(T, D, dtype, 5, pad)
    x, r = make(), make()
    big = {}

    def out(t, fill):
        buf = torch.full((T + 2, D + pad + off), fill, dtype=t, device=DEV)
        big[len(big)] = (buf, fill)
        return buf[1:T + 1, off:off + D]

    h, y = out(dtype, 7.0), out(dtype, 7.0)
    raw = torch.full((T + 2, D + pad + off), 0x55, dtype=torch.uint8, device=DEV)
    q = raw.view(torch.float8_e4m3fn)[1:T + 1, off:off + D]
    s = torch.empty((groups(D), T), device=DEV).t() if by_group else torch.empty((T, groups(D)), device=DEV)
    vnm.vnm_rmsnorm(x, w, EPS, residual=r, h=h, y=y, q=q, q_scale=s)
    _check_forward(x, r, w, h, y, None, q, s)
    for buf, fill in big.values():
        buf[1:T + 1, off:off + D] = fill
        assert (buf == fill).all()
    raw[1:T + 1, off:off + D] = 0x55
    assert (raw == 0x55).all()


@pytest.mark.parametrize("D", [256, 1001, 33000])
@pytest.mark.parametrize("which", ["h is residual", "h is x", "y is x", "h is residual, y is x"])
def test_in_place(D, which):
    T, dtype = 5, F16
    make, w = _inputs(T, D, dtype, 9)
    x, r = make(), make()
    x0, r0 = x.clone(), r.clone()
    h = r if "h is residual" in which else x if "h is x" in which else None
    y = x if "y is x" in which else torch.empty_like(x)
    vnm.vnm_rmsnorm(x, w, EPS, residual=r, h=h, y=y)
    _check_forward(x0, r0, w, h, y, None, None, None)


def test_zero_rows_and_non_finite_rows():
    T, D = 6, 300
    make, w = _inputs(T, D, F32, 11)
    x = make()
    x[0] = 0.0
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    x[4] = 1e-30
    y, rstd = torch.empty_like(x), torch.empty(T, device=DEV)
    q, s = torch.empty((T, D), dtype=torch.float8_e4m3fn, device=DEV), torch.empty((T, groups(D)), device=DEV)
    vnm.vnm_rmsnorm(x, w, EPS, y=y, rstd=rstd, q=q, q_scale=s)
    keep = [0, 1, 4, 5]
    _check_forward(x[keep], None, w, None, y[keep], rstd[keep], q[keep], s[keep])
    assert (y[0] == 0).all() and (s[0] == 2.0 ** -100).all() and (q[0].float() == 0).all()
    assert y[2].isnan().all() and rstd[2].isnan() and s[2].isnan().all() and q[2].float().isnan().all()
    # an Inf: its reciprocal root is 0, so its own place is NaN and the others 0
    assert rstd[3] == 0 and y[3, 200].isnan() and (y[3, :200] == 0).all()
    assert s[3, 1].isnan() and q[3, 128:256].float().isnan().all() and (q[3, :128].float() == 0).all()


def test_eps_zero_and_constant_rows():
    x = torch.full((2, 640), 3.0, dtype=F16, device=DEV)
    y = torch.empty_like(x)
    vnm.vnm_rmsnorm(x, None, 0.0, y=y)
    assert (y == 1.0).all()


def test_empty_sizes():
    w = torch.ones(64, dtype=F16, device=DEV)
    x = torch.empty((0, 64), dtype=F16, device=DEV)
    vnm.vnm_rmsnorm(x, w, EPS, y=torch.empty_like(x))
    dw = torch.full((64,), 5.0, device=DEV)
    vnm.vnm_rmsnorm_backward(x, x, w, torch.empty(0, device=DEV), torch.empty_like(x), dw)
    assert (dw == 0).all()


def test_other_stream():
    make, w = _inputs(64, 4096, BF16, 13)
    x, y = make(), torch.empty((64, 4096), dtype=BF16, device=DEV)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    vnm.vnm_rmsnorm(x, w, EPS, y=y, stream=st)
    st.synchronize()
    _check_forward(x, None, w, None, y, None, None, None)


# ------------------------------------------------------------------ backward


def _check_backward(dy, h, w, rstd, dres, dh, dw):
    d, hd, r = dy.double(), h.double(), rstd.double()[:, None]
    g = d if w is None else d * w.double()
    D, T = dy.shape[1], dy.shape[0]
    c = r.square() * (g * hd).mean(1, keepdim=True)
    want = r * (g - hd * c)
    # the mean's sum as RSTD_REL's, and six fp32 operations
    size = r * (g.abs() + hd.abs() * r.square() * (g * hd).abs().mean(1, keepdim=True))
    if dres is not None:
        want, size = want + dres.double(), size + dres.double().abs()
    u, tiny = ROUND[dy.dtype]
    if dh is not None:
        bound = 2.0 ** -17 * size
        assert ((dh.double() - want).abs() <= bound + u * (want.abs() + bound) + tiny).all()
    if dw is not None:
        terms = d * hd * r
        # every row added in fp32 in the worst case, one after another
        assert ((dw.double() - terms.sum(0)).abs() <= (T + 16) * 2.0 ** -24 * terms.abs().sum(0)).all()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("T,D", [(1, 1), (1, 4096), (3, 127), (700, 129), (5, 1001), (700, 128), (401, 4096), (320, 6000),
                                 (33, 11008), (2, 16388), (305, 20001)])
@pytest.mark.parametrize("residual", [True, False])
def test_backward(T, D, dtype, residual):
    make, w = _inputs(T, D, dtype, 17 + T + D)
    h, dy, dres = make(), make(), make() if residual else None
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    dh, dw = torch.empty_like(h), torch.full((D,), float("nan"), device=DEV)
    vnm.vnm_rmsnorm_backward(dy, h, w, rstd, dh, dw, dresidual=dres)
    _check_backward(dy, h, w, rstd, dres, dh, dw)
    again = torch.empty_like(dw)
    vnm.vnm_rmsnorm_backward(dy, h, w, rstd, None, again)
    assert torch.equal(dw, again)


@pytest.mark.parametrize("D", [260, 1001, 20000])
@pytest.mark.parametrize("which", ["dh is dy", "dh is dresidual", "no weight", "no dweight"])
def test_backward_in_place_and_optional(D, which):
    T, dtype = 7, F32
    make, w = _inputs(T, D, dtype, 19)
    h, dy, dres = make(), make(), make()
    w = None if which == "no weight" else w
    dy0, dres0 = dy.clone(), dres.clone()
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    dh = dy if which == "dh is dy" else dres if which == "dh is dresidual" else torch.empty_like(h)
    dw = None if which == "no dweight" else torch.empty(D, device=DEV)
    vnm.vnm_rmsnorm_backward(dy, h, w, rstd, dh, dw, dresidual=dres)
    _check_backward(dy0, h, w, rstd, dres0, dh, dw)


def test_backward_strides():
    T, D = 9, 250
    make, w = _inputs(T, D, F16, 23, pad=5)
    h, dy, dres = make(), make(), make()
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    buf = torch.full((T + 2, D + 5), 7.0, dtype=F16, device=DEV)
    dh, dw = buf[1:T + 1, :D], torch.empty(D, device=DEV)
    vnm.vnm_rmsnorm_backward(dy, h, w, rstd, dh, dw, dresidual=dres)
    _check_backward(dy, h, w, rstd, dres, dh, dw)
    buf[1:T + 1, :D] = 7.0
    assert (buf == 7.0).all()


def test_backward_against_differences():
    """dh and dw against central differences of the plain 64-bit norm: with step
    1e-4 of values of order 1 their error is below 1e-6 of the gradients' size."""
    T, D, eps = 2, 24, 1e-3
    g = torch.Generator(device=DEV).manual_seed(29)
    h, dy, w = (torch.randn(n, generator=g, device=DEV, dtype=F32) for n in ((T, D), (T, D), (D,)))
    y, rstd = torch.empty_like(h), torch.empty(T, device=DEV)
    vnm.vnm_rmsnorm(h, w, eps, y=y, rstd=rstd)
    dh, dw = torch.empty_like(h), torch.empty(D, device=DEV)
    vnm.vnm_rmsnorm_backward(dy, h, w, rstd, dh, dw)

    def loss(h64, w64):
        return (dy.double() * h64 / torch.sqrt(h64.square().mean(1, keepdim=True) + eps) * w64).sum()

    step, h64, w64 = 1e-4, h.double(), w.double()
    for t in range(T):
        for d in range(D):
            e = torch.zeros_like(h64)
            e[t, d] = step
            num = (loss(h64 + e, w64) - loss(h64 - e, w64)) / (2 * step)
            assert abs(dh[t, d].item() - num.item()) < 1e-4
    for d in range(D):
        e = torch.zeros_like(w64)
        e[d] = step
        num = (loss(h64, w64 + e) - loss(h64, w64 - e)) / (2 * step)
        assert abs(dw[d].item() - num.item()) < 1e-4


def test_binding_refusals():
    x = torch.zeros((4, 64), dtype=F16, device=DEV)
    w = torch.ones(64, dtype=F16, device=DEV)
    y, q, s = torch.empty_like(x), torch.empty((4, 64), dtype=torch.float8_e4m3fn, device=DEV), torch.empty((4, 1), device=DEV)
    for kw in (dict(y=y[:3]), dict(y=y.float()), dict(y=torch.empty((4, 64), dtype=F16)), dict(y=y, rstd=torch.empty(3, device=DEV)),
               dict(q=y, q_scale=s), dict(q=q, q_scale=s[:3]), dict(y=y.t().contiguous().t())):
        with pytest.raises(ValueError):
            vnm.vnm_rmsnorm(x, w, EPS, **kw)
    with pytest.raises(ValueError):
        vnm.vnm_rmsnorm(x, w[:63], EPS, y=y)
    with pytest.raises(ValueError):
        vnm.vnm_rmsnorm(x.to(torch.float64), w, EPS, y=y)
    for kw in (dict(), dict(y=y, h=y), dict(q=q), dict(y=y, q_scale=s)):
        with pytest.raises(vnm.VnmError) as e:
            vnm.vnm_rmsnorm(x, w, EPS, **kw)
        assert e.value.code == vnm.VNM_ERR_INVALID_ARG
    with pytest.raises(vnm.VnmError):
        vnm.vnm_rmsnorm(x, w, -1.0, y=y)
    with pytest.raises(vnm.VnmError) as e:
        vnm.vnm_rmsnorm_backward(x, x, w, torch.ones(4, device=DEV), None, torch.empty(64, device=DEV),
                                 workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.code == vnm.VNM_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        vnm.vnm_rmsnorm_backward(x, x, w, torch.ones(4, device=DEV), None, torch.empty(64, device=DEV),
                                 workspace=torch.empty(1 << 20, dtype=torch.uint8))


def test_overlapping_rows_are_refused():
    """An expanded tensor's rows have stride 0: no leading dimension describes them."""
    T, D = 4, 64
    w = torch.ones(D, dtype=F16, device=DEV)
    x, y, rstd, dw = torch.zeros((T, D), dtype=F16, device=DEV), torch.empty((T, D), dtype=F16, device=DEV), \
        torch.ones(T, device=DEV), torch.empty(D, device=DEV)
    wide, one = w.expand(T, D), torch.zeros((1, 1), dtype=F16, device=DEV).expand(T, 1)
    for kw in (dict(x=wide, y=y), dict(x=x, residual=wide, y=y), dict(x=x, y=wide)):
        with pytest.raises(ValueError):
            vnm.vnm_rmsnorm(kw.pop("x"), w, EPS, **kw)
    with pytest.raises(ValueError):
        vnm.vnm_rmsnorm(one, w[:1], EPS, y=torch.empty_like(one.contiguous()))
    with pytest.raises(ValueError):
        vnm.vnm_rmsnorm_backward(wide, x, w, rstd, y, dw)
    with pytest.raises(ValueError):
        vnm.vnm_rmsnorm_backward(x, x, w, rstd, y, dw,
                                 workspace=torch.empty(1, dtype=torch.uint8, device=DEV).expand(1 << 20))
    vnm.vnm_rmsnorm(wide[:1], w, EPS, y=y[:1])  # one row: any stride
    assert (y[0].double() - 1).abs().max() < 2e-3
