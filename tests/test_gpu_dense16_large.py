"""Outputs, checkpoints and workspaces of more than 2^31 elements, or whose rows lie more than 2^32 bytes apart in all: rows from both ends
and the middle against 64-bit forms on whole numbers."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense16_util import BF16, DEV, F32, NONE, RELU, generator, pitched, whole  # noqa: E402

T, R, K = 70003, 40008, 72


def rows_of(T):
    return torch.cat([torch.arange(0, 40), torch.arange(T // 2, T // 2 + 40), torch.arange(T - 300, T)]).to(DEV)


def free():
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


# (rows that start and end on 16 bytes; that do not; few rows far apart)
@pytest.mark.parametrize("out,rows,cols,ld", [(BF16, T, R, R), (BF16, T, R - 3, R - 3), (F32, T, R, R), (F32, T, R - 3, R - 3), (BF16, 16, 4096, 1 << 28),
                                              (F32, 40, 300, 1 << 27), (BF16, 700, 1500, 1 << 23)])
def test_products(out, rows, cols, ld):
    g = generator(rows, cols, 81)
    x, w = pitched(whole(g, rows, K, BF16)), pitched(whole(g, cols, K, BF16))
    buf = torch.empty(((rows - 1) * ld + cols,), dtype=out, device=DEV)
    Y = buf.as_strided((rows, cols), (ld, 1))
    Y.fill_(2)
    vnm.vnm_dense_linear(x, w, Y, residual=Y, act=RELU)
    at = rows_of(rows) if rows > 400 else torch.arange(rows, device=DEV)
    assert torch.equal(Y[at].double(), ((x[at].double() @ w.double().t()).clamp_min(0) + 2).to(out).double())
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK
    del Y, buf
    free()


@pytest.mark.parametrize("F", [R, R - 3])
def test_gated_pair_and_its_gradients(F):
    g = generator(F, 82)
    x, wg, wu = pitched(whole(g, T, K, BF16, 1)), pitched(whole(g, F, K, BF16, 1)), pitched(whole(g, F, K, BF16, 1))
    at = rows_of(T)
    G, U = x[at].double() @ wg.double().t(), x[at].double() @ wu.double().t()
    Y, a, b = (torch.empty((T, F), dtype=BF16, device=DEV) for _ in range(3))
    vnm.vnm_gated_linear(x, wg, wu, Y, act=NONE, g=a, u=b)
    assert torch.equal(a[at].double(), G) and torch.equal(b[at].double(), U) and torch.equal(Y[at], (G * U).bfloat16())
    del Y
    q = [torch.empty((T, F), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    s = [torch.empty((T, -(-F // 128)), device=DEV) for _ in range(2)]
    Y = torch.empty((T, F), dtype=BF16, device=DEV)
    vnm.vnm_gated_linear(x, wg, wu, Y, act=NONE, g=q[0], u=q[1], g_scale=s[0], u_scale=s[1])
    for v, p, want in ((q[0], s[0], G), (q[1], s[1], U)):  # (half a spacing of e4m3, of the scale's rounding a part)
        kept = v[at].double() * p[at].double().repeat_interleave(128, 1)[:, :F]
        top = p[at].double().repeat_interleave(128, 1)[:, :F] * 448
        assert ((kept - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -9 * top).all()
    del q, s
    free()
    # dY = 1 in a few rows and columns only: the gradients are sums that 64 bits can follow
    Y.zero_()
    Y[at] = 1
    dx, h = torch.empty((T, K), dtype=BF16, device=DEV), torch.empty((T, F), dtype=BF16, device=DEV)
    dwg, dwu = (torch.empty((F, K), dtype=F32, device=DEV) for _ in range(2))
    vnm.vnm_gated_linear_backward(Y, x, wg, wu, a, b, act=NONE, dx=dx, dwg=dwg, dwu=dwu, h=h)
    assert torch.equal(dwg.double(), U.t() @ x[at].double()) and torch.equal(dwu.double(), G.t() @ x[at].double())
    assert torch.equal(dx[at], (U @ wg.double() + G @ wu.double()).float().bfloat16())
    assert torch.equal(h[at], (G * U).bfloat16())
    untouched = torch.ones(T, dtype=torch.bool, device=DEV)
    untouched[at] = False
    assert (dx[untouched] == 0).all()
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK
    del Y, a, b, dx, h, dwg, dwu
    free()
