"""GELU of the 8-bit Linear layer, element by element against 64 bits: with operands of
zeros its argument is the bias itself."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense_util import DEV, groups  # noqa: E402

# In units of 2^-23 |z|: erff to 2 ulp and the sum 1 + erf, halved, 0.75; the argument's two
# roundings, half of erf's largest z erf'(z), 0.25; the last product 0.5.
REL = 1.5 * 2.0 ** -23


def _check(Y, z):
    want = z.double() * 0.5 * torch.erfc(-z.double() / 2.0 ** 0.5)
    off = (Y.double() - want).abs()
    worst = (off / z.double().abs().clamp_min(2.0 ** -126)).max().item()
    assert (off <= REL * z.double().abs() + 2.0 ** -149).all(), f"worst {worst:.3e} |z|"


def _run(T, R, K, bias, rows=128):
    e4m3 = torch.float8_e4m3fn
    q = [torch.zeros((n, K), dtype=torch.uint8, device=DEV).view(e4m3) for n in (T, R)]
    xs, ws = torch.ones((T, groups(K)), device=DEV), torch.ones((-(-R // rows), groups(K)), device=DEV)
    Y = torch.full((T, R), float("nan"), device=DEV)
    vnm.vnm_fp8_linear(q[0], xs, q[1], ws, Y, bias=bias, act=vnm.VNM_ACT_GELU)
    return Y


@pytest.mark.parametrize("lo,hi", [(-6.0, 6.0), (-0.5, 0.5), (-16.0, -4.0), (-1e-3, 1e-3)])
def test_sweep(lo, hi):
    z = torch.linspace(lo, hi, 1 << 20, device=DEV)
    _check(_run(1, z.numel(), 0, z), z[None])


# the kernel of a few tokens, tiles with W on the rows' side, pairs with one scale a block and with one a row
@pytest.mark.parametrize("T,R,rows", [(1, 4000, 128), (8, 4000, 1), (40, 4000, 128), (200, 4096, 128), (2500, 2000, 128),
                                      (2500, 2000, 1)])
def test_every_kernel(T, R, rows):
    g = torch.Generator(device=DEV).manual_seed(T)
    z = torch.empty(R, device=DEV).uniform_(-6.0, 6.0, generator=g)
    _check(_run(T, R, 128, z, rows), z.expand(T, R))


def test_the_ends_of_the_range():
    z = torch.tensor([0.0, -0.0, 1e30, 3e38, -1e30, 1e-38, -1e-38, 1e-45, float("inf"), float("nan"), -100.0], device=DEV)
    for Y in (_run(1, z.numel(), 0, z)[0], _run(3, z.numel(), 128, z)[2]):
        assert Y[:2].tolist() == [0.0, 0.0] and torch.equal(Y[2:4], z[2:4]) and Y[4] == 0.0 and Y[8] == float("inf")
        assert Y[9].isnan() and Y[10] == 0.0
        assert ((Y[5:8] - 0.5 * z[5:8]).abs() <= 2.0 ** -149).all()
