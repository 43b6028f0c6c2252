"""The few-token kernel of the dense 16-bit layers, bit for bit on whole numbers: every length of the last block of K, every
number of warps, one and two groups of tokens, operands that end where their memory ends."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense16_util import BF16, DEV, F16, F32, NONE, generator, whole  # noqa: E402


def tight(x, pitch):
    """x in rows of ``pitch`` elements that start on 16 bytes, NaN between them, and nothing behind the last one."""
    R, C = x.shape
    buf = torch.full(((R - 1) * pitch + C,), float("nan"), dtype=x.dtype, device=DEV)
    out = buf.as_strided((R, C), (pitch, 1))
    out.copy_(x)
    return out


def forward(T, R, K, dtype, gated):
    g = generator(T, R, K, 31)
    up = -(-K // 8) * 8
    x, w = tight(whole(g, T, K, dtype, 1), up + 8), tight(whole(g, R, K, dtype, 1), up)
    want = x.double() @ w.double().t()
    assert vnm.vnm_testing_dense_plan(3 if gated else 0, T, R, K, 152)[0] == 8
    if gated:
        wu = tight(whole(g, R, K, dtype, 1, 0.5), up + 16)
        U = x.double() @ wu.double().t()
        Y, a, b = (torch.full((T, R), float("nan"), dtype=dtype, device=DEV) for _ in range(3))
        vnm.vnm_gated_linear(x, w, wu, Y, act=NONE, g=a, u=b)
        assert torch.equal(a, want.to(dtype)) and torch.equal(b, U.to(dtype)) and torch.equal(Y, (want * U).float().to(dtype)), (T, R, K)
    else:
        for out in (dtype, F32):
            Y = torch.full((T, R), float("nan"), dtype=out, device=DEV)
            vnm.vnm_dense_linear(x, w, Y)
            assert torch.equal(Y, want.float().to(out)), (T, R, K, out)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T", [1, 5, 16])
def test_every_last_block(T, gated):
    for K in list(range(1, 70)) + list(range(1024, 1024 + 65)):
        forward(T, 35, K, BF16, gated)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T", [1, 2, 8, 9, 13, 16])
@pytest.mark.parametrize("R,K", [(1, 2048), (35, 2111), (2431, 2050), (2432, 2560), (300, 2047), (2433, 700), (4863, 1030), (4865, 640), (9001, 203)])
def test_every_number_of_warps(T, R, K, dtype, gated):
    if T > 8 and R > (2432 if gated else 4864):
        pytest.skip("the narrow tiles' size")
    forward(T, R, K, dtype, gated)


@pytest.mark.parametrize("T,R,K", [(1, 200, 20000), (8, 100, 11001), (16, 600, 9000)])
def test_long_rows(T, R, K):
    forward(T, R, K, F16, False)
    if T <= 8:
        forward(T, R, K, F16, True)


def test_nan_and_infinity_stay_in_their_rows():
    """In the last block too, where the loads are of pieces."""
    T, R, K = 8, 40, 2101
    g = generator(32)
    x, w = whole(g, T, K, F16, 1), whole(g, R, K, F16, 1)
    want = x.double() @ w.double().t()
    x[7, K - 1], w[5, K - 2], w[6, 3] = float("nan"), float("inf"), float("nan")
    up = -(-K // 8) * 8
    Y = torch.empty((T, R), dtype=F16, device=DEV)
    vnm.vnm_dense_linear(tight(x, up), tight(w, up), Y)
    clean = torch.ones(R, dtype=torch.bool, device=DEV)
    clean[5] = clean[6] = False
    assert Y[7].isnan().all() and Y[:, 6].isnan().all() and not torch.isfinite(Y[:, 5]).any()
    assert torch.equal(Y[:7][:, clean], want[:7][:, clean].half())
