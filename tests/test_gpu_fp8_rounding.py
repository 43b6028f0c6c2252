"""The 8-bit values are the fp8 nearest to the fp32 quotient of an element and its
group's scale, near the middle between two fp8 values too: bit for bit."""
import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense_util import DEV, FP8_MAX, groups  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def _nearest(x, s, rows, fp8):
    """fp8 bytes of x / s by a division and a conversion, s one scale for each rows x 128 block."""
    R, C = x.shape
    each = s.repeat_interleave(rows, 0)[:R].repeat_interleave(128, 1)[:, :C]
    top = FP8_MAX[fp8]
    return (x.float() / each).clamp(-top, top).to(fp8).view(torch.uint8)


def _randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


def _near_ties(R, C, fp8, seed):
    """Elements within three fp32 steps of the middle between two fp8 values of their group,
    whose largest element and scale vary."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.zeros((R, groups(C) * 128), device=DEV)
    m = torch.exp(torch.empty((R, groups(C)), device=DEV).uniform_(-20.0, 20.0, generator=g))
    s = m * (1.0 / FP8_MAX[fp8])
    bits = 3 if fp8 == E4M3 else 2
    e = torch.randint(-5, 8, x.shape, generator=g, device=DEV).float()
    k = torch.randint(2 ** bits, 2 ** (bits + 1), x.shape, generator=g, device=DEV).float()
    mid = (2 * k + 1) * torch.exp2(e - bits - 1)  # at most 15.5 * 2^4 < 448
    x = (mid * s.repeat_interleave(128, 1))
    step = torch.randint(-3, 4, x.shape, generator=g, device=DEV, dtype=torch.int32)
    x = (x.view(torch.int32) + step).view(F32)
    x *= torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    x.view(R, -1, 128)[:, :, 17] = m
    return x[:, :C].contiguous()


@pytest.mark.parametrize("fp8", [E4M3, E5M2])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("R,C", [(512, 1024), (130, 333)])
def test_quantize(R, C, dtype, rows, fp8):
    x = (_randn(R, C, seed=R) * torch.exp(2 * _randn(R, 1, seed=1))).to(dtype)
    x[0, :7] = -0.0
    q, qt = torch.empty((R, C), dtype=fp8, device=DEV), torch.empty((C, R), dtype=fp8, device=DEV)
    s, st = torch.empty((-(-R // rows), groups(C)), device=DEV), torch.empty((-(-C // rows), groups(R)), device=DEV)
    vnm.vnm_fp8_quantize(x, q, s, qt, st, block_rows=rows)
    assert torch.equal(q.view(torch.uint8), _nearest(x, s, rows, fp8))
    assert torch.equal(qt.view(torch.uint8), _nearest(x.t(), st, rows, fp8))


@pytest.mark.parametrize("fp8", [E4M3, E5M2])
@pytest.mark.parametrize("transposed", [False, True])
def test_quantize_near_the_middle_between_two_values(transposed, fp8):
    x = _near_ties(256, 512, fp8, seed=2)
    if transposed:
        q, s = torch.empty((256, 512), dtype=fp8, device=DEV), torch.empty((256, 4), device=DEV)
        vnm.vnm_fp8_quantize(x.t().contiguous(), qt=q, st=s)
    else:
        q, s = torch.empty((256, 512), dtype=fp8, device=DEV), torch.empty((256, 4), device=DEV)
        vnm.vnm_fp8_quantize(x, q, s)
    assert torch.equal(q.view(torch.uint8), _nearest(x, s, 1, fp8))


@pytest.mark.parametrize("fp8", [E4M3, E5M2])
@pytest.mark.parametrize("T,D", [(700, 1024), (33, 1001), (5, 12288), (3, 20000)])
def test_norm(T, D, fp8):
    """In 32 bits y is the value that the 8-bit form is made of."""
    x, w = _randn(T, D, seed=T), 1 + 0.2 * _randn(D, seed=3)
    y, q, s = torch.empty_like(x), torch.empty((T, D), dtype=fp8, device=DEV), torch.empty((T, groups(D)), device=DEV)
    vnm.vnm_rmsnorm(x, w, 1e-6, y=y, q=q, q_scale=s)
    assert torch.equal(q.view(torch.uint8), _nearest(y, s, 1, fp8))
