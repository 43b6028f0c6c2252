"""Inputs, plain 64-bit forms and error bounds of the dense 16-bit layers.

Most tests use small whole numbers (times a power of two): every sum is then exact in
fp32 whatever its order and however it truncates, and the results are compared bit for bit
up to the one rounding of the output. With real numbers, products of 16-bit operands are
exact in fp32, and each of the K additions of a sum may truncate, 2^-23 of the products'
magnitudes (``mag``); a split or a chunk adds a few more."""
import math

import torch

DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
# unit roundoff, and half the spacing of the subnormals
ROUND = {F16: (2.0 ** -11, 2.0 ** -25), BF16: (2.0 ** -8, 2.0 ** -134), F32: (2.0 ** -24, 2.0 ** -150)}
ULP = 2.0 ** -23
NONE, RELU, GELU, SILU = 0, 1, 2, 3


def generator(*key):
    return torch.Generator(device=DEV).manual_seed(hash(key) % (1 << 31))


def pitched(x, pad=0, fill=float("nan")):
    """x with rows of a multiple of 8 elements plus ``pad`` (a multiple of 8), NaN in the padding."""
    R, C = x.shape
    buf = torch.full((R, -(-max(C, 1) // 8) * 8 + pad), fill, dtype=x.dtype, device=x.device)
    buf[:, :C] = x
    return buf[:, :C]


def whole(g, rows, cols, dtype, top=3, unit=1.0):
    return (torch.randint(-top, top + 1, (rows, cols), generator=g, device=DEV) * unit).to(dtype)


def operand(x, transposed, pad=0):
    """x, in rows that start on 16 bytes; transposed: a view of its transpose stored so."""
    return pitched(x.t().contiguous(), pad).t() if transposed else pitched(x, pad)


def canvas(rows, cols, dtype, pad=0, offset=0):
    """A rows x cols output inside a buffer of NaN: (view, buffer). ``offset``: elements before it."""
    buf = torch.full((rows * (cols + pad) + offset + 16,), float("nan"), dtype=dtype, device=DEV)
    return buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], buf


def untouched(view, buf):
    """Whether nothing of the buffer outside the view has been written."""
    outside = torch.ones(buf.numel(), dtype=torch.bool, device=DEV)
    start = view.storage_offset()
    r = torch.arange(view.shape[0], device=DEV)[:, None] * view.stride(0) + torch.arange(view.shape[1], device=DEV) + start
    outside[r.reshape(-1)] = False
    return bool(buf[outside].isnan().all()) if buf.is_floating_point() else True


def act64(z, act):
    if act == RELU:
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == GELU:
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    return z * torch.sigmoid(z) if act == SILU else z


def slope64(z, act):
    if act == RELU:
        return (z > 0).double()
    if act == GELU:
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == SILU:
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def act_bound(z, act):
    """Error of the kernels' activation of an exact z: GELU within 1.5 * 2^-23 |z|; SiLU's expf (2
    ulp), sum, quotient (2 ulp) and product stay within 8 * 2^-23 |z|."""
    return (8 * ULP if act in (GELU, SILU) else 0.0) * z.abs()


def check(got, want, bound, what=""):
    """|got - want| <= bound (of the unrounded value) plus one rounding to got's type."""
    r, tiny = ROUND[got.dtype]
    total = bound + r * (want.abs() + bound) + tiny
    off = (got.double() - want).abs()
    assert torch.isfinite(got.float()).all(), what
    assert (off <= total).all(), f"{what}: worst {(off - total).max().item()}, {(off > total).sum().item()} of {off.numel()}"


def widened(q, s):
    """The values that an 8-bit checkpoint stands for (16-bit ones as they are), in 64 bits; each the fp32 product."""
    if s is None:
        return q.double()
    return (q.float() * s.repeat_interleave(128, 1)[:, : q.shape[1]]).double()
