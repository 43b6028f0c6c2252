"""Plain 64-bit forms of the norm, the 8-bit quantiser and the 8-bit Linear
layer, and the error bounds the kernels are held to."""
import torch

DEV = "cuda"
GROUP = 128
FP8_MAX = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
# (mantissa bits, exponent of the smallest normal value)
FP8_SHAPE = {torch.float8_e4m3fn: (3, -6), torch.float8_e5m2: (2, -14)}
# unit roundoff, and half the spacing of the subnormals
ROUND = {torch.float16: (2.0 ** -11, 2.0 ** -25), torch.bfloat16: (2.0 ** -8, 2.0 ** -134),
         torch.float32: (2.0 ** -24, 2.0 ** -150)}


def groups(n):
    return -(-n // GROUP)


def padded(rows, cols, dtype, pad=0, fill=0):
    """A rows x cols matrix whose rows are `pad` elements further apart."""
    return torch.full((rows, cols + pad), fill, dtype=dtype, device=DEV)[:, :cols]


def scale64(x, rows, fp8):
    """The definition's scales in 64 bits."""
    R, C = x.shape
    b = torch.nn.functional.pad(x.double(), (0, -C % GROUP, 0, -R % rows))
    b = b.view(b.shape[0] // rows, rows, -1, GROUP).abs()
    m = b.amax((1, 3))
    m = torch.where(torch.isfinite(b).all(3).all(1), m, torch.full_like(m, float("nan")))
    return torch.where(m.isnan(), m, (m / FP8_MAX[fp8]).clamp_min(2.0 ** -100))


def spread(s, rows, shape):
    """One scale an element."""
    return s.double().repeat_interleave(rows, 0)[: shape[0]].repeat_interleave(GROUP, 1)[:, : shape[1]]


def check_quantized(q, s, x, rows, rel, what=""):
    """q, s against the 8-bit form of x (64 bits), whose own relative error is at
    most `rel`. The scale is one rounded division: rel + 2^-23. An element is
    the nearest fp8 value to a number that is off by at most rel + 2^-22 (the
    scale, the reciprocal, the product): half a spacing at its magnitude, plus that."""
    want = scale64(x, rows, q.dtype)
    bad = want.isnan()
    assert torch.equal(bad, s.isnan()), what
    # the floor 2^-100 is exact; relative errors elsewhere
    assert ((s.double() - want).abs()[~bad] <= (rel + 2.0 ** -23) * want[~bad]).all(), what
    nan = spread(bad.double(), rows, x.shape) > 0
    qf = q.float().double()
    assert torch.equal(qf.isnan(), nan), what
    v = torch.where(nan, torch.zeros_like(qf), x.double() / spread(torch.where(bad, torch.ones_like(want), want), rows, x.shape))
    bits, emin = FP8_SHAPE[q.dtype]
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -1000))).clamp_min(emin)
    half = 0.5 * 2.0 ** (e - bits)
    off = torch.where(nan, torch.zeros_like(qf), (qf - v).abs())
    bound = half + (rel + 2.0 ** -22) * v.abs()
    assert (off <= bound).all(), f"{what}: {(off - bound).max().item()}"


def norm64(x, residual, w, eps, dtype):
    """(h as stored, rstd, y) of the norm in 64 bits from h as stored."""
    h = x if residual is None else (x.float() + residual.float()).to(dtype)
    hd = h.double()
    rstd = 1.0 / torch.sqrt(hd.square().mean(1) + eps)
    y = hd * rstd[:, None]
    return h, rstd, y if w is None else y * w.double()


def quantize(x, rows, fp8, pad_to=16):
    """(q, s) of x by plain torch operations in 64 bits, rows 16-byte aligned."""
    s = scale64(x, rows, fp8).float()
    v = (x.double() / spread(s, rows, x.shape)).clamp(-FP8_MAX[fp8], FP8_MAX[fp8]).float().to(fp8)
    buf = torch.zeros((x.shape[0], -(-x.shape[1] // pad_to) * pad_to), dtype=torch.uint8, device=x.device)
    buf[:, : x.shape[1]] = v.view(torch.uint8)
    return buf.view(fp8)[:, : x.shape[1]], s


def linear64(xq, xs, wq, ws, bias, act):
    """(Y, sum of the products' magnitudes, value before the activation) in 64 bits."""
    rows = 1 if ws.shape[0] == wq.shape[0] else GROUP
    x = xq.float().double() * spread(xs, 1, xq.shape)
    w = wq.float().double() * spread(ws, rows, wq.shape)
    z, mag = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    y = z
    if act == 1:
        y = torch.where(z < 0, torch.zeros_like(z), z)
    elif act == 2:
        y = z * 0.5 * torch.erfc(-z / 2.0 ** 0.5)
    return y, mag, z


def check_linear(Y, ref, K, act, what=""):
    """The kernel's sums: 128 exact products of a block added in fp32 (each of at
    most 132 additions may truncate, 2^-23 of the magnitudes), then ceil(K / 128)
    scaled blocks, the splits and the bias (2^-23 each). GELU: its slope is
    below 1.13, erff is good to 2 ulp and 1 + erf loses up to 2^-23 absolutely, which
    v / 2 multiplies. Then one rounding to Y's type."""
    y, mag, z = ref
    bound = (132 + groups(K) + 12) * 2.0 ** -23 * mag
    if act == 2:
        bound = 1.13 * bound + 4 * 2.0 ** -23 * z.abs()
    r, tiny = ROUND[Y.dtype]
    bound = bound + r * (y.abs() + bound) + tiny
    off = (Y.double() - y).abs()
    assert torch.isfinite(Y.float()).all(), what
    assert (off <= bound).all(), f"{what}: worst {((off - bound).max()).item()} of {mag.max().item()}"
