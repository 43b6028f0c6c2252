"""The feed-forward example: norm, 8-bit up projection, pruned down projection, and
the gradients of the first two, against plain 64-bit forms of the unquantised block."""
import os
import sys

import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


# one token, a few, a ragged prompt
@pytest.mark.parametrize("T", [1, 16, 200])
def test_block(T):
    from fp8_ffn import FeedForward
    D, F = 512, 1024
    ffn = FeedForward(D, F, V=64, M=8)
    g = torch.Generator(device="cuda").manual_seed(T)
    x, residual, dz, later = ((s * torch.randn(T, n, generator=g, device="cuda")).half()
                              for s, n in ((1, D), (1, D), (0.01, F), (0.01, D)))
    y, h = ffn.forward(x, residual, ffn.buffers(T))
    dh, dweight, dwu = ffn.train_step(x, residual, dz, later)
    assert vnm.vnm_get_status(ffn.down) == vnm.VNM_OK

    down = torch.empty((D, F), dtype=torch.float16, device="cuda")
    vnm.vnm_decompress(ffn.down, down)
    h64 = h.double().requires_grad_(True)
    w64, up = ffn.norm_weight.double().requires_grad_(True), ffn.up.double().requires_grad_(True)
    assert torch.equal(h, (x.float() + residual.float()).half())
    yn = h64 / torch.sqrt(h64.square().mean(1, keepdim=True) + ffn.eps) * w64
    z = yn @ up.t()
    a = z.detach() + ffn.up_bias.double()
    want = (a * 0.5 * torch.erfc(-a / 2 ** 0.5)) @ down.double().t()
    z.backward(dz.double())

    # each 8-bit product has two operands rounded to 2^-4 (e4m3) or 2^-3 (e5m2) at most, at
    # random: a few hundredths of the result's norm; 16 bits elsewhere
    def far(got, ref):
        return ((got.double() - ref).norm() / ref.norm()).item()

    assert far(y, want) < 0.1
    assert far(dh, h64.grad + later.double()) < 0.12
    assert far(dweight, w64.grad) < 0.12
    assert far(dwu, up.grad) < 0.12
