"""The gated feed-forward example: a training step's outputs and gradients, added up over two
micro-batches, and decoding with the pruned down projection, against plain 64-bit forms."""
import os
import sys

import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def far(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


# one token, a few, a ragged batch
@pytest.mark.parametrize("T", [1, 16, 200])
def test_block(T):
    from gated_ffn import GatedFeedForward
    D, F = 512, 1024
    block = GatedFeedForward(D, F)
    g = torch.Generator(device="cuda").manual_seed(T)
    want = [torch.zeros(s, dtype=torch.float64, device="cuda") for s in ((F, D), (F, D), (D, F))]
    for _ in range(2):
        x, residual, dz = ((s * torch.randn(T, D, generator=g, device="cuda")).half() for s in (1, 1, 0.01))
        z, dh, dweight = block.train_step(x, residual, lambda out: dz)
        h = (x.float() + residual.float()).half().double().requires_grad_(True)
        w = [v.double().requires_grad_(True) for v in (block.gate, block.up, block.down, block.norm_weight)]
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + block.eps) * w[3]
        a = torch.nn.functional.silu(y @ w[0].t()) * (y @ w[1].t())
        ref = a @ w[2].t() + h
        ref.backward(dz.double())
        for total, v in zip(want, w):
            total += v.grad
        # z: a few roundings to fp16, 2^-11 each; the gradients go through the 8-bit checkpoint, 2^-4 at most an element and
        # its half on average over many, in each of two factors
        assert far(z, ref.detach()) < 2.0 ** -9
        assert far(dh, h.grad) < 0.1 and far(dweight, w[3].grad) < 0.1
    for k, total in zip(("gate", "up", "down"), want):
        assert far(block.grad[k], total) < 0.1, k
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK

    out, stream = block.decode(x, residual, block.buffers(T))
    pruned = torch.empty((D, F), dtype=torch.float16, device="cuda")
    vnm.vnm_decompress(block.pruned, pruned)
    assert torch.equal(stream.double(), h.detach())
    assert far(out, a.detach() @ pruned.double().t()) < 2.0 ** -8
