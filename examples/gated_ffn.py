"""A gated feed-forward block trained with dense 16-bit weights, and used for decoding with its down
projection pruned.

    h, y = rmsnorm(x + residual)         vnm_rmsnorm
    a = SiLU(y . Wg^T) * (y . Wu^T)      vnm_gated_linear: both projections in one kernel, kept in 8 bits for training
    z = a . Wd^T + h                     vnm_dense_linear: the residual stream added in the epilogue

`train_step` is the forward and the backward pass: between them stay h, y, the norm's 1/rms and two bytes a
feature; a is computed again from those, for the down projection's gradient, which is added to the
32-bit gradients of the micro-batches before. `decode` runs the norm and the gated pair
for a few tokens and the down projection on V:N:M-pruned weights (vnm_linear).

Usage: python examples/gated_ffn.py [tokens] [D] [F]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from structured_sparse_matmul_gb300 import vnm  # noqa: E402


class GatedFeedForward:
    def __init__(self, D, F, V=64, M=8, eps=1e-6, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.D, self.F, self.eps, self.device = D, F, eps, device
        self.norm_weight = (1 + 0.1 * torch.randn(D, generator=g, device=device)).half()
        self.gate, self.up = ((0.02 * torch.randn(F, D, generator=g, device=device)).half() for _ in range(2))
        self.down = (0.02 * torch.randn(D, F, generator=g, device=device)).half()
        self.grad = {k: torch.zeros_like(getattr(self, k), dtype=torch.float32) for k in ("gate", "up", "down")}
        self.pruned = vnm.vnm_matrix_alloc(D, F, V, M, torch.device(device, torch.cuda.current_device()))
        vnm.vnm_compress(self.pruned, self.down)

    def train_step(self, x, residual, gradient):
        """Forward, then backward with `gradient(z)`, the gradient of the block's output: (z, dh, dweight of the norm); the
        projections' gradients are added to ``grad``."""
        T, D, F, half = x.shape[0], self.D, self.F, dict(dtype=torch.float16, device=self.device)
        h, y, z, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty(T, device=self.device)
        a = torch.empty((T, F), **half)
        kept = {k: torch.empty((T, F), dtype=torch.float8_e4m3fn, device=self.device) for k in ("g", "u")}
        kept.update({k: torch.empty((T, -(-F // 128)), device=self.device) for k in ("g_scale", "u_scale")})
        vnm.vnm_rmsnorm(x, self.norm_weight, self.eps, residual=residual, h=h, y=y, rstd=rstd)
        vnm.vnm_gated_linear(y, self.gate, self.up, a, **kept)
        vnm.vnm_dense_linear(a, self.down, z, residual=h)
        del a

        dz = gradient(z)
        da, dy, dh, hidden = torch.empty((T, F), **half), torch.empty_like(x), torch.empty_like(x), torch.empty((T, F), **half)
        dweight = torch.empty(D, device=self.device)
        vnm.vnm_dense_linear(dz, self.down.t(), da)  # dz . Wd
        vnm.vnm_gated_linear_backward(da, y, self.gate, self.up, **kept, dx=dy, dwg=self.grad["gate"], dwu=self.grad["up"], h=hidden,
                                      accumulate=True)
        vnm.vnm_dense_linear(dz.t(), hidden.t(), self.grad["down"], residual=self.grad["down"])  # + dz^T . a
        vnm.vnm_rmsnorm_backward(dy, h, self.norm_weight, rstd, dh, dweight, dresidual=dz)
        return z, dh, dweight

    def buffers(self, T):
        """What a decode loop keeps for T tokens."""
        half = dict(dtype=torch.float16, device=self.device)
        n = vnm.vnm_linear_workspace_size(self.pruned, T)
        return dict(h=torch.empty((T, self.D), **half), y=torch.empty((T, self.D), **half), a=torch.empty((T, self.F), **half),
                    z=torch.empty((T, self.D), **half), workspace=torch.empty(n, dtype=torch.uint8, device=self.device) if n else None)

    def decode(self, x, residual, b):
        """(z, h): the pruned block's output, to be added to the residual stream h by the next norm, in b's buffers."""
        vnm.vnm_rmsnorm(x, self.norm_weight, self.eps, residual=residual, h=b["h"], y=b["y"])
        vnm.vnm_gated_linear(b["y"], self.gate, self.up, b["a"])
        vnm.vnm_linear(self.pruned, b["a"], b["z"], workspace=b["workspace"])
        return b["z"], b["h"]


def main():
    T, D, F = (int(v) for v in (sys.argv[1:] + ["256", "1024", "4096"][len(sys.argv) - 1:]))
    block = GatedFeedForward(D, F)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, residual = (torch.randn(T, D, generator=g, device="cuda").half() for _ in range(2))
    z, dh, dweight = block.train_step(x, residual, lambda out: 0.01 * out)
    few = min(T, 4)
    out, _ = block.decode(x[:few], residual[:few], block.buffers(few))
    assert vnm.vnm_get_status(block.pruned) == vnm.VNM_OK and vnm.vnm_dense_get_status() == vnm.VNM_OK
    norms = ", ".join(f"|d{k}| = {v.norm().item():.4f}" for k, v in block.grad.items())
    print(f"{T} tokens, D = {D}, F = {F}: |z| = {z.float().norm().item():.3f}, |dh| = {dh.float().norm().item():.4f}, "
          f"|dweight| = {dweight.norm().item():.4f}, {norms}; {few} decoded: |z| = {out.float().norm().item():.4f}")


if __name__ == "__main__":
    main()
