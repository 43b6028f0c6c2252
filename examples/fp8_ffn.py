"""A transformer's feed-forward block with a dense 8-bit up projection and a
pruned down projection, as a decode loop and a training step run it.

    h, xq = rmsnorm(x + residual)        vnm_rmsnorm: 8-bit form of y and the residual stream in one pass
    a = GELU(xq . Wu^T + bu)             vnm_fp8_linear: block-scaled 8-bit weights (F x D)
    y = a . Wd^T                         vnm_linear: V:N:M-pruned weights (D x F)

`train_step` adds the backward pass of the first two lines: the gradients of the
residual stream, of the norm's weight and of Wu, the products again in 8 bits.

Usage: python examples/fp8_ffn.py [tokens] [D] [F]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from structured_sparse_matmul_gb300 import vnm  # noqa: E402

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def fp8_matrix(rows, cols, fp8, device):
    """An 8-bit matrix whose rows are 16-byte aligned, as vnm_fp8_linear reads them."""
    return torch.zeros((rows, -(-cols // 16) * 16), dtype=torch.uint8, device=device).view(fp8)[:, :cols]


def scales(rows, cols, device):
    return torch.empty((rows, -(-cols // 128)), device=device)


def quantized(x, block_rows, fp8, plain=True, transposed=False):
    """(q, s, qt, st) of x; those not asked for are None."""
    R, C = x.shape
    q = s = qt = st = None
    if plain:
        q, s = fp8_matrix(R, C, fp8, x.device), scales(-(-R // block_rows), C, x.device)
    if transposed:
        qt, st = fp8_matrix(C, R, fp8, x.device), scales(-(-C // block_rows), R, x.device)
    vnm.vnm_fp8_quantize(x, q, s, qt, st, block_rows=block_rows)
    return q, s, qt, st


class FeedForward:
    """Weights of the block: the up projection in 8 bits (128 x 128 blocks), the down
    projection pruned to 2 of every M columns in blocks of V rows."""

    def __init__(self, D, F, V=64, M=8, eps=1e-6, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.D, self.F, self.eps, self.device = D, F, eps, device
        self.norm_weight = (1 + 0.1 * torch.randn(D, generator=g, device=device)).half()
        self.up = (0.02 * torch.randn(F, D, generator=g, device=device)).half()
        self.up_bias = (0.1 * torch.randn(F, generator=g, device=device)).half()
        self.down_dense = (0.02 * torch.randn(D, F, generator=g, device=device)).half()
        self.down = vnm.vnm_matrix_alloc(D, F, V, M, torch.device(device, torch.cuda.current_device()))
        vnm.vnm_compress(self.down, self.down_dense)
        self.wq, self.ws, self.wtq, self.wts = quantized(self.up, 128, E4M3, transposed=True)

    def buffers(self, T):
        """What a decode loop keeps: outputs and scratch for T tokens."""
        half = dict(dtype=torch.float16, device=self.device)
        n = vnm.vnm_linear_workspace_size(self.down, T)
        return dict(h=torch.empty((T, self.D), **half), xq=fp8_matrix(T, self.D, E4M3, self.device),
                    xs=scales(T, self.D, self.device), a=torch.empty((T, self.F), **half),
                    y=torch.empty((T, self.D), **half),
                    workspace=torch.empty(n, dtype=torch.uint8, device=self.device) if n else None)

    def forward(self, x, residual, b):
        """(y, h): the block's output and the updated residual stream, in b's buffers."""
        vnm.vnm_rmsnorm(x, self.norm_weight, self.eps, residual=residual, h=b["h"], q=b["xq"], q_scale=b["xs"])
        vnm.vnm_fp8_linear(b["xq"], b["xs"], self.wq, self.ws, b["a"], bias=self.up_bias, act=vnm.VNM_ACT_GELU)
        vnm.vnm_linear(self.down, b["a"], b["y"], workspace=b["workspace"])
        return b["y"], b["h"]

    def train_step(self, x, residual, dz, dh_later):
        """Gradients of the norm and the up projection for dz, the gradient of
        z = y_norm . Wu^T (before the bias's activation), and dh_later, what reaches the
        residual stream past the norm: (dh, dweight of the norm, dWu)."""
        T, D, F, dev = x.shape[0], self.D, self.F, self.device
        h, yn = torch.empty_like(x), torch.empty_like(x)
        rstd = torch.empty(T, device=dev)
        vnm.vnm_rmsnorm(x, self.norm_weight, self.eps, residual=residual, h=h, y=yn, rstd=rstd)
        _, _, ytq, yts = quantized(yn, 1, E4M3, plain=False, transposed=True)  # groups along the tokens
        dq, ds, dtq, dts = quantized(dz, 1, E5M2, transposed=True)
        dyn = torch.empty((T, D), dtype=x.dtype, device=dev)
        vnm.vnm_fp8_linear(dq, ds, self.wtq, self.wts, dyn)  # dz . Wu
        dwu = torch.empty((F, D), device=dev)
        vnm.vnm_fp8_linear(dtq, dts, ytq, yts, dwu)          # dz^T . y_norm
        dh, dweight = torch.empty_like(x), torch.empty(D, device=dev)
        vnm.vnm_rmsnorm_backward(dyn, h, self.norm_weight, rstd, dh, dweight, dresidual=dh_later)
        return dh, dweight, dwu


def main():
    T, D, F = (int(v) for v in (sys.argv[1:] + ["16", "1024", "4096"][len(sys.argv) - 1:]))
    ffn = FeedForward(D, F)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, residual, dz, dh = ((s * torch.randn(T, n, generator=g, device="cuda")).half()
                           for s, n in ((1, D), (1, D), (0.01, F), (0.01, D)))
    b = ffn.buffers(T)
    y, h = ffn.forward(x, residual, b)
    grads = ffn.train_step(x, residual, dz, dh)
    assert vnm.vnm_get_status(ffn.down) == vnm.VNM_OK and vnm.vnm_fp8_linear_get_status() == vnm.VNM_OK
    print(f"{T} tokens, D = {D}, F = {F}: |y| = {y.float().norm().item():.4f}, "
          f"|dh| = {grads[0].float().norm().item():.4f}, |dw| = {grads[1].norm().item():.4f}, |dWu| = {grads[2].norm().item():.4f}")


if __name__ == "__main__":
    main()
