"""Kernels that a norm's backward pass launches, counted in a captured graph."""
import ctypes

import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense_util import DEV  # noqa: E402


def _launches(call):
    """Nodes of the graph that call(stream) is captured into."""
    cu = ctypes.CDLL("libcuda.so.1")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    s, graph, n = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p(), ctypes.c_size_t()
    assert cu.cuStreamBeginCapture_v2(s, 2) == 0  # relaxed
    try:
        call(side)
    finally:
        end = cu.cuStreamEndCapture(s, ctypes.byref(graph))
    assert end == 0
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    cu.cuGraphDestroy(graph)
    return n.value


# rows that stay in registers: dh and dweight in one pass; longer ones: one pass each
@pytest.mark.parametrize("D,both,dweight,dh", [(4096, 2, 2, 1), (20000, 3, 2, 1)])
def test_backward(D, both, dweight, dh):
    T = 40
    x, out, w = (torch.ones((n, D), dtype=torch.float16, device=DEV) for n in (T, T, 1))
    rstd, dw = torch.ones(T, device=DEV), torch.empty(D, device=DEV)
    ws = torch.empty(vnm.vnm_rmsnorm_backward_workspace_size(T, D), dtype=torch.uint8, device=DEV)
    vnm.vnm_rmsnorm_backward(x, x, w[0], rstd, out, dw, workspace=ws)
    for want, args in ((both, (out, dw)), (dweight, (None, dw)), (dh, (out, None))):
        assert _launches(lambda s: vnm.vnm_rmsnorm_backward(x, x, w[0], rstd, *args, workspace=ws, stream=s)) == want
