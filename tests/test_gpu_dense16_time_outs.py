"""A stage that never arrives in the gated pair's kernels and in its backward pass's two grids: every wait runs out, the
warps that share a barrier leave it together, the error is kept, and the next call is right."""
import time

import pytest
import torch

from structured_sparse_matmul_gb300 import vnm

pytestmark = pytest.mark.gpu

from dense16_util import BF16, DEV, F16, NONE, generator, pitched, whole  # noqa: E402
from dense16_shapes import SMS  # noqa: E402
from dense_util import check_quantized  # noqa: E402
from test_gpu_gated import E4M3, E5M2, groups, layer  # noqa: E402


def _sms():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sms != SMS:
        pytest.skip(f"the shapes are for {SMS} SMs")


def _timed(call):
    """The call's error, its waits bounded: one runs out after a second, and a few follow one another."""
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK
    t0 = time.time()
    call()
    code = vnm.vnm_dense_get_status()
    assert time.time() - t0 < 30
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK
    return code


# (pairs of CTAs: in a first tile, in a later tile, in a later chunk of K; K over pairs; clusters of two narrow tiles, with and
# without splits of K)
@pytest.mark.parametrize("plan,T,F,K,skips,keep", [
    ((0, 256, 1), 3100, 2600, 200, (0, 3, 9), E4M3), ((0, 256, 1), 2048, 2048, 4096, (2, 20, 33, 50, 63), E4M3),
    ((0, 256, 1), 3100, 2600, 200, (9,), E5M2), ((0, 256, 2), 606, 965, 1116, (4,), E5M2), ((0, 256, 4), 911, 344, 1263, (2,), E4M3),
    ((128, 0, 1), 366, 2434, 3715, (3, 30), E4M3), ((16, 0, 2), 272, 197, 746, (4,), E4M3), ((64, 0, 4), 370, 286, 2542, (0, 7), E5M2)])
def test_8_bit_checkpoints(plan, T, F, K, skips, keep):
    _sms()
    assert vnm.vnm_testing_dense_plan(3, T, F, K, SMS, keep=2 if keep == E4M3 else 3) == plan
    x, wg, wu = layer(generator(T, F, K, 41), T, F, K, F16)
    Y = torch.empty((T, F), dtype=F16, device=DEV)
    kept = {k: torch.empty((T, F), dtype=keep, device=DEV) for k in "gu"}
    kept.update({k + "_scale": torch.empty((T, groups(F)), device=DEV) for k in "gu"})
    G, U = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    for skip in skips:
        assert _timed(lambda: vnm.vnm_testing_gated_linear_skip_stage(x, wg, wu, Y, skip, act=NONE, **kept)) == vnm.VNM_ERR_TIMEOUT
        vnm.vnm_gated_linear(x, wg, wu, Y, act=NONE, **kept)
        assert vnm.vnm_dense_get_status() == vnm.VNM_OK
        check_quantized(kept["g"], kept["g_scale"], G, 1, 0.0)
        check_quantized(kept["u"], kept["u_scale"], U, 1, 0.0)
        assert torch.equal(Y, (G * U).float().half())


@pytest.mark.parametrize("plan,T,F,K,skip", [
    ((0, 192, 1), 3928, 261, 3, 0), ((0, 256, 1), 3100, 2600, 200, 9), ((0, 256, 2), 868, 802, 3063, 5), ((32, 0, 4), 292, 137, 1168, 2)])
@pytest.mark.parametrize("keep", [False, True])
def test_other_checkpoints(plan, T, F, K, skip, keep):
    x, wg, wu = layer(generator(T, F, K, 42), T, F, K, BF16)
    Y, a, b = (torch.empty((T, F), dtype=BF16, device=DEV) for _ in range(3))
    kept = dict(g=a, u=b) if keep else {}
    own = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert _timed(lambda: vnm.vnm_testing_gated_linear_skip_stage(x, wg, wu, Y, skip, act=NONE, **kept)) == vnm.VNM_ERR_TIMEOUT
    assert _timed(lambda: vnm.vnm_testing_gated_linear_skip_stage(x, wg, wu, Y, skip, act=NONE, status=own, **kept)) == vnm.VNM_OK
    assert own[0].item() == vnm.VNM_ERR_TIMEOUT
    vnm.vnm_gated_linear(x, wg, wu, Y, act=NONE, **kept)
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK
    assert torch.equal(Y, ((x.double() @ wg.double().t()) * (x.double() @ wu.double().t())).float().bfloat16())


# (both products by narrow tiles; dX by narrow tiles, the weights by pairs; both by pairs; K over pairs)
@pytest.mark.parametrize("T,F,K", [(42, 1576, 125), (736, 1280, 149), (1397, 587, 2792), (1024, 4096, 1024)])
@pytest.mark.parametrize("skip_dx,skip_dw", [(1, -1), (-1, 0), (0, 0)])
def test_grids_side_by_side(T, F, K, skip_dx, skip_dw):
    """The grid that did not lose a stage has the right values, and what follows follows both."""
    g = generator(T, F, K, 43)
    dy, x, wg, wu = (pitched(whole(g, *s, BF16, 1)) for s in ((T, F), (T, K), (F, K), (F, K)))
    gate, up = (whole(g, T, F, BF16, 1) for _ in range(2))
    ws = torch.empty(vnm.vnm_gated_linear_backward_workspace_size(T, F), dtype=torch.uint8, device=DEV)
    dG, dU = (dy * up).double(), (dy * gate).double()  # (of whole numbers up to 1: exact)
    want = (dG @ wg.double() + dU @ wu.double()).float().bfloat16(), (dG.t() @ x.double()).float(), (dU.t() @ x.double()).float()
    out = [torch.full(v.shape, float("nan"), dtype=v.dtype, device=DEV) for v in want]
    call = lambda: vnm.vnm_testing_gated_linear_backward_skip_stage(dy, x, wg, wu, gate, up, *out, ws, skip_dx, skip_dw, act=NONE)
    assert _timed(call) == vnm.VNM_ERR_TIMEOUT
    if skip_dx < 0:
        assert torch.equal(out[0], want[0])
    if skip_dw < 0:
        assert torch.equal(out[1], want[1]) and torch.equal(out[2], want[2])
    vnm.vnm_gated_linear_backward(dy, x, wg, wu, gate, up, act=NONE, dx=out[0], dwg=out[1], dwu=out[2], workspace=ws)
    assert vnm.vnm_dense_get_status() == vnm.VNM_OK
    assert all(torch.equal(a, b) for a, b in zip(out, want))
