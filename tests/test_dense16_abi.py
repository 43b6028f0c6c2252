"""The dense 16-bit entry points without a GPU: sizes, and argument checks that fail before any CUDA call."""
import ctypes

import pytest

from test_abi import libvnm  # noqa: F401  (fixture)

P = 256       # an aligned pointer that is never followed
INVALID = 1


def _call(lib, name, order, defaults, **change):
    return getattr(lib, name)(*[{**defaults, **change}[k] for k in order])


DENSE = "x ld_x xt w ld_w wt type T R K bias b_type act res ld_r y ld_y y_type status stream".split()
DENSE_OK = dict(x=P, ld_x=64, xt=0, w=P, ld_w=64, wt=0, type=0, T=4, R=32, K=64, bias=P, b_type=0, act=3, res=P, ld_r=32, y=P + 512,
                ld_y=32, y_type=0, status=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(type=1), dict(type=3), dict(y_type=2), dict(y_type=5), dict(T=-1), dict(R=-1), dict(K=-1), dict(K=1 << 31), dict(xt=2),
    dict(wt=-1), dict(x=None), dict(x=P + 8), dict(w=None), dict(w=P + 2), dict(ld_x=63), dict(ld_x=68), dict(ld_w=56), dict(ld_w=68),
    dict(xt=1, ld_x=0), dict(wt=1, ld_w=24), dict(b_type=3), dict(bias=P + 1), dict(act=4), dict(act=-1), dict(y=None), dict(y=P + 1),
    dict(y_type=1, y=P + 2), dict(ld_y=31), dict(res=P + 1), dict(ld_r=31), dict(status=P + 1), dict(res=P + 512, ld_r=40)])
def test_dense_refusals(libvnm, change):  # noqa: F811
    assert _call(libvnm, "vnm_dense_linear", DENSE, DENSE_OK, **change) == INVALID


@pytest.mark.parametrize("change", [dict(T=0), dict(R=0), dict(T=0, x=None, w=None, y=None)])
def test_dense_without_work(libvnm, change):  # noqa: F811
    assert _call(libvnm, "vnm_dense_linear", DENSE, DENSE_OK, **change) == 0


GATED = ("x ld_x wg ld_wg wu ld_wu type T F K act y ld_y keep g ld_g gs gs_rs gs_cs u ld_u us us_rs us_cs status stream").split()
GATED_OK = dict(x=P, ld_x=64, wg=P, ld_wg=64, wu=P, ld_wu=64, type=2, T=4, F=32, K=64, act=3, y=P, ld_y=32, keep=2, g=P, ld_g=32, gs=P,
                gs_rs=1, gs_cs=1, u=P, ld_u=32, us=P, us_rs=1, us_cs=1, status=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(type=1), dict(keep=4), dict(keep=-1), dict(act=4), dict(T=-1), dict(F=1 << 31), dict(x=P + 4), dict(ld_x=60), dict(wg=None),
    dict(wu=P + 8), dict(ld_wu=63), dict(y=None), dict(ld_y=31), dict(g=None), dict(u=None), dict(gs=None), dict(us=P + 2),
    dict(ld_g=31), dict(keep=1, u=P + 1), dict(status=P + 2)])
def test_gated_refusals(libvnm, change):  # noqa: F811
    assert _call(libvnm, "vnm_gated_linear", GATED, GATED_OK, **change) == INVALID


@pytest.mark.parametrize("change", [dict(T=0), dict(F=0)])
def test_gated_without_work(libvnm, change):  # noqa: F811
    assert _call(libvnm, "vnm_gated_linear", GATED, GATED_OK, **change) == 0


BACK = ("dy ld_dy x ld_x wg ld_wg wu ld_wu type T F K act keep g ld_g gs gs_rs gs_cs u ld_u us us_rs us_cs dx ld_dx dwg dwu ld_dw "
        "w_type accumulate h ld_h ws ws_bytes status stream").split()
BACK_OK = dict(dy=P, ld_dy=30, x=P, ld_x=64, wg=P, ld_wg=64, wu=P, ld_wu=64, type=0, T=4, F=30, K=64, act=3, keep=2, g=P, ld_g=30, gs=P,
               gs_rs=1, gs_cs=1, u=P, ld_u=30, us=P, us_rs=1, us_cs=1, dx=P, ld_dx=64, dwg=P, dwu=P + 16, ld_dw=64, w_type=1,
               accumulate=0, h=P + 16, ld_h=30, ws=P, ws_bytes=4 * 4 * 32, status=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(type=1), dict(keep=0), dict(keep=5), dict(act=4), dict(T=-1), dict(w_type=2), dict(accumulate=2), dict(dwu=None), dict(dwg=None),
    dict(dwu=P), dict(dy=None), dict(dy=P + 1), dict(ld_dy=29), dict(x=None), dict(x=P + 8), dict(ld_x=68), dict(wg=None),
    dict(ld_wg=66), dict(wu=P + 2), dict(g=None), dict(gs=None), dict(us=P + 1), dict(ld_u=29), dict(dx=P + 1), dict(ld_dx=63),
    dict(ld_dw=63), dict(dwg=P + 2), dict(h=P + 1), dict(ld_h=29), dict(ws=None), dict(ws=P + 8), dict(ws_bytes=4 * 4 * 32 - 1),
    dict(h=P, ld_h=40), dict(status=P + 1)])
def test_gated_backward_refusals(libvnm, change):  # noqa: F811
    assert _call(libvnm, "vnm_gated_linear_backward", BACK, BACK_OK, **change) == INVALID


def test_gated_backward_without_work(libvnm):  # noqa: F811
    assert _call(libvnm, "vnm_gated_linear_backward", BACK, BACK_OK, dx=None, dwg=None, dwu=None, h=None) == 0
    assert _call(libvnm, "vnm_gated_linear_backward", BACK, BACK_OK, T=0, dwg=None, dwu=None) == 0
    assert _call(libvnm, "vnm_gated_linear_backward", BACK, BACK_OK, K=0, h=None) == 0


def test_gated_backward_workspace_size(libvnm):  # noqa: F811
    n = ctypes.c_size_t()
    for T, F, want in ((0, 5, 0), (3, 30, 4 * 3 * 32), (8192, 11008, 4 * 8192 * 11008)):
        assert libvnm.vnm_gated_linear_backward_workspace_size(T, F, ctypes.byref(n)) == 0 and n.value == want
    assert libvnm.vnm_gated_linear_backward_workspace_size(-1, 4, ctypes.byref(n)) == INVALID
    assert libvnm.vnm_gated_linear_backward_workspace_size(4, 4, None) == INVALID


def test_the_other_layers_still_refuse_silu(libvnm):  # noqa: F811
    assert libvnm.vnm_fp8_linear(P, 64, 0, P, 1, 1, P, 64, 0, P, 1, 1, 128, 4, 32, 64, None, 0, 3, P, 32, 0, None, None) == INVALID
